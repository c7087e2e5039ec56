"""ctypes binding of the page operations (declarations in include/entmaxkv_pages.h): counting, forking, growing,
compacting and copying the pages of a paged cache, bf16 or 4-bit, of any number of layers that share one page table.

There is no allocator object: a block is in use when the page table reaches it (or ``hold`` keeps it), and a sequence
is freed by setting its length to 0 or forking its row away.  Everything runs on the device and on the caller's
stream.  Argument marshalling only, as in ``native``.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import native as nv
from .kv4 import arg, current, on_current_device, room

EXPORTED = ("entmaxkv_pages_workspace_size", "entmaxkv_pages_refs", "entmaxkv_pages_fork", "entmaxkv_pages_grow",
            "entmaxkv_pages_compact", "entmaxkv_pages_copy")
STATUS_NO_BLOCK, STATUS_BAD_ROW = 64, 128
MAX_BUFFERS = 256


class _CBuffers(C.Structure):
    _fields_ = [("count", C.c_int32), ("block_bytes", C.c_int64), ("base", C.POINTER(C.c_void_p))]


class Buffers:
    """The caches (or metadata buffers) that share one page table, as the calls take them: contiguous tensors of one
    shape and dtype whose first dimension is the block (a 1-D uint8 tensor, as kv4.alloc_cache gives, is cut into
    num_blocks equal blocks).  Made once and used for every call; it keeps the tensors alive."""

    def __init__(self, tensors, num_blocks=None):
        self.tensors = tuple(tensors)
        if len(self.tensors) > MAX_BUFFERS:
            raise ValueError(f"at most {MAX_BUFFERS} buffers, got {len(self.tensors)}")
        if num_blocks is not None and num_blocks < 1:
            raise ValueError(f"buffers: at least one block, got {num_blocks}")
        for t in self.tensors:
            if t.numel() == 0 or t.dim() == 0:
                raise ValueError("buffers: must hold at least one block")
            if t.device.type != "cuda" and not t.is_pinned():
                raise ValueError("buffers: CUDA or pinned host tensors")
            if not t.is_contiguous():
                raise ValueError("buffers: must be contiguous")
            if t.shape != self.tensors[0].shape or t.dtype != self.tensors[0].dtype:
                raise ValueError("buffers: must have one shape and dtype")
            if t.device != self.tensors[0].device:
                raise ValueError("buffers: must live on one device")
        size = self.tensors[0].numel() * self.tensors[0].element_size() if self.tensors else 0
        self.nbytes = size
        self.num_blocks = num_blocks if num_blocks else self.tensors[0].shape[0] if self.tensors else 0
        if self.tensors and size % self.num_blocks:
            raise ValueError(f"buffers: {size} bytes are not {self.num_blocks} equal blocks")
        self.base = (C.c_void_p * max(1, len(self.tensors)))(*[t.data_ptr() for t in self.tensors])
        self.c = _CBuffers(len(self.tensors), size // self.num_blocks if self.tensors else 0, self.base)
        self.ref = C.byref(self.c)
        self.device = self.tensors[0].get_device() if self.tensors else -1  # -1: host memory

    def on(self, device):
        """The buffers have to live on the current device `device`, or in host memory."""
        if self.device >= 0 and self.device != device:
            on_current_device(self.tensors[0])


_ready = None


def lib():
    global _ready
    if _ready is None:
        L = nv.lib()
        vp, i32, sz, sp, bp = C.c_void_p, C.c_int32, C.c_size_t, C.POINTER(nv.Shape), C.POINTER(_CBuffers)
        L.entmaxkv_pages_workspace_size.restype = sz
        L.entmaxkv_pages_workspace_size.argtypes = [sp]
        L.entmaxkv_pages_refs.argtypes = [sp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.entmaxkv_pages_fork.argtypes = [sp, vp, vp, vp, vp, vp, vp, bp, bp, bp, vp, sz, vp]
        L.entmaxkv_pages_grow.argtypes = [sp, vp, vp, vp, vp, vp, sz, vp]
        L.entmaxkv_pages_compact.argtypes = [sp, vp, vp, vp, vp, bp, vp, vp, vp, sz, vp]
        L.entmaxkv_pages_copy.argtypes = [bp, i32, bp, i32, vp, vp, i32, vp]
        _ready = L
    return _ready


def workspace_size(shape: nv.Shape) -> int:
    return lib().entmaxkv_pages_workspace_size(C.byref(shape))


def alloc_workspace(shape: nv.Shape, device) -> torch.Tensor:
    n = workspace_size(shape)
    if n == (1 << 64) - 1:
        raise nv.EntmaxKVError("entmaxkv_pages_workspace_size", -2, "invalid shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _i32(t, shape, name, device):
    return arg(t, torch.int32, shape, name, device)


def _buffers(b, shape, name, device):
    if b is None:
        return None
    if not isinstance(b, Buffers):
        raise TypeError(f"{name}: expected pages.Buffers")
    if b.tensors and b.num_blocks != shape.num_blocks:
        raise ValueError(f"{name}: {b.num_blocks} blocks, the shape has {shape.num_blocks}")
    b.on(device)
    return b.ref


def _metas(b, shape, name, device):
    if b is None:
        return None
    if not isinstance(b, Buffers):
        raise TypeError(f"{name}: expected pages.Buffers")
    if b.tensors and b.nbytes != nv.meta_bytes(shape):
        raise ValueError(f"{name}: metadata buffers of {nv.meta_bytes(shape)} bytes expected, got {b.nbytes}")
    b.on(device)
    return b.ref


def entmaxkv_pages_refs(shape, page_table, seq_lens, refs=None, n_free=None, hold=None, *, workspace, stream=None):
    """refs (int32 [num_blocks]): rows that reach each block, plus holds; n_free (int32 [1]): blocks without any."""
    B, nb = shape.B, shape.num_blocks
    dev, st = current(stream)
    nv._check("entmaxkv_pages_refs", lib().entmaxkv_pages_refs(
        C.byref(shape), _i32(page_table, (B, shape.max_pages), "page_table", dev),
        _i32(seq_lens, (B,), "seq_lens", dev), _i32(hold, (nb,), "hold", dev), _i32(refs, (nb,), "refs", dev),
        _i32(n_free, (1,), "n_free", dev), room(workspace, dev), workspace.numel(), st))


def entmaxkv_pages_fork(shape, parent, table_in, lens_in, table_out, lens_out, buffers, meta_in=None, meta_out=None,
                        hold=None, *, workspace, stream=None):
    """Row b of the new table continues row parent[b] of the old one (-1: empty); full pages are shared, partial last
    pages copied in every buffer; metadata buffers follow their rows.  In place when the out tensors are the in ones."""
    B, table = shape.B, (shape.B, shape.max_pages)
    dev, st = current(stream)
    nv._check("entmaxkv_pages_fork", lib().entmaxkv_pages_fork(
        C.byref(shape), _i32(parent, (B,), "parent", dev), _i32(table_in, table, "table_in", dev),
        _i32(lens_in, (B,), "lens_in", dev), _i32(hold, (shape.num_blocks,), "hold", dev),
        _i32(table_out, table, "table_out", dev), _i32(lens_out, (B,), "lens_out", dev),
        _buffers(buffers, shape, "buffers", dev), _metas(meta_in, shape, "meta_in", dev),
        _metas(meta_out, shape, "meta_out", dev), room(workspace, dev), workspace.numel(), st))


def entmaxkv_pages_grow(shape, n_add, page_table, seq_lens, hold=None, *, workspace, stream=None):
    """Sequence b grows by n_add[b] tokens, in place: new pages get the lowest free blocks."""
    B = shape.B
    dev, st = current(stream)
    nv._check("entmaxkv_pages_grow", lib().entmaxkv_pages_grow(
        C.byref(shape), _i32(n_add, (B,), "n_add", dev), _i32(hold, (shape.num_blocks,), "hold", dev),
        _i32(page_table, (B, shape.max_pages), "page_table", dev), _i32(seq_lens, (B,), "seq_lens", dev),
        room(workspace, dev), workspace.numel(), st))


def entmaxkv_pages_compact(shape, table_in, seq_lens, table_out, buffers, remap, n_live, hold=None, *, workspace,
                           stream=None):
    """Used blocks move below n_live, their count; the table follows (table_out may be table_in)."""
    table, nb = (shape.B, shape.max_pages), (shape.num_blocks,)
    dev, st = current(stream)
    nv._check("entmaxkv_pages_compact", lib().entmaxkv_pages_compact(
        C.byref(shape), _i32(table_in, table, "table_in", dev), _i32(seq_lens, (shape.B,), "seq_lens", dev),
        _i32(hold, nb, "hold", dev), _i32(table_out, table, "table_out", dev), _buffers(buffers, shape, "buffers", dev),
        _i32(remap, nb, "remap", dev), _i32(n_live, (1,), "n_live", dev), room(workspace, dev), workspace.numel(), st))


def entmaxkv_pages_copy(src, dst, src_ids, dst_ids, stream=None):
    """Block dst_ids[i] of every dst buffer := block src_ids[i] of the src buffer of the same number.  Either side
    may be pinned host memory."""
    dev, st = current(stream)
    for b, name in ((src, "src"), (dst, "dst")):
        if not isinstance(b, Buffers):
            raise TypeError(f"{name}: expected pages.Buffers")
        b.on(dev)
    if not isinstance(src_ids, torch.Tensor) or src_ids.dim() != 1:
        raise ValueError("src_ids: expected one dimension")
    ids = (src_ids.shape[0],)
    nv._check("entmaxkv_pages_copy", lib().entmaxkv_pages_copy(
        src.ref, src.num_blocks, dst.ref, dst.num_blocks, _i32(src_ids, ids, "src_ids", dev),
        _i32(dst_ids, ids, "dst_ids", dev), ids[0], st))
