"""ctypes binding of the 4-bit paged cache (declarations in include/entmaxkv_kv4.h).

Rows go in with ``entmaxkv_kv4_write`` (a prompt's rows or one token a
sequence, with the metadata of the pages they touch), come back with
``entmaxkv_kv4_read``, and are attended over by ``entmaxkv_kv4_decode``
(softmax or alpha-entmax, over every page or over a selection).  Scores and
selections come from ``native.entmaxkv_score_pages`` and
``native.entmaxkv_select`` as for a bf16 cache.

Argument marshalling only, as in ``native``; beyond its checks, every tensor
has to have the size the shape asks for and live on the current device.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import native as nv

EXPORTED = ("entmaxkv_kv4_bytes", "entmaxkv_kv4_write", "entmaxkv_kv4_read", "entmaxkv_kv4_workspace_size",
            "entmaxkv_kv4_decode")
_ROWS = {torch.bfloat16: 0, torch.float32: 1}

_ready = None


def lib():
    global _ready
    if _ready is None:
        L = nv.lib()
        vp, i32, i64, f32, sz, sp = C.c_void_p, C.c_int32, C.c_int64, C.c_float, C.c_size_t, C.POINTER(nv.Shape)
        L.entmaxkv_kv4_bytes.restype = sz
        L.entmaxkv_kv4_bytes.argtypes = [sp]
        L.entmaxkv_kv4_workspace_size.restype = sz
        L.entmaxkv_kv4_workspace_size.argtypes = [sp]
        L.entmaxkv_kv4_write.argtypes = [sp, vp, vp, i64, vp, i32, vp, vp, vp, vp, vp, vp]
        L.entmaxkv_kv4_read.argtypes = [sp, vp, vp, i64, vp, i32, vp, vp, i32, vp, vp, vp]
        L.entmaxkv_kv4_decode.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp, vp, sz, vp]
        _ready = L
    return _ready


def on_current_device(*tensors):
    """Every CUDA tensor given has to live on the current device (a kernel runs there)."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.is_cuda and t.get_device() != cur:
            raise ValueError(f"tensor on cuda:{t.get_device()}, but the current device is cuda:{cur}")


def sized(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def bytes_of(shape: nv.Shape) -> int:
    """Bytes of one 4-bit cache (keys or values)."""
    return lib().entmaxkv_kv4_bytes(C.byref(shape))


def alloc_cache(shape: nv.Shape, device):
    """(k4, v4), uninitialised."""
    n = bytes_of(shape)
    if n == 0:
        raise nv.EntmaxKVError("entmaxkv_kv4_bytes", -2, "invalid shape")
    return tuple(torch.empty(n, dtype=torch.uint8, device=device) for _ in range(2))


def workspace_size(shape: nv.Shape) -> int:
    return lib().entmaxkv_kv4_workspace_size(C.byref(shape))


def alloc_workspace(shape: nv.Shape, device) -> torch.Tensor:
    n = workspace_size(shape)
    if n == (1 << 64) - 1:
        raise nv.EntmaxKVError("entmaxkv_kv4_workspace_size", -2, "invalid shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _cache_args(shape, k4, v4, page_table, seq_lens):
    n = bytes_of(shape)
    sized(k4, (n,), "k4")
    sized(v4, (n,), "v4")
    sized(page_table, (shape.B, shape.max_pages), "page_table")
    sized(seq_lens, (shape.B,), "seq_lens")
    on_current_device(k4, v4, page_table, seq_lens)


def _rows(shape, x, name, dtypes, pinned_ok):
    """(pointer, row stride) of rows [n, Hkv, d] whose heads are packed; consecutive rows may lie apart."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {x.dtype}")
    if not x.is_cuda and not (pinned_ok and x.device.type == "cpu" and x.is_pinned()):
        raise ValueError(f"{name}: must be a CUDA tensor" + (" or pinned" if pinned_ok else ""))
    if x.dim() != 3 or x.shape[1] != shape.Hkv or x.shape[2] != shape.d:
        raise ValueError(f"{name}: expected [rows, {shape.Hkv}, {shape.d}], got {tuple(x.shape)}")
    if x.stride(2) != 1 or (shape.Hkv > 1 and x.stride(1) != shape.d):
        raise ValueError(f"{name}: the heads of a row must be packed")
    row = shape.Hkv * shape.d
    return C.c_void_p(x.data_ptr()), x.stride(0) if x.shape[0] > 1 else row


def _row_pair(shape, k, v, names, dtypes, row_start, pinned_ok=False):
    pk, sk = _rows(shape, k, names[0], dtypes, pinned_ok)
    pv, sv = _rows(shape, v, names[1], dtypes, pinned_ok)
    if k.shape[0] != v.shape[0] or sk != sv or k.dtype != v.dtype:
        raise ValueError(f"{names[0]} and {names[1]}: expected the same rows, strides and dtype")
    if row_start is None:
        if k.shape[0] != shape.B:
            raise ValueError(f"{names[0]}: one row a sequence ({shape.B}) without row_start, got {k.shape[0]}")
    else:
        sized(row_start, (shape.B + 1,), "row_start")
    on_current_device(k, v, row_start)
    return pk, pv, sk, nv._ptr(row_start, torch.int32, "row_start")


def entmaxkv_kv4_write(shape, k_new, v_new, row_start, page_table, seq_lens, k4, v4, meta=None, stream=None):
    """Rows bf16 [n, Hkv, d] (row b of every sequence b when row_start is None) into the cache, as the last tokens of
    their sequences; with meta, the records of the pages they touch.  Rows may be pinned host tensors."""
    pk, pv, stride, ps = _row_pair(shape, k_new, v_new, ("k_new", "v_new"), (torch.bfloat16,), row_start, True)
    _cache_args(shape, k4, v4, page_table, seq_lens)
    if meta is not None:
        sized(meta, (nv.meta_bytes(shape),), "meta")
        on_current_device(meta)
    nv._check("entmaxkv_kv4_write", lib().entmaxkv_kv4_write(
        C.byref(shape), pk, pv, stride, ps, k_new.shape[0], nv._ptr(page_table, torch.int32, "page_table"),
        nv._ptr(seq_lens, torch.int32, "seq_lens"), nv._ptr(k4, torch.uint8, "k4"), nv._ptr(v4, torch.uint8, "v4"),
        nv._ptr(meta, torch.uint8, "meta"), nv._stream(stream)))


def entmaxkv_kv4_read(shape, k4, v4, row_start, page_table, seq_lens, k_out, v_out, stream=None):
    """The last tokens of every sequence into rows [n, Hkv, d], bf16 or fp32: the inverse of entmaxkv_kv4_write."""
    pk, pv, stride, ps = _row_pair(shape, k_out, v_out, ("k_out", "v_out"), tuple(_ROWS), row_start)
    _cache_args(shape, k4, v4, page_table, seq_lens)
    nv._check("entmaxkv_kv4_read", lib().entmaxkv_kv4_read(
        C.byref(shape), nv._ptr(k4, torch.uint8, "k4"), nv._ptr(v4, torch.uint8, "v4"), stride, ps, k_out.shape[0],
        nv._ptr(page_table, torch.int32, "page_table"), nv._ptr(seq_lens, torch.int32, "seq_lens"),
        _ROWS[k_out.dtype], pk, pv, nv._stream(stream)))


def entmaxkv_kv4_decode(shape, q, k4, v4, page_table, seq_lens, alpha, out, tau_out=None, sel=None, cnt=None, *,
                        workspace, stream=None):
    """Attention of q (bf16 [B, Hq, d]) over the 4-bit cache into out (fp32 [B, Hq, d]): softmax (alpha = 1) or
    alpha-entmax, over the selected pages, or over all of them without sel and cnt."""
    heads = (shape.B, shape.Hq)
    _cache_args(shape, k4, v4, page_table, seq_lens)
    sized(q, heads + (shape.d,), "q")
    sized(out, heads + (shape.d,), "out")
    sized(tau_out, heads, "tau_out")
    sized(sel, heads + (shape.max_pages,), "sel")
    sized(cnt, heads, "cnt")
    on_current_device(q, out, tau_out, sel, cnt, workspace)
    nv._check("entmaxkv_kv4_decode", lib().entmaxkv_kv4_decode(
        C.byref(shape), nv._ptr(q, torch.bfloat16, "q"), nv._ptr(k4, torch.uint8, "k4"),
        nv._ptr(v4, torch.uint8, "v4"), nv._ptr(page_table, torch.int32, "page_table"),
        nv._ptr(seq_lens, torch.int32, "seq_lens"), nv._ptr(sel, torch.int32, "sel"),
        nv._ptr(cnt, torch.int32, "cnt"), float(alpha), nv._ptr(out, torch.float32, "out", pinned_ok=True),
        nv._ptr(tau_out, torch.float32, "tau_out"), nv._ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        nv._stream(stream)))
