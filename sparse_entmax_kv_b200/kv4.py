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


def current(stream):
    """The current device, and the stream to launch on (the current one, unless another is given)."""
    device = torch._C._cuda_getDevice()
    return device, torch._C._cuda_getCurrentRawStream(device) if stream is None else nv._stream(stream)


def arg(t, dtype, shape, name, device, pinned_ok=False):
    """Address of a contiguous tensor of this dtype and shape on the current device `device` (None stays None)."""
    if t is None:
        return None
    try:
        if t.dtype == dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    p = nv._ptr(t, dtype, name, pinned_ok=pinned_ok)
    sized(t, shape, name)
    on_current_device(t)
    return p


def room(workspace, device):
    """Address of a workspace."""
    if isinstance(workspace, torch.Tensor) and workspace.dtype == torch.uint8 and workspace.get_device() == device \
            and workspace.is_contiguous():
        return workspace.data_ptr()
    p = nv._ptr(workspace, torch.uint8, "workspace")
    on_current_device(workspace)
    return p


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


def _cache_bytes(shape):
    return shape.num_blocks * shape.Hkv * shape.page_size * shape.d // 16 * 9


def _meta_bytes(shape):
    return shape.B * shape.Hkv * ((shape.max_pages + 31) // 32) * 384 * shape.d


def _cache_args(shape, k4, v4, page_table, seq_lens, device):
    n = (_cache_bytes(shape),)
    return (arg(k4, torch.uint8, n, "k4", device), arg(v4, torch.uint8, n, "v4", device),
            arg(page_table, torch.int32, (shape.B, shape.max_pages), "page_table", device),
            arg(seq_lens, torch.int32, (shape.B,), "seq_lens", device))


def _rows(shape, x, name, dtypes, pinned_ok):
    """(address, row stride) of rows [n, Hkv, d] whose heads are packed; consecutive rows may lie apart."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {x.dtype}")
    if not x.is_cuda and not (pinned_ok and x.device.type == "cpu" and x.is_pinned()):
        raise ValueError(f"{name}: must be a CUDA tensor" + (" or pinned" if pinned_ok else ""))
    Hkv, d = shape.Hkv, shape.d
    n, row, form = x.shape[0] if x.dim() else 0, Hkv * d, x.stride()
    if x.shape != (n, Hkv, d):
        raise ValueError(f"{name}: expected [rows, {Hkv}, {d}], got {tuple(x.shape)}")
    if form[2] != 1 or (Hkv > 1 and form[1] != d):
        raise ValueError(f"{name}: the heads of a row must be packed")
    return x.data_ptr(), form[0] if n > 1 else row


def _row_pair(shape, k, v, names, dtypes, row_start, stream, pinned_ok=False):
    """Addresses of the key and value rows and their stride, of row_start, the number of rows, device and stream."""
    Hkv, d = shape.Hkv, shape.d
    n = -1
    if isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and k.is_cuda:
        device, st = current(stream)
        form, steps = k.shape, k.stride()
        if len(form) == 3 and form[1] == Hkv and form[2] == d and steps[2] == 1 and (steps[1] == d or Hkv == 1) \
                and k.dtype in dtypes and v.dtype == k.dtype and v.shape == form and v.stride() == steps \
                and k.get_device() == device and v.get_device() == device:
            n, stride, pk, pv = form[0], steps[0], k.data_ptr(), v.data_ptr()
            if n <= 1:
                stride = Hkv * d
    if n < 0:  # pinned rows, or something to refuse
        pk, stride = _rows(shape, k, names[0], dtypes, pinned_ok)
        pv, other = _rows(shape, v, names[1], dtypes, pinned_ok)
        n = k.shape[0]
        if n != v.shape[0] or stride != other or k.dtype != v.dtype:
            raise ValueError(f"{names[0]} and {names[1]}: expected the same rows, strides and dtype")
        device, st = current(stream)
        on_current_device(k, v)
    if row_start is None:
        if n != shape.B:
            raise ValueError(f"{names[0]}: one row a sequence ({shape.B}) without row_start, got {n}")
        return pk, pv, stride, None, n, device, st
    return pk, pv, stride, arg(row_start, torch.int32, (shape.B + 1,), "row_start", device), n, device, st


def entmaxkv_kv4_write(shape, k_new, v_new, row_start, page_table, seq_lens, k4, v4, meta=None, stream=None):
    """Rows bf16 [n, Hkv, d] (row b of every sequence b when row_start is None) into the cache, as the last tokens of
    their sequences; with meta, the records of the pages they touch.  Rows may be pinned host tensors."""
    pk, pv, stride, ps, n, device, st = _row_pair(shape, k_new, v_new, ("k_new", "v_new"), (torch.bfloat16,), row_start,
                                                  stream, True)
    c4k, c4v, pt, sl = _cache_args(shape, k4, v4, page_table, seq_lens, device)
    m = None if meta is None else arg(meta, torch.uint8, (_meta_bytes(shape),), "meta", device)
    rc = lib().entmaxkv_kv4_write(C.byref(shape), pk, pv, stride, ps, n, pt, sl, c4k, c4v, m, st)
    if rc:
        nv._check("entmaxkv_kv4_write", rc)


def entmaxkv_kv4_read(shape, k4, v4, row_start, page_table, seq_lens, k_out, v_out, stream=None):
    """The last tokens of every sequence into rows [n, Hkv, d], bf16 or fp32: the inverse of entmaxkv_kv4_write."""
    pk, pv, stride, ps, n, device, st = _row_pair(shape, k_out, v_out, ("k_out", "v_out"), _ROWS, row_start, stream)
    c4k, c4v, pt, sl = _cache_args(shape, k4, v4, page_table, seq_lens, device)
    rc = lib().entmaxkv_kv4_read(C.byref(shape), c4k, c4v, stride, ps, n, pt, sl, _ROWS[k_out.dtype], pk, pv, st)
    if rc:
        nv._check("entmaxkv_kv4_read", rc)


def entmaxkv_kv4_decode(shape, q, k4, v4, page_table, seq_lens, alpha, out, tau_out=None, sel=None, cnt=None, *,
                        workspace, stream=None):
    """Attention of q (bf16 [B, Hq, d]) over the 4-bit cache into out (fp32 [B, Hq, d]): softmax (alpha = 1) or
    alpha-entmax, over the selected pages, or over all of them without sel and cnt."""
    device, st = current(stream)
    B, Hq = shape.B, shape.Hq
    heads, rows = (B, Hq), (B, Hq, shape.d)
    c4k, c4v, pt, sl = _cache_args(shape, k4, v4, page_table, seq_lens, device)
    ps = pc = None
    if sel is not None:
        ps = arg(sel, torch.int32, (B, Hq, shape.max_pages), "sel", device)
    if cnt is not None:
        pc = arg(cnt, torch.int32, heads, "cnt", device)
    rc = lib().entmaxkv_kv4_decode(
        C.byref(shape), arg(q, torch.bfloat16, rows, "q", device), c4k, c4v, pt, sl, ps, pc, float(alpha),
        arg(out, torch.float32, rows, "out", device, True), arg(tau_out, torch.float32, heads, "tau_out", device),
        room(workspace, device), workspace.numel(), st)
    if rc:
        nv._check("entmaxkv_kv4_decode", rc)
