"""The operators around the expert layer, on torch tensors.

Torch allocates outputs and scratch and supplies the current stream of the
tensors' device; every value is computed by the kernels behind include/moe.h
(``moe_add_rms_norm``, ``moe_sort_*``, ``moe_unsort_*``, ``moe_clip_grad_norm``),
whose entries describe the mathematics, the limits and the errors. Activations
are fp32 or bf16 matrices whose last dimension is contiguous (any row stride).
Wrong devices, types and shapes raise ValueError here; what the library
refuses raises MoEError.
"""
from __future__ import annotations

import array
import ctypes
from typing import Dict, Optional, Sequence

from . import (MOE_BF16, MOE_FP32, MOE_OK, MoEError, load_library, moe_clip_workspace_size,
               moe_norm_bwd_args_t, moe_norm_fwd_args_t, moe_norm_workspace_size, moe_sort_rows_cap,
               moe_sorted_t)

MOE_NORM_PLAIN, MOE_NORM_FP8_BLOCK, MOE_NORM_MXFP8 = 0, 1, 2

_torch = None
_lib = None
_stream = None
_dtypes: Dict[object, int] = {}


def _load():
    global _torch, _lib, _stream
    if _lib is None:
        import torch
        _torch = torch
        _dtypes.update({torch.float32: MOE_FP32, torch.bfloat16: MOE_BF16})
        # the current stream as a number, without a Stream object (2.8 us of a call)
        _stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _lib = load_library()                # last: another thread's call takes it as the sign that the rest is there
    return _lib


def _call(where, dev, fn, *args):
    """fn(*args, the current stream of device dev) with dev current; raises on a status."""
    cuda = _torch.cuda
    if cuda.current_device() == dev:
        st = fn(*args, _stream(dev))
    else:
        with cuda.device(dev):
            st = fn(*args, _stream(dev))
    if st != MOE_OK:
        raise MoEError(st, where)


def _act(t, name, shape=None, like=None):
    """Checks an activation matrix; returns its row stride."""
    sh = t.shape
    if like is None:
        if not t.is_cuda or len(sh) != 2 or t.dtype not in _dtypes:
            raise ValueError(f"{name}: a 2-D fp32 or bf16 CUDA tensor is needed, got {len(sh)}-D {t.dtype} on {t.device}")
    elif t.dtype != like.dtype or t.get_device() != like.get_device():
        raise ValueError(f"{name}: {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")
    if shape is not None and sh != shape:
        raise ValueError(f"{name}: shape {tuple(sh)}, expected {tuple(shape)}")
    ld, one = t.stride()
    rows, H = sh
    if one != 1 and H > 1:
        raise ValueError(f"{name}: the last dimension has to be contiguous")
    return ld if rows > 1 else H


def _vec(t, name, n, dtype, like):
    if t.dtype != dtype or t.numel() != n or t.get_device() != like.get_device() or not t.is_contiguous():
        raise ValueError(f"{name}: {n} contiguous {dtype} values on {like.device} are needed")
    return t.data_ptr()


def _like(x, ldx):
    """A new contiguous matrix of x's shape and type."""
    return _torch.empty_like(x) if ldx == x.shape[1] else _torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _p(t):
    return None if t is None else t.data_ptr()


def add_rms_norm(x, weight, residual=None, *, eps: float = 1e-6, quant: int = MOE_NORM_PLAIN, want_y: bool = True,
                 want_rstd: bool = False, h=None, y=None):
    """``s = x + residual``, ``y = s / rms(s) * weight`` (moe_add_rms_norm).

    Returns a dict with ``h`` (the sum in x's type; only with a residual),
    ``y`` (unless ``want_y`` is false and there is an 8-bit output), ``rstd``
    (with ``want_rstd``; the backward needs it) and, for an 8-bit ``quant``,
    ``codes`` (uint8, E4M3) and ``scales`` (fp32 rows x H/128, or the uint8
    scale atoms of MXFP8). ``h`` and ``y`` may be given, x and the residual
    themselves included."""
    lib = _load()
    t = _torch
    ldx = _act(x, "x")
    shape = rows, H = x.shape
    a = moe_norm_fwd_args_t(x.data_ptr(), None, _vec(weight, "weight", H, t.float32, x))
    a.ldx = ldx
    out = {}
    if residual is not None:
        a.ldr = _act(residual, "residual", shape, x)
        a.residual = residual.data_ptr()
        if h is None:
            h = _like(x, ldx)
            a.ldh = H
        else:
            a.ldh = _act(h, "h", shape, x)
        a.h = h.data_ptr()
        out["h"] = h
    elif h is not None:
        raise ValueError("h: without a residual there is no sum to store")
    if want_y or y is not None or quant == MOE_NORM_PLAIN:
        if y is None:
            y = _like(x, ldx)
            a.ldy = H
        else:
            a.ldy = _act(y, "y", shape, x)
        a.y = y.data_ptr()
        out["y"] = y
    if want_rstd:
        out["rstd"] = t.empty(rows, dtype=t.float32, device=x.device)
        a.rstd = out["rstd"].data_ptr()
    if quant != MOE_NORM_PLAIN:
        out["codes"] = t.empty((rows, H), dtype=t.uint8, device=x.device)
        if quant == MOE_NORM_FP8_BLOCK:
            out["scales"] = t.empty((rows, H // 128), dtype=t.float32, device=x.device)
        else:
            out["scales"] = t.empty((rows + 127) // 128 * (H // 128) * 512, dtype=t.uint8, device=x.device)
        a.codes = out["codes"].data_ptr()
        a.scales = out["scales"].data_ptr()
    _call("moe_add_rms_norm", x.get_device(), lib.moe_add_rms_norm, rows, H, _dtypes[x.dtype], quant, eps, ctypes.byref(a))
    return out


def add_rms_norm_backward(dy, h, rstd, weight, dh=None, *, dx=None, want_dweight: bool = True, ws=None):
    """Gradients of add_rms_norm (moe_add_rms_norm_backward): ``(dx, dweight)``
    from the gradient of y, the normalised sum ``h`` (x itself without a
    residual), the forward's ``rstd`` and the gradient ``dh`` that reaches h
    along the residual stream. dx is the gradient of x and of the residual.
    ``ws``: scratch of moe_norm_workspace_size bytes, else allocated here."""
    lib = _load()
    t = _torch
    lddy = _act(dy, "dy")
    shape = rows, H = dy.shape
    a = moe_norm_bwd_args_t(dy.data_ptr(), h.data_ptr(), _vec(rstd, "rstd", rows, t.float32, dy),
                            _vec(weight, "weight", H, t.float32, dy))
    a.lddy, a.ldh = lddy, _act(h, "h", shape, dy)
    if dh is not None:
        a.lddh = _act(dh, "dh", shape, dy)
        a.dh = dh.data_ptr()
    if dx is None:
        dx = _like(dy, lddy)
        a.lddx = H
    else:
        a.lddx = _act(dx, "dx", shape, dy)
    a.dx = dx.data_ptr()
    dweight = None
    if want_dweight:
        dweight = t.empty(H, dtype=t.float32, device=dy.device)
        a.dweight = dweight.data_ptr()
        if ws is None:
            ws = t.empty(moe_norm_workspace_size(rows, H), dtype=t.uint8, device=dy.device)
        elif ws.get_device() != dy.get_device() or not ws.is_contiguous():
            raise ValueError("ws: contiguous scratch on dy's device is needed")
    _call("moe_add_rms_norm_backward", dy.get_device(), lib.moe_add_rms_norm_backward, rows, H, _dtypes[dy.dtype],
          ctypes.byref(a), _p(ws), 0 if ws is None else ws.numel() * ws.element_size())
    return dx, dweight


def sort_index(topk, E: int, align: int = 1) -> Dict[str, object]:
    """Sort the slots of ``topk`` (T x k int32; values outside [0, E) drop a
    slot) by expert (moe_sort_index): a dict of int32 tensors ``counts`` (E),
    ``offsets`` (E + 1, multiples of ``align``), ``row_of`` (T x k) and
    ``slot_of`` (moe_sort_rows_cap rows)."""
    lib = _load()
    t = _torch
    if not topk.is_cuda or topk.dim() != 2 or topk.dtype != t.int32 or not topk.is_contiguous():
        raise ValueError("topk: a contiguous T x k int32 CUDA tensor is needed")
    T, k = topk.shape
    n = T * k
    if n == 0 or E < 1 or align < 1:
        rows = moe_sort_rows_cap(T, k, E, align)
    else:                                    # the same, without the call
        rows = -(-(n + min(E, n) * (align - 1)) // align) * align
    dev, i32 = topk.device, t.int32
    counts, offsets = t.empty(E, dtype=i32, device=dev), t.empty(E + 1, dtype=i32, device=dev)
    row_of, slot_of = t.empty_like(topk), t.empty(rows, dtype=i32, device=dev)
    _call("moe_sort_index", topk.get_device(), lib.moe_sort_index, T, k, E, align, topk.data_ptr(), counts.data_ptr(),
          offsets.data_ptr(), row_of.data_ptr(), slot_of.data_ptr(), rows)
    return {"counts": counts, "offsets": offsets, "row_of": row_of, "slot_of": slot_of}


def _sorted(index, H, dtype, like, rows, padding=True):
    row_of, slot_of = index.get("row_of"), index.get("slot_of")
    if row_of is None:
        raise ValueError("index: row_of is missing")
    t = _torch
    if row_of.dim() != 2 or row_of.dtype != t.int32 or row_of.device != like.device or not row_of.is_contiguous():
        raise ValueError("row_of: a contiguous T x k int32 tensor on the rows' device is needed")
    s = moe_sorted_t(row_of.shape[0], row_of.shape[1], H, _dtypes[dtype], rows, row_of.data_ptr())
    if padding and slot_of is not None:
        offsets, counts = index.get("offsets"), index.get("counts")
        dev = like.get_device()
        # the rows in use stand after the last expert's offset
        if offsets is None or offsets.numel() < 2 or (counts is not None and offsets.numel() != counts.numel() + 1):
            raise ValueError("offsets: one value for each expert and one more are needed")
        if (slot_of.numel() < rows or slot_of.dtype != t.int32 or offsets.dtype != t.int32 or slot_of.get_device() != dev or
                offsets.get_device() != dev or not slot_of.is_contiguous() or not offsets.is_contiguous()):
            raise ValueError(f"slot_of, offsets: contiguous int32 on the rows' device, for each of the {rows} rows")
        s.slot_of = slot_of.data_ptr()
        s.in_use = offsets.data_ptr() + 4 * (offsets.numel() - 1)
    return s


def sort_rows(x, index, out=None):
    """The tokens' rows in expert order (moe_sort_rows): a matrix of as many
    rows as ``slot_of`` (or ``out``), padding rows zero; rows from offsets[E]
    on are not written. With ``slot_of`` an index has ``offsets`` of exactly
    E + 1 values (checked against ``counts`` where it has those too). An index
    without ``slot_of`` (the ``row_of`` of a layer's routing) needs ``out``,
    and its padding rows are left alone; a layer with a ``capacity_factor``
    gives dropped slots rows there too (moe_sorted_t says which)."""
    lib = _load()
    ldx = _act(x, "x")
    T, H = x.shape
    if out is None:
        if index.get("slot_of") is None:
            raise ValueError("out: an index without slot_of does not say how many rows there are")
        out = _torch.empty((index["slot_of"].numel(), H), dtype=x.dtype, device=x.device)
    ldp = _act(out, "out", (out.shape[0], H), x)
    s = _sorted(index, H, x.dtype, x, out.shape[0])
    if s.T != T:
        raise ValueError(f"x: {T} rows, the index has {s.T} tokens")
    _call("moe_sort_rows", x.get_device(), lib.moe_sort_rows, ctypes.byref(s), x.data_ptr(), ldx, out.data_ptr(), ldp)
    return out


def unsort_rows(rows, index, gates=None, residual=None, out=None):
    """``y[t] = residual[t] + sum_j gates[t, j] rows[row_of[t, j]]``
    (moe_unsort_rows). Without ``gates`` (T x k fp32) the weights are 1: the
    gradient of sort_rows."""
    lib = _load()
    t = _torch
    ldp = _act(rows, "rows")
    R, H = rows.shape
    s = _sorted(index, H, rows.dtype, rows, R, padding=False)
    g = None if gates is None else _vec(gates, "gates", s.T * s.k, t.float32, rows)
    ldr = H if residual is None else _act(residual, "residual", (s.T, H), rows)
    if out is None:
        out = t.empty((s.T, H), dtype=rows.dtype, device=rows.device)
    ldy = _act(out, "out", (s.T, H), rows)
    _call("moe_unsort_rows", rows.get_device(), lib.moe_unsort_rows, ctypes.byref(s), rows.data_ptr(), ldp, g,
          _p(residual), ldr, out.data_ptr(), ldy)
    return out


def unsort_rows_backward(dY, rows, index, gates=None, out=None, want_dgates: bool = True):
    """Gradients of unsort_rows (moe_unsort_rows_backward): ``(drows, dgates)``;
    padding rows of drows are zero. ``out`` may be ``rows`` itself."""
    lib = _load()
    t = _torch
    lddy = _act(dY, "dY")
    T, H = dY.shape
    ldp = _act(rows, "rows", (rows.shape[0], H), dY)
    s = _sorted(index, H, dY.dtype, dY, rows.shape[0])
    if s.T != T:
        raise ValueError(f"dY: {T} rows, the index has {s.T} tokens")
    g = None if gates is None else _vec(gates, "gates", T * s.k, t.float32, dY)
    if out is None:
        out = t.empty((rows.shape[0], H), dtype=dY.dtype, device=dY.device)
    ldd = _act(out, "out", (rows.shape[0], H), dY)
    dg = t.empty((T, s.k), dtype=t.float32, device=dY.device) if want_dgates else None
    _call("moe_unsort_rows_backward", dY.get_device(), lib.moe_unsort_rows_backward, ctypes.byref(s), dY.data_ptr(), lddy,
          rows.data_ptr(), ldp, g, out.data_ptr(), ldd, _p(dg))
    return out, dg


def clip_grad_norm(grads: Sequence, max_norm: float, outs: Optional[Sequence] = None, *, clip: bool = True, ws=None):
    """The global norm of ``grads`` (contiguous fp32 or bf16 tensors on one
    device) as a 0-dim fp32 tensor; each gradient times min(1, max_norm / norm)
    goes to ``outs`` (default: in place). ``clip=False``: the norm alone."""
    lib = _load()
    t = _torch
    grads = list(grads)
    if not grads or (outs is not None and len(outs) != len(grads)):
        raise ValueError("grads: at least one tensor, and as many outs")
    tensor = t.Tensor
    dev = grads[0].get_device()
    ns = list(map(tensor.numel, grads))
    kinds = [_dtypes.get(g.dtype, -1) for g in grads]
    if dev < 0 or -1 in kinds or any(d != dev for d in map(tensor.get_device, grads)) or not all(map(tensor.is_contiguous, grads)):
        raise ValueError("grads: contiguous fp32 or bf16 CUDA tensors on one device are needed")
    ptrs = list(map(tensor.data_ptr, grads))
    to = ptrs
    if not clip:
        to = [0] * len(grads)
    elif outs is not None:
        if (list(map(tensor.numel, outs)) != ns or [_dtypes.get(o.dtype, -1) for o in outs] != kinds or
                any(d != dev for d in map(tensor.get_device, outs)) or not all(map(tensor.is_contiguous, outs))):
            raise ValueError("outs: types, sizes and device of the gradients, contiguous")
        to = list(map(tensor.data_ptr, outs))
    table = array.array("q", [v for entry in zip(ptrs, to, ns, kinds) for v in entry])
    if ws is None:
        ws = t.empty(moe_clip_workspace_size(len(grads)), dtype=t.uint8, device=grads[0].device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws: contiguous scratch on the gradients' device is needed")
    norm = t.empty((), dtype=t.float32, device=grads[0].device)
    _call("moe_clip_grad_norm", dev, lib.moe_clip_grad_norm, len(grads), table.buffer_info()[0], max_norm,
          norm.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size())
    return norm
