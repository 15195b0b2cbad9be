"""The operators around the expert layer, on torch tensors.

Torch allocates outputs and scratch and supplies the current stream of the
tensors' device; every value is computed by the kernels behind include/moe.h
(``moe_add_rms_norm``, ``moe_sort_*``, ``moe_unsort_*``, ``moe_clip_grad_norm``,
``moe_grouped_*``, ``moe_fp8_matmul``, ``moe_quantize_rows``), whose entries
describe the mathematics, the limits and the errors. Activations are fp32 or bf16
matrices whose last dimension is contiguous (any row stride).
Wrong devices, types and shapes raise ValueError here; what the library
refuses raises MoEError.
"""
from __future__ import annotations

import array
import ctypes
from typing import Dict, Optional, Sequence

from . import (MOE_BF16, MOE_FP32, MOE_OK, MOE_Q_TILES, MoEError, load_library, moe_clip_workspace_size,
               moe_fp8_matmul_args_t, moe_groups_t, moe_norm_bwd_args_t, moe_norm_fwd_args_t,
               moe_norm_workspace_size, moe_sort_rows_cap, moe_sorted_t)

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


def _groups(index, rows, E, dtype, dev):
    """The segments of an index (or, None, of one expert that has all rows)."""
    if index is None:
        if E != 1:
            raise ValueError("index: without one there is one expert")
        return moe_groups_t(1, _dtypes[dtype], rows, None, None)
    offsets, counts = index.get("offsets"), index.get("counts")
    i32 = _torch.int32
    if (offsets is None or offsets.dtype != i32 or offsets.get_device() != dev or not offsets.is_contiguous() or
            offsets.numel() != E + 1):
        raise ValueError(f"offsets: {E + 1} contiguous int32 values on the rows' device are needed")
    if counts is None:
        return moe_groups_t(E, _dtypes[dtype], rows, offsets.data_ptr(), None)
    if counts.dtype != i32 or counts.get_device() != dev or not counts.is_contiguous() or counts.numel() != E:
        raise ValueError(f"counts: {E} contiguous int32 values on the rows' device are needed")
    return moe_groups_t(E, _dtypes[dtype], rows, offsets.data_ptr(), counts.data_ptr())


def _experts(w, name, dtype, dev, shape=None):
    """Checks E x K x N weights; returns (row stride, stride of an expert, whether
    they are stored N x K). Either of the last two dimensions is contiguous."""
    if w.get_device() != dev or dev < 0 or w.dtype != dtype or len(w.shape) != 3 or (shape is not None and w.shape != shape):
        raise ValueError(f"{name}: an {'E x K x N' if shape is None else tuple(shape)} {dtype} tensor on the rows' device is "
                         f"needed, got {tuple(w.shape)} {w.dtype} on {w.device}")
    E, K, N = w.shape
    se, sk, sn = w.stride()
    if N == 1 and sk == 1:
        ld, nk, least = K, 1, K
    elif sn == 1 or N == 1:
        ld, nk, least = (sk if K > 1 else N), 0, (K - 1) * sk + N
    elif sk == 1 or K == 1:
        ld, nk, least = sn, 1, (N - 1) * sn + K
    else:
        raise ValueError(f"{name}: one of the last two dimensions has to be contiguous")
    return ld, se if E > 1 else least, nk


def _rows_out(out, name, rows, H, like, dtype):
    """The output rows (new ones if None) and their stride."""
    if out is None:
        return _torch.empty((rows, H), dtype=dtype, device=like.device), H
    if out.shape != (rows, H) or out.get_device() != like.get_device() or out.dtype != dtype:
        raise ValueError(f"{name}: {tuple(out.shape)} {out.dtype} on {out.device}, expected ({rows}, {H}) {dtype} on {like.device}")
    ld, one = out.stride()
    if one != 1 and H > 1:
        raise ValueError(f"{name}: the last dimension has to be contiguous")
    return out, ld if rows > 1 else H


def grouped_matmul(rows, w, index, out=None):
    """``out[r] = rows[r] @ w[e]`` for the rows of each expert's segment
    (moe_grouped_matmul): ``rows`` (R x K) as sort_rows gives them, ``w`` (E x K
    x N) contiguous in either of its last two dimensions (weights stored out x
    in are passed as their transposed view), ``index`` the sort's or a layer's
    ``offsets`` and, where there is padding, ``counts``. Padding rows come out as
    zeros; rows behind the last segment are neither read nor written. Each tensor
    starts on a 16-byte boundary (a slice that does not is refused); its strides
    are free."""
    lib = _load()
    ldx = _act(rows, "rows")
    R, K = rows.shape
    dev = rows.get_device()
    ldw, sw, nk = _experts(w, "w", rows.dtype, dev)
    E, Kw, N = w.shape
    if Kw != K:
        raise ValueError(f"w: {Kw} x {N} for rows of {K}")
    g = _groups(index, R, E, rows.dtype, dev)
    out, ldy = _rows_out(out, "out", R, N, rows, rows.dtype)
    _call("moe_grouped_matmul", dev, lib.moe_grouped_matmul, ctypes.byref(g), K, N, rows.data_ptr(), ldx, w.data_ptr(), ldw,
          sw, nk, out.data_ptr(), ldy)
    return out


def grouped_matmul_backward(dY, rows, w, index, *, want_drows: bool = True, want_dw: bool = True, drows=None, dw=None):
    """Gradients of grouped_matmul (moe_grouped_matmul, moe_grouped_wgrad):
    ``(drows, dw)``, ``drows[r] = dY[r] @ w[e].T`` with rows outside the segments
    as there, and ``dw[e]`` the sum of its rows' ``rows[r].T @ dY[r]``, zeros for
    an expert without rows, laid out as ``w``. ``drows`` and ``dw`` may be given
    (apart from each other and from what the call reads).
    ``rows`` is only read for dw, ``w`` only for drows (then its shape and strides
    still say dw's)."""
    lib = _load()
    t = _torch
    lddy = _act(dY, "dY")
    R, N = dY.shape
    dev = dY.get_device()
    ldw, sw, nk = _experts(w, "w", dY.dtype, dev)
    E, K, Nw = w.shape
    if Nw != N:
        raise ValueError(f"w: {K} x {Nw} for gradients of {N}")
    ldx = _act(rows, "rows", (R, K), dY)
    g = _groups(index, R, E, dY.dtype, dev)
    if want_drows and want_dw:           # drows is written first; the library sees one product at a time
        for out, name, others in ((drows, "drows", (rows, dw)), (dw, "dw", (w, drows))):
            if out is not None and R > 0 and any(o is not None and o.data_ptr() == out.data_ptr() for o in others):
                raise ValueError(f"{name}: at the address of another tensor of the call")
    if want_drows:
        drows, ldd = _rows_out(drows, "drows", R, K, dY, dY.dtype)
        _call("moe_grouped_matmul", dev, lib.moe_grouped_matmul, ctypes.byref(g), N, K, dY.data_ptr(), lddy, w.data_ptr(),
              ldw, sw, 1 - nk, drows.data_ptr(), ldd)
    if want_dw:
        if dw is None:
            dw = t.empty((E, N, K), dtype=w.dtype, device=w.device).transpose(1, 2) if nk else t.empty(
                (E, K, N), dtype=w.dtype, device=w.device)
        ldg, sg, gnk = _experts(dw, "dw", dY.dtype, dev, w.shape)
        if gnk:
            _call("moe_grouped_wgrad", dev, lib.moe_grouped_wgrad, ctypes.byref(g), N, K, dY.data_ptr(), lddy,
                  rows.data_ptr(), ldx, dw.data_ptr(), ldg, sg)
        else:
            _call("moe_grouped_wgrad", dev, lib.moe_grouped_wgrad, ctypes.byref(g), K, N, rows.data_ptr(), ldx,
                  dY.data_ptr(), lddy, dw.data_ptr(), ldg, sg)
    return (drows if want_drows else None), (dw if want_dw else None)


def _bytes(t, name, dtype, dev, shape):
    if t.dtype != dtype or t.get_device() != dev or dev < 0 or t.shape != shape:
        raise ValueError(f"{name}: {tuple(shape)} {dtype} on the codes' device is needed, got {tuple(t.shape)} {t.dtype} on {t.device}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the last dimension has to be contiguous")
    return ld if shape[0] > 1 else shape[1]


def fp8_matmul(codes, scales, w_codes, w_scales, index=None, *, dtype=None, out=None):
    """The product on E4M3 codes with a scale for each block of 128
    (moe_fp8_matmul): ``codes`` (R x K uint8) with ``scales`` (R x K/128 fp32), as
    add_rms_norm and quantize_rows give them, times ``w_codes`` (E x K x N uint8,
    or K x N without an index) with ``w_scales`` (E x K/128 x ceil(N/128)), as
    quantize_tiles gives them. Either of the weights' last two dimensions may be
    the contiguous one, the same in both tensors: the transposed views of codes
    and scales give the product with the transposed weights. ``dtype`` (default
    bf16) or ``out`` says fp32 or bf16; padding rows and rows behind the last
    segment as in grouped_matmul. Each tensor starts on a 16-byte boundary, and so
    does every row of codes (in either tensor)."""
    lib = _load()
    t = _torch
    if codes.dim() != 2 or codes.dtype != t.uint8 or not codes.is_cuda:
        raise ValueError("codes: a 2-D uint8 CUDA tensor is needed")
    dev = codes.get_device()
    R, K = codes.shape
    if w_codes.dim() == 2:
        if index is not None:
            raise ValueError("w_codes: E x K x N codes are needed with an index")
        w_codes, w_scales = w_codes[None], w_scales[None]
    if K % 128:
        raise ValueError(f"codes: {K} columns are not a multiple of 128")
    ldb, sb, nk = _experts(w_codes, "w_codes", t.uint8, dev)
    E, Kw, N = w_codes.shape
    if Kw != K:
        raise ValueError(f"w_codes: {Kw} x {N} for codes of {K}")
    nb = -(-N // 128)
    _experts(w_scales, "w_scales", t.float32, dev, (E, K // 128, nb))
    se, sk, sn = w_scales.stride()
    if nk:                               # the scales' rows run along n
        if sk != 1 and K > 128:
            raise ValueError("w_scales: contiguous in the dimension in which w_codes is")
        ldsb = sn if nb > 1 else K // 128
    else:
        if sn != 1 and nb > 1:
            raise ValueError("w_scales: contiguous in the dimension in which w_codes is")
        ldsb = sk if K > 128 else nb
    if out is not None:
        dtype = out.dtype if dtype is None else dtype
    elif dtype is None:
        dtype = t.bfloat16
    if dtype not in _dtypes:
        raise ValueError(f"dtype: fp32 or bf16, got {dtype}")
    a = moe_fp8_matmul_args_t(codes.data_ptr(), _bytes(codes, "codes", t.uint8, dev, codes.shape))
    a.ldsa = _bytes(scales, "scales", t.float32, dev, (R, K // 128))
    a.SA, a.B, a.ldb, a.sb, a.b_nk = scales.data_ptr(), w_codes.data_ptr(), ldb, sb, nk
    a.SB, a.ldsb, a.ssb = w_scales.data_ptr(), ldsb, se if E > 1 else nb * (K // 128)
    g = _groups(index, R, E, dtype, dev)
    out, a.ldy = _rows_out(out, "out", R, N, codes, dtype)
    a.Y = out.data_ptr()
    _call("moe_fp8_matmul", dev, lib.moe_fp8_matmul, ctypes.byref(g), K, N, ctypes.byref(a))
    return out


def quantize_rows(x, index=None, *, codes=None, scales=None):
    """E4M3 codes (uint8) and fp32 scales of 1x128 blocks of activation rows
    (moe_quantize_rows), any number of rows, columns a multiple of 128. With an
    ``index`` only the rows in use are read and written."""
    lib = _load()
    t = _torch
    ldx = _act(x, "x")
    R, K = x.shape
    dev = x.get_device()
    if K % 128:
        raise ValueError(f"x: {K} columns are not a multiple of 128")
    if codes is None:
        codes = t.empty((R, K), dtype=t.uint8, device=x.device)
    if scales is None:
        scales = t.empty((R, K // 128), dtype=t.float32, device=x.device)
    ldc, lds = _bytes(codes, "codes", t.uint8, dev, (R, K)), _bytes(scales, "scales", t.float32, dev, (R, K // 128))
    in_use = None
    if index is not None:
        offsets = index.get("offsets")
        if (offsets is None or offsets.dtype != t.int32 or offsets.get_device() != dev or not offsets.is_contiguous() or
                offsets.numel() < 2):
            raise ValueError("offsets: contiguous int32, one value for each expert and one more, on the rows' device")
        in_use = offsets.data_ptr() + 4 * (offsets.numel() - 1)
    _call("moe_quantize_rows", dev, lib.moe_quantize_rows, R, K, _dtypes[x.dtype], x.data_ptr(), ldx, codes.data_ptr(), ldc,
          scales.data_ptr(), lds, in_use)
    return codes, scales


def quantize_tiles(w):
    """E4M3 codes and fp32 scales of 128x128 tiles of bf16 weights (moe_fp8_quantize
    with MOE_Q_TILES): E x K x N or K x N, contiguous, K and N multiples of 128.
    Their transposed views are the codes and scales of the transposed weights."""
    lib = _load()
    t = _torch
    if not w.is_cuda or w.dtype != t.bfloat16 or w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("w: a contiguous 2-D or 3-D bf16 CUDA tensor is needed")
    K, N = w.shape[-2:]
    if K % 128 or N % 128 or w.numel() == 0 or w.numel() // N >= 2 ** 31:
        raise ValueError(f"w: {K} x {N} is not a multiple of 128 x 128, or there are too many rows")
    codes = t.empty(w.shape, dtype=t.uint8, device=w.device)
    scales = t.empty((*w.shape[:-2], K // 128, N // 128), dtype=t.float32, device=w.device)
    _call("moe_fp8_quantize", w.get_device(), lib.moe_fp8_quantize, w.numel() // N, N, MOE_Q_TILES, w.data_ptr(),
          codes.data_ptr(), scales.data_ptr(), None, None)
    return codes, scales


def products_status(device: Optional[int] = None) -> int:
    """Waits for the current stream of a device (default: the current one) and
    returns moe_products_status: MOE_OK, or MOE_ERR_DEVICE_TIMEOUT if a product's
    device-side wait ran out there since the last call."""
    lib = _load()
    cuda = _torch.cuda
    dev = cuda.current_device() if device is None else device
    with cuda.device(dev):
        return lib.moe_products_status(_stream(dev))
