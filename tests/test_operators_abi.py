"""Refusals of the operators around the layer (CPU): every bad argument is
turned into a status before any launch; no pointer here is ever read."""
import ctypes

import pytest

import mixture_experts_layer_sigmoid_gb300 as moe
from mixture_experts_layer_sigmoid_gb300 import _build

P = 4096          # an aligned address that nothing dereferences
ARG, ALIGN, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_MISALIGNED, moe.MOE_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load_library()


def norm_args(**kw):
    base = dict(x=P, weight=P, y=P, ldx=256, ldr=256, ldh=256, ldy=256)
    base.update(kw)
    return moe.moe_norm_fwd_args_t(**base)


@pytest.mark.parametrize("change,call,want", [
    (dict(x=None), {}, ARG), (dict(weight=None), {}, ARG), (dict(y=None), {}, ARG), (dict(codes=P), {}, ARG),
    (dict(scales=P), {}, ARG), (dict(h=P), {}, ARG), (dict(ldx=255), {}, ARG), (dict(ldy=0), {}, ARG),
    (dict(residual=P, ldr=100), {}, ARG), (dict(residual=P, h=P, ldh=-256), {}, ARG),
    ({}, dict(rows=-1), ARG), ({}, dict(rows=2 ** 31 - 1), ARG), ({}, dict(H=0), ARG), ({}, dict(H=(1 << 20) + 1), ARG), ({}, dict(dtype=2), ARG),
    ({}, dict(dtype=-1), ARG), ({}, dict(quant=3), ARG), ({}, dict(quant=-1), ARG), ({}, dict(eps=-1e-6), ARG),
    ({}, dict(eps=float("nan")), ARG), ({}, dict(eps=float("inf")), ARG), ({}, dict(quant=1), ARG),
    (dict(codes=P), dict(quant=1), ARG), (dict(scales=P), dict(quant=2), ARG),
    (dict(codes=P, scales=P), dict(quant=1, H=192), ARG), (dict(codes=P, scales=P, ldx=257), dict(quant=2), ALIGN),
    (dict(x=P + 2), {}, ALIGN), (dict(weight=P + 4), {}, ALIGN), (dict(rstd=P + 8), {}, ALIGN),
    (dict(codes=P + 1, scales=P), dict(quant=1), ALIGN),
])
def test_norm_forward_refuses(lib, change, call, want):
    c = dict(rows=4, H=256, dtype=1, quant=0, eps=1e-6)
    c.update(call)
    a = norm_args(**change)
    assert lib.moe_add_rms_norm(c["rows"], c["H"], c["dtype"], c["quant"], c["eps"], ctypes.byref(a), None) == want


def test_norm_null_args_and_empty(lib):
    assert lib.moe_add_rms_norm(4, 256, 1, 0, 1e-6, None, None) == ARG
    a = moe.moe_norm_fwd_args_t(weight=P, ldx=256, ldy=256)
    assert lib.moe_add_rms_norm(0, 256, 1, 0, 1e-6, ctypes.byref(a), None) == moe.MOE_OK


@pytest.mark.parametrize("change,call,want", [
    (dict(dy=None), {}, ARG), (dict(h=None), {}, ARG), (dict(rstd=None), {}, ARG), (dict(weight=None), {}, ARG),
    (dict(dx=None), {}, ARG), (dict(lddx=1), {}, ARG), (dict(dh=P, lddh=8), {}, ARG), ({}, dict(rows=-5), ARG),
    ({}, dict(H=0), ARG), ({}, dict(dtype=4), ARG), (dict(dy=P + 2), {}, ALIGN), (dict(dweight=P + 4), {}, ALIGN),
    (dict(dweight=P), dict(ws=None), ARG), (dict(dweight=P), dict(bytes=4 * 256 * 4 - 1), WS),
    ({}, dict(ws=P + 8), ALIGN),
])
def test_norm_backward_refuses(lib, change, call, want):
    c = dict(rows=4, H=256, dtype=0, ws=P, bytes=1 << 20)
    c.update(call)
    base = dict(dy=P, h=P, rstd=P, weight=P, dx=P, lddy=256, ldh=256, lddh=256, lddx=256)
    base.update(change)
    a = moe.moe_norm_bwd_args_t(**base)
    assert lib.moe_add_rms_norm_backward(c["rows"], c["H"], c["dtype"], ctypes.byref(a), c["ws"], c["bytes"], None) == want


def test_workspace_sizes(lib):
    assert moe.moe_norm_workspace_size(0, 64) == 0
    assert moe.moe_norm_workspace_size(4, 256) >= 4 * 256 * 4
    with pytest.raises(moe.MoEError):
        moe.moe_norm_workspace_size(-1, 64)
    assert moe.moe_clip_workspace_size(0) > 0
    assert moe.moe_clip_workspace_size(100000) > moe.moe_clip_workspace_size(10)
    with pytest.raises(moe.MoEError):
        moe.moe_clip_workspace_size(-1)
    assert lib.moe_clip_workspace_size(3, None) == ARG and lib.moe_norm_workspace_size(3, 3, None) == ARG


@pytest.mark.parametrize("T,k,E,align,rows", [(0, 1, 1, 1, 0), (1, 1, 1, 1, 1), (1, 1, 1, 128, 128), (10, 2, 4, 16, 80),
                                              (2, 2, 256, 128, 512), (5, 1, 3, 4, 16)])
def test_sort_rows_cap(lib, T, k, E, align, rows):
    n = T * k
    assert moe.moe_sort_rows_cap(T, k, E, align) == rows == -(-(n + min(E, n) * (align - 1)) // align) * align


@pytest.mark.parametrize("bad", [(-1, 1, 1, 1), (1, 0, 1, 1), (1, 33, 64, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                                 (1, 1, 1, 4097), (1 << 30, 2, 8, 1), (1 << 30, 1, 1024, 4096 * 0 + 4096)])
def test_sort_limits(lib, bad):
    n = ctypes.c_longlong()
    if bad == (1 << 30, 1, 1024, 4096):       # fits: 2^30 + 1024 * 4095 rows
        assert lib.moe_sort_rows_cap(*bad, ctypes.byref(n)) == moe.MOE_OK
        return
    assert lib.moe_sort_rows_cap(*bad, ctypes.byref(n)) == ARG
    assert lib.moe_sort_index(*bad, P, P, P, P, P, 1 << 30, None) == ARG


def test_sort_index_refuses(lib):
    ok = dict(T=4, k=2, E=8, align=1, topk=P, counts=P, offsets=P, row_of=P, slot_of=P, rows=8)
    f = lambda **kw: lib.moe_sort_index(*{**ok, **kw}.values(), None)  # noqa: E731
    for n in ("topk", "counts", "offsets", "row_of", "slot_of"):
        assert f(**{n: None}) == ARG
        assert f(**{n: P + 4}) == ALIGN
    assert f(rows=7) == ARG and f(rows=1 << 31) == ARG


def sorted_args(**kw):
    base = dict(T=4, k=2, H=64, dtype=1, rows=8, row_of=P, slot_of=P, in_use=P)
    base.update(kw)
    return moe.moe_sorted_t(**base)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), ARG), (dict(k=0), ARG), (dict(k=33), ARG), (dict(H=0), ARG), (dict(H=(1 << 20) + 1), ARG), (dict(dtype=2), ARG), (dict(rows=-1), ARG),
    (dict(rows=1 << 31), ARG), (dict(row_of=None), ARG), (dict(row_of=P + 4), ALIGN),
    (dict(T=1 << 30, k=2), ARG)])
def test_movers_refuse_a_bad_index(lib, change, want):
    s = ctypes.byref(sorted_args(**change))
    assert lib.moe_sort_rows(s, P, 64, P, 64, None) == want
    assert lib.moe_unsort_rows(s, P, 64, None, None, 0, P, 64, None) == want
    assert lib.moe_unsort_rows_backward(s, P, 64, P, 64, None, P, 64, None, None) == want


def test_movers_refuse(lib):
    s = ctypes.byref(sorted_args())
    for bad in (sorted_args(in_use=None), sorted_args(slot_of=P + 8), sorted_args(in_use=P + 2)):
        want = ARG if bad.in_use is None else ALIGN
        assert lib.moe_sort_rows(ctypes.byref(bad), P, 64, P, 64, None) == want
        assert lib.moe_unsort_rows_backward(ctypes.byref(bad), P, 64, P, 64, None, P, 64, None, None) == want
    assert lib.moe_sort_rows(None, P, 64, P, 64, None) == ARG
    for a, want in (((None, 64, P, 64), ARG), ((P, 63, P, 64), ARG), ((P, 64, None, 64), ARG), ((P, 64, P, 0), ARG),
                    ((P + 2, 64, P, 64), ALIGN), ((P, 64, P + 2, 64), ALIGN)):
        assert lib.moe_sort_rows(s, *a, None) == want
    for a, want in (((None, 64, P, P, 64, P, 64), ARG), ((P, 60, P, P, 64, P, 64), ARG), ((P, 64, P, P, 60, P, 64), ARG),
                    ((P, 64, P, P, 64, None, 64), ARG), ((P, 64, P, P, 64, P, 63), ARG), ((P, 64, P + 4, P, 64, P, 64), ALIGN),
                    ((P, 64, P, P + 2, 64, P, 64), ALIGN)):
        assert lib.moe_unsort_rows(s, *a, None) == want
    for a, want in (((None, 64, P, 64, P, P, 64, P), ARG), ((P, 6, P, 64, P, P, 64, P), ARG), ((P, 64, None, 64, P, P, 64, P), ARG),
                    ((P, 64, P, 6, P, P, 64, P), ARG), ((P, 64, P, 64, P, None, 64, P), ARG), ((P, 64, P, 64, P, P, 6, P), ARG),
                    ((P, 64, P, 64, P + 4, P, 64, P), ALIGN), ((P, 64, P, 64, P, P, 64, P + 4), ALIGN)):
        assert lib.moe_unsort_rows_backward(s, *a, None) == want


def test_clip_refuses(lib):
    def f(entries, max_norm=1.0, norm=P, ws=P, nbytes=1 << 20, count=None):
        t = (moe.moe_grad_t * max(1, len(entries)))(*[moe.moe_grad_t(*e) for e in entries])
        return lib.moe_clip_grad_norm(len(entries) if count is None else count, ctypes.addressof(t), max_norm, norm, ws,
                                      nbytes, None)

    good = (P, P, 10, 0, 0)
    for m in (0.0, -1.0, float("nan")):
        assert f([good], m) == ARG
    assert f([good], norm=None) == ARG and f([good], ws=None) == ARG and f([good], count=-1) == ARG
    assert lib.moe_clip_grad_norm(1, None, 1.0, P, P, 1 << 20, None) == ARG
    for e in ((None, P, 10, 0, 0), (P, P, -1, 0, 0), (P, P, 10, 2, 0), (P, P, 10, 0, 1), (P, P, 1 << 62, 0, 0),
              (P, P, 1 << 45, 0, 0)):
        assert f([good, e]) == ARG
    for e in ((P + 2, P, 10, 0, 0), (P, P + 2, 10, 0, 0), (P + 1, P, 10, 1, 0), (P, P + 1, 10, 1, 0)):
        assert f([good, e]) == ALIGN
    assert f([good], norm=P + 2) == ALIGN and f([good], ws=P + 8) == ALIGN
    assert f([good], nbytes=moe.moe_clip_workspace_size(1) - 1) == WS


def test_python_checks_need_no_gpu():
    import torch
    x = torch.zeros((4, 64))
    for call in (lambda: moe.add_rms_norm(x, torch.ones(64)), lambda: moe.sort_rows(x, {}),
                 lambda: moe.add_rms_norm_backward(x, x, torch.ones(4), torch.ones(64)),
                 lambda: moe.sort_index(torch.zeros((4, 2), dtype=torch.int32), 8), lambda: moe.unsort_rows(x, {}),
                 lambda: moe.unsort_rows_backward(x, x, {}), lambda: moe.clip_grad_norm([x], 1.0),
                 lambda: moe.clip_grad_norm([], 1.0)):
        with pytest.raises(ValueError):
            call()
