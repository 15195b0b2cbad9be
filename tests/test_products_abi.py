"""Refusals of the products over sorted rows (CPU): every bad argument is turned
into a status or a ValueError before any launch; no pointer here is ever read."""
import ctypes

import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from mixture_experts_layer_sigmoid_gb300 import _build, operators

P = 4096          # aligned addresses that nothing dereferences
Q, R = 8192, 12288
ARG, ALIGN = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_MISALIGNED
BIG = (1 << 20) + 1


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load_library()


def groups(**kw):
    return moe.moe_groups_t(**{**dict(E=4, dtype=1, rows=10, offsets=P, counts=P), **kw})


BAD_GROUPS = [(dict(E=0), ARG), (dict(E=1025), ARG), (dict(dtype=2), ARG), (dict(dtype=-1), ARG), (dict(rows=-1), ARG),
              (dict(rows=2 ** 31 - 1), ARG), (dict(offsets=None), ARG), (dict(offsets=None, E=1), ARG), (dict(offsets=P + 2), ALIGN),
              (dict(counts=P + 1), ALIGN)]


def rows_call(lib, g=None, **kw):
    c = dict(K=64, N=32, X=P, ldx=64, W=Q, ldw=32, sw=64 * 32, w_nk=0, Y=R, ldy=32)
    c.update(kw)
    return lib.moe_grouped_matmul(ctypes.byref(g or groups()), *c.values(), None)


def wgrad_call(lib, g=None, **kw):
    c = dict(M=64, N=32, A=P, lda=64, B=Q, ldb=32, D=R, ldd=32, sd=64 * 32)
    c.update(kw)
    return lib.moe_grouped_wgrad(ctypes.byref(g or groups()), *c.values(), None)


def fp8_call(lib, g=None, K=256, N=64, **kw):
    a = moe.moe_fp8_matmul_args_t(**{**dict(A=P, lda=256, SA=Q, ldsa=2, B=P, ldb=64, sb=256 * 64, SB=Q, ldsb=1, ssb=2, b_nk=0, Y=R,
                                            ldy=64), **kw})
    return lib.moe_fp8_matmul(ctypes.byref(g or groups()), K, N, ctypes.byref(a), None)


@pytest.mark.parametrize("change,want", BAD_GROUPS)
def test_bad_groups(lib, change, want):
    for call in (rows_call, wgrad_call, fp8_call):
        assert call(lib, groups(**change)) == want


def test_null_arguments(lib):
    assert lib.moe_grouped_matmul(None, 64, 32, P, 64, P, 32, 2048, 0, P, 32, None) == ARG
    assert lib.moe_grouped_wgrad(None, 64, 32, P, 64, P, 32, P, 32, 2048, None) == ARG
    assert lib.moe_fp8_matmul(None, 256, 64, None, None) == ARG
    assert lib.moe_fp8_matmul(ctypes.byref(groups()), 256, 64, None, None) == ARG


@pytest.mark.parametrize("change,want", [
    (dict(K=0), ARG), (dict(N=0), ARG), (dict(K=BIG, ldx=BIG), ARG), (dict(N=BIG, ldw=BIG, ldy=BIG), ARG), (dict(X=None), ARG),
    (dict(W=None), ARG), (dict(Y=None), ARG), (dict(ldx=63), ARG), (dict(ldy=31), ARG), (dict(ldw=31), ARG), (dict(ldx=-64), ARG),
    (dict(w_nk=1), ARG), (dict(w_nk=2), ARG), (dict(w_nk=-1), ARG), (dict(sw=64 * 32 - 1), ARG), (dict(sw=0), ARG),
    (dict(ldx=1 << 50), ARG), (dict(sw=1 << 50), ARG), (dict(X=P + 2), ALIGN), (dict(W=P + 8), ALIGN), (dict(Y=P + 4), ALIGN), (dict(Y=P), ARG),
    (dict(Y=Q), ARG)])
def test_grouped_matmul_refuses(lib, change, want):
    assert rows_call(lib, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(M=0), ARG), (dict(N=-1), ARG), (dict(M=BIG, lda=BIG), ARG), (dict(A=None), ARG), (dict(B=None), ARG), (dict(D=None), ARG),
    (dict(lda=63), ARG), (dict(ldb=31), ARG), (dict(ldd=31), ARG), (dict(sd=64 * 32 - 1), ARG), (dict(A=P + 2), ALIGN),
    (dict(B=P + 2), ALIGN), (dict(D=P + 2), ALIGN), (dict(D=P), ARG), (dict(D=Q), ARG)])
def test_grouped_wgrad_refuses(lib, change, want):
    assert wgrad_call(lib, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(K=192), ARG), (dict(K=0), ARG), (dict(N=0), ARG), (dict(A=None), ARG), (dict(SA=None), ARG), (dict(B=None), ARG),
    (dict(SB=None), ARG), (dict(Y=None), ARG), (dict(lda=240), ARG), (dict(ldsa=1), ARG), (dict(ldb=48), ARG), (dict(ldsb=0), ARG),
    (dict(ldy=63), ARG), (dict(sb=16), ARG), (dict(ssb=1), ARG), (dict(b_nk=1), ARG), (dict(b_nk=3), ARG), (dict(A=P + 8), ALIGN),
    (dict(SA=P + 4), ALIGN), (dict(B=P + 1), ALIGN), (dict(SB=P + 4), ALIGN), (dict(Y=P + 2), ALIGN), (dict(lda=257), ALIGN),
    (dict(ldb=72, sb=256 * 72), ALIGN), (dict(sb=256 * 64 + 8), ALIGN), (dict(Y=P), ARG), (dict(Y=Q), ARG)])
def test_fp8_matmul_refuses(lib, change, want):
    assert fp8_call(lib, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), ARG), (dict(rows=2 ** 31 - 1), ARG), (dict(K=0), ARG), (dict(K=100), ARG), (dict(dtype=2), ARG), (dict(x=None), ARG),
    (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(ldx=255), ARG), (dict(ldc=128), ARG), (dict(lds=1), ARG),
    (dict(x=P + 2), ALIGN), (dict(codes=P + 8), ALIGN), (dict(scales=P + 4), ALIGN), (dict(ldx=257), ALIGN), (dict(ldc=264), ALIGN),
    (dict(in_use=P + 2), ALIGN), (dict(codes=P), ARG), (dict(scales=P), ARG), (dict(scales=Q), ARG)])
def test_quantize_rows_refuses(lib, change, want):
    c = dict(rows=4, K=256, dtype=1, x=P, ldx=256, codes=Q, ldc=256, scales=R, lds=2, in_use=None)
    c.update(change)
    assert lib.moe_quantize_rows(*c.values(), None) == want


def test_no_rows_need_no_device(lib):
    g = groups(rows=0)
    assert rows_call(lib, g, X=None, W=None, Y=None) == moe.MOE_OK
    assert fp8_call(lib, g, A=None, SA=None, B=None, SB=None, Y=None) == moe.MOE_OK
    assert lib.moe_quantize_rows(0, 256, 1, None, 256, None, 256, None, 2, None, None) == moe.MOE_OK


def test_python_checks_need_no_gpu():
    x, w = torch.zeros((4, 128)), torch.zeros((2, 128, 64))
    c, s = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 1))
    for call in (lambda: moe.grouped_matmul(x, w, {}), lambda: moe.grouped_matmul_backward(x, x, w, {}),
                 lambda: moe.fp8_matmul(c, s, c, s), lambda: moe.quantize_rows(x), lambda: moe.quantize_tiles(w)):
        with pytest.raises(ValueError):
            call()


def test_layouts_of_weights():
    """Row stride, expert stride and orientation, on host tensors of the check's device number."""
    _build.build()
    operators._load()
    f = torch.zeros
    check = lambda w: operators._experts(w, "w", torch.float32, -1)  # noqa: E731
    with pytest.raises(ValueError):
        check(f((2, 3, 4)))
    one = lambda w: operators._experts(Fake(w), "w", torch.float32, 0)  # noqa: E731
    assert one(f((2, 3, 4))) == (4, 12, 0)
    assert one(f((2, 4, 3)).transpose(1, 2)) == (3, 12, 1)
    assert one(f((2, 3, 8))[:, :, :4]) == (8, 24, 0)
    assert one(f((1, 3, 4)))[1] >= 12
    assert one(f((2, 1, 4)))[0] >= 4 and one(f((2, 4, 1))) == (4, 4, 1) and one(f((2, 4, 8))[:, :, :1]) == (8, 32, 0)
    for bad in (f((3, 4)), f((2, 3, 8))[:, :, ::2], f((2, 3, 4), dtype=torch.float64)):
        with pytest.raises(ValueError):
            one(bad)


class Fake:
    """A host tensor that says it stands on device 0."""

    def __init__(self, t):
        self.t = t
        self.shape, self.dtype, self.device = t.shape, t.dtype, "cuda:0"

    def get_device(self):
        return 0

    def stride(self):
        return self.t.stride()


@pytest.mark.parametrize("bad", [dict(offsets=5), dict(offsets=7), dict(counts=4), dict(counts=6), dict(none=True)])
def test_an_index_of_another_length_is_refused(bad):
    _build.build()
    operators._load()
    i32 = dict(dtype=torch.int32)
    ix = dict(offsets=torch.zeros(bad.get("offsets", 6), **i32), counts=torch.zeros(bad.get("counts", 5), **i32))
    if bad.get("none"):
        del ix["offsets"]
    with pytest.raises(ValueError):
        operators._groups(ix, 10, 5, torch.float32, -1)


def test_without_an_index_there_is_one_expert():
    _build.build()
    operators._load()
    with pytest.raises(ValueError):
        operators._groups(None, 10, 2, torch.float32, 0)
    assert operators._groups(None, 10, 1, torch.float32, 0).E == 1
