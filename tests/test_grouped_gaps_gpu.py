"""Outputs in wider rows: what stands between a row's last value and the next row keeps its
values, where rows start on 16-byte boundaries and end inside 16 bytes too; and what stands
there in the operands (NaN) reaches no value."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import Banded, assert_within
from products import bound, product64, segments, wgrad64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def inside(t, gap):
    """The same values in a tensor whose last dimension is `gap` longer, NaN there."""
    big = torch.full((*t.shape[:-1], t.shape[-1] + gap), NAN, dtype=t.dtype, device="cuda")
    view = big[..., :t.shape[-1]]
    view.copy_(t)
    return big, view


def to16(n):
    return -n % 8 or 8


#: FEW tiles, single CTAs, pairs (with a unit of at most 128 rows), and the 64 x 64 tiles of fp32
LENGTHS = {"few": [3, 0, 20, 1], "single": [40, 0, 100, 65], "pairs": [300, 257, 0, 129]}


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("K,N", [(1, 7), (119, 65), (63, 255), (250, 113), (257, 518), (136, 33)])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_gaps_keep_their_values(lengths, K, N, layout, dtype):
    g = torch.Generator(device="cuda").manual_seed(K + N)
    ix, R, seg = segments(LENGTHS[lengths], 1, 2)
    E, used = len(seg), R - 2
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, dy = inside(r(R, K), to16(K))[1], inside(r(R, N), to16(N))[1]
    if layout == "kn":
        w = inside(r(E, K, N), to16(N))[1]
        dbig, dw = inside(torch.zeros_like(w), to16(N))
    else:
        w = inside(r(E, N, K), to16(K))[1].transpose(1, 2)
        dbig, dw = inside(torch.zeros((E, N, K), dtype=dtype, device="cuda"), to16(K))
        dw = dw.transpose(1, 2)
    y, dx = Banded(R, N, dtype, N + to16(N)), Banded(R, K, dtype, K + to16(K))
    moe.grouped_matmul(x, w, ix, out=y.t)
    moe.grouped_matmul_backward(dy, x, w, ix, drows=dx.t, dw=dw)
    assert y.intact() and dx.intact()
    assert bool(dbig[..., (N if layout == "kn" else K):].isnan().all())
    for got, (ref, mags), n in ((y.t[:used], product64(x, w, seg), K), (dx.t[:used], product64(dy, w.transpose(1, 2), seg), N)):
        assert_within(got, ref[:used], bound(ref, mags, n, dtype)[:used])
    ref, mags = wgrad64(x, dy, seg)
    assert_within(dw, ref, bound(ref, mags, 300, dtype))


def test_the_other_half_of_stored_weights():
    """A gradient of 250 columns beside the 262 that follow them."""
    ix, R, _ = segments([70, 0, 200])
    x, dy = torch.randn((R, 128), device="cuda").to(BF), torch.randn((R, 250), device="cuda").to(BF)
    w, both = torch.empty((3, 128, 250), dtype=BF, device="cuda"), torch.full((3, 128, 512), 5.0, dtype=BF, device="cuda")
    moe.grouped_matmul_backward(dy, x, w, ix, want_drows=False, dw=both[:, :, :250])
    assert bool((both[:, :, 250:] == 5).all())


@pytest.mark.parametrize("N", [1, 100, 129, 250])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gaps_of_8_bit_products(N, dtype):
    g = torch.Generator(device="cuda").manual_seed(N)
    codes, scales = moe.quantize_rows(torch.randn((200, 256), generator=g, device="cuda"))
    w = torch.zeros((256, N + 16 + -N % 16), dtype=torch.uint8, device="cuda")
    w[:, N:] = 127
    y = Banded(200, N, dtype, N + to16(N))
    moe.fp8_matmul(codes, scales, w[:, :N], torch.ones((2, -(-N // 128)), device="cuda"), out=y.t)
    assert y.intact() and bool((y.t == 0).all())
