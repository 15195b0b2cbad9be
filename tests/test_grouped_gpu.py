"""grouped_matmul and its gradients against 64-bit products: segments of any
length, padding, rows of others, layouts, strides and types."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import Banded, assert_within, strided
from products import bound, product64, segments, used_mask, wgrad64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def make(lengths, K, N, dtype, align=1, behind=0, layout="kn", counts=True, seed=0, fill=NAN):
    """Rows, weights and output gradients; every row outside the segments' own holds ``fill``."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ix, R, seg = segments(lengths, align, behind, counts)
    E = len(lengths)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, dy = r(R, K), r(R, N)
    m = used_mask(R, seg)
    x[~m], dy[~m] = fill, fill
    w = r(E, K, N) if layout == "kn" else r(E, N, K).transpose(1, 2)
    return ix, seg, m, x, dy, w


def check_rows(y, ref, mags, terms, used, in_use, what):
    """Values of the used rows, zeros of the padding, untouched rows behind (NaN from the start)."""
    assert_within(y[used], ref[used], bound(ref, mags, terms, y.dtype)[used], what)
    pad = ~used
    pad[in_use:] = False
    assert bool((y[pad] == 0).all()), what + ": padding"
    assert bool(y[in_use:].isnan().all()), what + ": rows behind the segments"


def run_all(lengths, K, N, dtype, align=1, behind=3, layout="kn", counts=True, ld=0, seed=0):
    fill = NAN if counts else 0.0          # without counts the padding rows are rows like the others
    ix, seg, m, x, dy, w = make(lengths, K, N, dtype, align, behind, layout, counts, seed, fill)
    R, in_use = x.shape[0], int(ix["offsets"][-1])
    if not counts:
        x[in_use:], dy[in_use:] = NAN, NAN
    if ld:
        x, dy = strided(x, K + ld), strided(dy, N + ld)
    y, dx = Banded(R, N, dtype, N + ld), Banded(R, K, dtype, K + ld)
    assert moe.grouped_matmul(x, w, ix, out=y.t) is y.t
    dw = torch.full_like(w, NAN)
    moe.grouped_matmul_backward(dy, x, w, ix, drows=dx.t, dw=dw)
    assert moe.products_status() == moe.MOE_OK
    assert y.intact() and dx.intact()
    check_rows(y.t, *product64(x, w, seg), K, m, in_use, "y")
    check_rows(dx.t, *product64(dy, w.transpose(1, 2), seg), N, m, in_use, "dx")
    ref, mags = wgrad64(x, dy, seg)
    longest = max(lengths, default=0)
    assert_within(dw, ref, bound(ref, mags, longest, dtype), "dw")
    for e, n in enumerate(lengths):
        if n == 0:
            assert bool((dw[e] == 0).all()), "an expert without rows"


LENGTHS = {"one_row": [1], "one_expert": [200], "mixed": [5, 0, 130, 1, 0, 64, 257], "empty_ends": [0, 0, 37, 0],
           "tile_edges": [127, 128, 129, 255, 256, 257], "many": [i % 7 for i in range(70)], "none": [0, 0, 0]}


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_products_of_segments(lengths, dtype, layout):
    run_all(LENGTHS[lengths], 136, 200, dtype, layout=layout)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,N", [(1, 1), (1, 8), (8, 1), (7, 5), (63, 65), (64, 64), (65, 127), (128, 256), (129, 257), (96, 520),
                                 (1001, 771), (515, 264), (264, 515)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_products_of_widths(K, N, dtype, layout):
    run_all([33, 0, 150], K, N, dtype, layout=layout, seed=K + N)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("align,counts", [(16, True), (128, True), (128, False), (1, False), (7, False)])
def test_padded_segments(align, counts, dtype):
    run_all([5, 0, 130, 1, 300], 144, 272, dtype, align=align, counts=counts, behind=40)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("ld", [1, 3, 8, 24])
def test_row_strides(ld, dtype):
    run_all([40, 3, 129], 136, 264, dtype, ld=ld)


@pytest.mark.parametrize("lengths", [[600, 511, 513, 0, 1025], [2000], [384] * 9])
@pytest.mark.parametrize("K,N", [(512, 768), (768, 520), (520, 1024)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_longer_segments(lengths, K, N, layout):
    run_all(lengths, K, N, BF, align=1, layout=layout)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33])
def test_a_few_rows_of_many_experts(rows, dtype):
    """A decoded batch: rows spread over a part of the experts."""
    g = torch.Generator().manual_seed(rows)
    lengths = [0] * 40
    for e in torch.randint(0, 40, (rows,), generator=g).tolist():
        lengths[e] += 1
    run_all(lengths, 1024, 640, dtype, behind=2)
    run_all(lengths, 640, 1000, dtype, layout="nk", behind=0)


def test_weights_inside_a_larger_tensor():
    """The gate half of stored [gate | up] weights, and the gradient into the up half."""
    ix, seg, m, x, dy, _ = make([70, 0, 200], 128, 256, BF)
    both = torch.randn((3, 128, 512), device="cuda").to(BF)
    dboth = torch.full_like(both, NAN)
    y = moe.grouped_matmul(x, both[:, :, :256], ix)
    moe.grouped_matmul_backward(dy, x, both[:, :, 256:], ix, dw=dboth[:, :, 256:])
    ref, mags = product64(x, both[:, :, :256], seg)
    assert_within(y[m], ref[m], bound(ref, mags, 128, BF)[m])
    ref, mags = wgrad64(x, dy, seg)
    assert_within(dboth[:, :, 256:], ref, bound(ref, mags, 200, BF))
    assert bool(dboth[:, :, :256].isnan().all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_against_differences(dtype):
    """<Y(x + h u) - Y(x), dy> = h <u, dx>, for x and for w: the product is linear in each."""
    ix, seg, m, x, dy, w = make([9, 0, 60, 31], 72, 88, dtype, fill=0.0)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, ix)
    g = torch.Generator(device="cuda").manual_seed(9)
    u, v = torch.randn(x.shape, generator=g, device="cuda").to(dtype), torch.randn(w.shape, generator=g, device="cuda").to(dtype)
    u[~m] = 0
    for left, right, n in ((moe.grouped_matmul(u, w, ix).double() * dy.double(), u.double() * dx.double(), 88),
                           (moe.grouped_matmul(x, v, ix).double() * dy.double(), v.double() * dw.double(), 60)):
        # each side is a sum of values off by half a step of the type and the fp32 sums behind them
        tol = (2 * 2.0 ** -8 if dtype == BF else 2.0 ** -22) * (left.abs().sum() + right.abs().sum()) + 1e-6 * n
        assert abs(float(left.sum() - right.sum())) <= float(tol)


def test_only_one_gradient():
    ix, seg, m, x, dy, w = make([9, 0, 60], 64, 128, BF)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, ix)
    a, none = moe.grouped_matmul_backward(dy, x, w, ix, want_dw=False)
    assert none is None and torch.equal(a[m], dx[m])
    none, b = moe.grouped_matmul_backward(dy, x, w, ix, want_drows=False)
    assert none is None and torch.equal(b, dw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), NAN])
def test_an_infinity_stays_with_its_row_and_expert(bad, dtype):
    ix, seg, m, x, dy, w = make([20, 40, 30], 136, 72, dtype)
    y0, (dx0, dw0) = moe.grouped_matmul(x, w, ix), moe.grouped_matmul_backward(dy, x, w, ix)
    x2, dy2 = x.clone(), dy.clone()
    x2[25, 3], dy2[70, 5] = bad, bad
    y, (dx, dw) = moe.grouped_matmul(x2, w, ix), moe.grouped_matmul_backward(dy2, x2, w, ix)
    keep = m.clone()
    keep[25] = False
    assert torch.equal(y[keep], y0[keep]) and not bool(y[25].isfinite().any())
    keep = m.clone()
    keep[70] = False
    assert torch.equal(dx[keep], dx0[keep]) and not bool(dx[70].isfinite().any())
    assert torch.equal(dw[0], dw0[0])
    assert not bool(dw[1][3].isfinite().any()) and torch.equal(dw[1][4:], dw0[1][4:])
    assert not bool(dw[2][:, 5].isfinite().any()) and torch.equal(dw[2][:, 6:], dw0[2][:, 6:])


def test_large_magnitudes_and_zeros():
    ix, seg, m, x, dy, w = make([64, 3], 64, 64, BF)
    x[:64] *= 2.0 ** 60
    w *= 2.0 ** -60
    y = moe.grouped_matmul(x, w, ix)
    ref, mags = product64(x, w, seg)
    assert_within(y[m], ref[m], bound(ref, mags, 64, BF)[m])
    z = moe.grouped_matmul(torch.zeros_like(x), w, ix)
    assert bool((z[m] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_same_inputs_give_the_same_bits(dtype):
    ix, seg, m, x, dy, w = make([300, 1, 0, 77, 520], 264, 392, dtype)
    first = (moe.grouped_matmul(x, w, ix)[m], *moe.grouped_matmul_backward(dy, x, w, ix))
    for _ in range(3):
        again = (moe.grouped_matmul(x, w, ix)[m], *moe.grouped_matmul_backward(dy, x, w, ix))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1][m], again[1][m]) and torch.equal(first[2], again[2])


def test_offsets_that_leave_the_buffers_are_clamped():
    """An index of a larger batch over smaller buffers: rows past them do not exist."""
    ix, seg, m, x, dy, w = make([50, 60, 70], 64, 64, BF)
    for bad in ([0, 50, 110, 400], [0, 50, 300, 400], [-5, 50, 110, 180], [0, 110, 50, 180]):
        ix2 = dict(offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        y = Banded(180, 64, BF)
        moe.grouped_matmul(x, w, ix2, out=y.t)
        dw = torch.full_like(w, NAN)
        moe.grouped_matmul_backward(dy, x, w, ix2, dw=dw, drows=y.t)
        assert moe.products_status() == moe.MOE_OK and y.intact()
        assert torch.equal(y.t[:50], moe.grouped_matmul_backward(dy, x, w, ix)[0][:50])
    ix3 = dict(ix, counts=torch.tensor([1000, -4, 70], dtype=torch.int32, device="cuda"))
    y = Banded(180, 64, BF)
    moe.grouped_matmul(x, w, ix3, out=y.t)
    assert y.intact() and bool((y.t[50:110] == 0).all()) and torch.equal(y.t[:50], moe.grouped_matmul(x, w, ix)[:50])


def test_no_rows():
    w = torch.randn((3, 64, 32), device="cuda")
    ix = dict(offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    x, dy = torch.empty((0, 64), device="cuda"), torch.empty((0, 32), device="cuda")
    assert moe.grouped_matmul(x, w, ix).shape == (0, 32)
    dx, dw = moe.grouped_matmul_backward(dy, x, w, ix)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_past_32_bits(dtype):
    """Rows, weights and gradients whose byte and element offsets pass 2^32."""
    K, N, E = 8192, 8192, 40 if dtype == BF else 20
    R = 300000 if dtype == BF else 270000
    x = torch.zeros((R, 16384), device="cuda", dtype=dtype)[:, :K]
    w = torch.zeros((E, K, 2 * N), device="cuda", dtype=dtype)[:, :, :N]
    lengths = [0] * E
    lengths[0], lengths[E - 2], lengths[E - 1] = R - 40, 23, 17
    offsets = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    # the first expert's rows are padding of its segment but for three
    counts = torch.tensor([3] + lengths[1:], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    used = torch.cat([torch.arange(3), torch.arange(R - 40, R)]).cuda()
    x[used] = torch.randn((43, K), generator=g, device="cuda").to(dtype)
    for e in (0, E - 2, E - 1):
        w[e] = torch.randn((K, N), generator=g, device="cuda").to(dtype)
    ix = dict(offsets=offsets, counts=counts)
    y = moe.grouped_matmul(x, w, ix)
    dx, dw = moe.grouped_matmul_backward(y, x, w, ix)
    assert moe.products_status() == moe.MOE_OK
    at = 0
    for e, n in ((0, 3), (E - 2, 23), (E - 1, 17)):
        rows = used[at:at + n]
        at += n
        xe, we, ye = x[rows].double(), w[e].double(), y[rows].double()
        ref, mags = xe @ we, xe.abs() @ we.abs()
        assert_within(y[rows], ref, bound(ref, mags, K, dtype), f"y of {e}")
        ref, mags = ye @ we.T, ye.abs() @ we.abs().T
        assert_within(dx[rows], ref, bound(ref, mags, N, dtype), f"dx of {e}")
        ref, mags = xe.T @ ye, xe.abs().T @ ye.abs()
        assert_within(dw[e], ref, bound(ref, mags, n, dtype), f"dw of {e}")
    assert bool((dw[1:E - 2] == 0).all()) and bool((y[3:R - 40:997] == 0).all())
