"""fp8_matmul, quantize_rows and quantize_tiles: the product of the codes' values
in 64 bits, the codes against a division in fp32, and the way from rows to
products."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import Banded, assert_within
from products import bound, product64, segments, tile_values8, used_mask, values8

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def rand_codes(g, *shape):
    """Any finite E4M3 code."""
    c = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.int32)
    return torch.where((c & 127) == 127, c - 1, c).to(torch.uint8)


def make(lengths, K, N, align=1, behind=0, layout="kn", counts=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ix, R, seg = segments(lengths, align, behind, counts)
    E, nb = len(lengths), -(-N // 128)
    a, sa = rand_codes(g, R, K), torch.rand((R, K // 128), generator=g, device="cuda") + 0.1
    if layout == "kn":
        b, sb = rand_codes(g, E, K, -(-N // 16) * 16)[:, :, :N], torch.rand((E, K // 128, nb), generator=g, device="cuda")
    else:
        b, sb = rand_codes(g, E, N, K).transpose(1, 2), torch.rand((E, nb, K // 128), generator=g, device="cuda").transpose(1, 2)
    m = used_mask(R, seg)
    if counts:                                  # what is not a row of an expert is NaN
        a[~m], sa[~m] = 127, NAN
    return ix, seg, m, a, sa, b, sb


def run(lengths, K, N, dtype, align=1, behind=3, layout="kn", counts=True, seed=0):
    ix, seg, m, a, sa, b, sb = make(lengths, K, N, align, behind, layout, counts, seed)
    R, in_use = a.shape[0], int(ix["offsets"][-1])
    if not counts:
        seg = [(int(o), int(n - o)) for o, n in zip(ix["offsets"][:-1], ix["offsets"][1:])]
        m = used_mask(R, seg)
    y = Banded(R, N, dtype, N + (0 if N % 8 else 8))
    moe.fp8_matmul(a, sa, b, sb, ix, out=y.t)
    assert moe.products_status() == moe.MOE_OK and y.intact()
    ref, mags = product64(values8(a, sa), tile_values8(b, sb), seg)
    # the code products and their sums as any fp32 sum, and two more roundings for a block's scales
    assert_within(y.t[m], ref[m], bound(ref, mags, K + 2, dtype)[m], "y")
    pad = ~m
    pad[in_use:] = False
    assert bool((y.t[pad] == 0).all()) and bool(y.t[in_use:].isnan().all())


LENGTHS = {"one_row": [1], "one_expert": [200], "mixed": [5, 0, 130, 1, 0, 64, 257], "tile_edges": [127, 128, 129, 255, 256, 257],
           "many": [i % 7 for i in range(70)], "none": [0, 0, 0]}


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_products_of_segments(lengths, dtype, layout):
    run(LENGTHS[lengths], 384, 272, dtype, layout=layout)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("K,N", [(128, 1), (128, 16), (256, 100), (128, 128), (640, 129), (256, 256), (1024, 520), (2048, 1000)])
def test_products_of_widths(K, N, layout):
    run([33, 0, 150], K, N, BF, layout=layout, seed=N)
    run([300], K, N, F32, layout=layout, seed=N)


@pytest.mark.parametrize("align,counts", [(16, True), (128, True), (128, False), (1, False)])
def test_padded_segments(align, counts):
    run([5, 0, 130, 1, 300], 256, 272, BF, align=align, counts=counts, behind=40)


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 33])
def test_a_few_rows_of_many_experts(rows):
    g = torch.Generator().manual_seed(rows)
    lengths = [0] * 40
    for e in torch.randint(0, 40, (rows,), generator=g).tolist():
        lengths[e] += 1
    run(lengths, 1024, 640, BF, behind=2)
    run(lengths, 2048, 400, F32, layout="nk", behind=0)


@pytest.mark.parametrize("M", [1, 8, 17, 128, 300, 1111])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_dense(M, layout):
    """Without an index: one matrix of weights for all rows."""
    ix, seg, m, a, sa, b, sb = make([M], 1024, 784, layout=layout)
    y = moe.fp8_matmul(a, sa, b[0], sb[0])
    assert y.dtype == BF
    ref, mags = product64(values8(a, sa), tile_values8(b, sb), seg)
    assert_within(y, ref, bound(ref, mags, 1026, BF))
    z = moe.fp8_matmul(a, sa, b[0], sb[0], dtype=F32)
    assert_within(z, ref, bound(ref, mags, 1026, F32))


def test_the_transposed_view_of_the_same_codes():
    """quantize_tiles once, the product and that of the gradient from it."""
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randn((3, 256, 384), generator=g, device="cuda").to(BF)
    codes, scales = moe.quantize_tiles(w)
    tiles = w.float().view(3, 2, 128, 3, 128).abs().amax((2, 4))
    assert torch.equal(scales, tiles / torch.full_like(tiles, 448))
    ix, R, seg = segments([40, 0, 90])
    x, dy = torch.randn((R, 256), generator=g, device="cuda").to(BF), torch.randn((R, 384), generator=g, device="cuda").to(BF)
    (a, sa), (d, sd) = moe.quantize_rows(x), moe.quantize_rows(dy)
    y = moe.fp8_matmul(a, sa, codes, scales, ix)
    dx = moe.fp8_matmul(d, sd, codes.transpose(1, 2), scales.transpose(1, 2), ix)
    wv = tile_values8(codes, scales)
    ref, mags = product64(values8(a, sa), wv, seg)
    assert_within(y, ref, bound(ref, mags, 258, BF))
    ref, mags = product64(values8(d, sd), wv.transpose(1, 2), seg)
    assert_within(dx, ref, bound(ref, mags, 386, BF))
    # the codes stand for the values within half a step of E4M3 each (and its smallest step)
    full, fm = product64(x, w, seg)
    step = (2 * 2.0 ** -4 + 2.0 ** -8) * fm
    small = 2.0 ** -10 * (sa.double().repeat_interleave(128, 1).amax(1, keepdim=True) * wv.abs().amax() * 256 +
                          scales.amax().double() * values8(a, sa).abs().amax() * 256)
    assert_within(y, full, step + small + 2.0 ** -8 * full.abs() + 1e-3)
    sq, tq = moe.quantize_tiles(w[1].contiguous())
    assert torch.equal(sq, codes[1]) and torch.equal(tq, scales[1])


def test_norm_codes_into_a_product():
    """One decoded token: the norm's blockwise codes times 8-bit weights."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x, wn = torch.randn((5, 512), generator=g, device="cuda").to(BF), torch.rand(512, generator=g, device="cuda") + 0.5
    n = moe.add_rms_norm(x, wn, quant=moe.MOE_NORM_FP8_BLOCK, want_y=False)
    codes, scales = moe.quantize_tiles(torch.randn((512, 256), generator=g, device="cuda").to(BF))
    y = moe.fp8_matmul(n["codes"], n["scales"], codes, scales)
    a, w = values8(n["codes"], n["scales"]), tile_values8(codes, scales)
    ref, mags = a @ w, a.abs() @ w.abs()
    assert_within(y, ref, bound(ref, mags, 514, BF))


def test_nan_codes_and_infinite_scales_stay_with_their_row():
    ix, seg, m, a, sa, b, sb = make([20, 40, 30], 256, 144)
    y0 = moe.fp8_matmul(a, sa, b, sb, ix)
    a2, sa2 = a.clone(), sa.clone()
    a2[25, 3], sa2[70, 1] = 127, float("inf")
    y = moe.fp8_matmul(a2, sa2, b, sb, ix)
    keep = m.clone()
    keep[25], keep[70] = False, False
    assert torch.equal(y[keep], y0[keep])
    assert bool(y[25].isnan().all()) and not bool(y[70].isfinite().any())


@pytest.mark.parametrize("M", [1, 1000, 4096])
def test_the_same_inputs_give_the_same_bits(M):
    ix, seg, m, a, sa, b, sb = make([M, 3], 512, 656)
    y = moe.fp8_matmul(a, sa, b, sb, ix)
    for _ in range(3):
        assert torch.equal(moe.fp8_matmul(a, sa, b, sb, ix), y)


def test_offsets_past_32_bits():
    """Codes whose offsets pass 2^32 on either side."""
    K, N, E = 8192, 8192, 70
    R = 600000
    a = torch.zeros((R, K), dtype=torch.uint8, device="cuda")
    sa = torch.ones((R, K // 128), device="cuda")
    b = torch.zeros((E, K, N), dtype=torch.uint8, device="cuda")
    sb = torch.ones((E, K // 128, N // 128), device="cuda")
    lengths = [0] * E
    lengths[0], lengths[E - 1] = R - 40, 40
    ix = dict(offsets=torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device="cuda"),
              counts=torch.tensor([3] + lengths[1:], dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(1)
    used = torch.cat([torch.arange(3), torch.arange(R - 40, R)]).cuda()
    a[used] = rand_codes(g, 43, K)
    for e in (0, E - 1):
        b[e] = rand_codes(g, K, N)
    y = moe.fp8_matmul(a, sa, b, sb, ix)
    for e, rows in ((0, used[:3]), (E - 1, used[3:])):
        av, bv = values8(a[rows], sa[rows]), tile_values8(b[e], sb[e])
        ref, mags = av @ bv, av.abs() @ bv.abs()
        assert_within(y[rows], ref, bound(ref, mags, K + 2, BF), f"{e}")
    assert bool((y[3:R - 40:997] == 0).all())


def reference_codes(x):
    b = x.float().cpu().view(x.shape[0], -1, 128)
    amax = b.abs().amax(2)
    s = amax / torch.full_like(amax, 448)
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(x.shape), s


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,K", [(1, 128), (3, 256), (33, 7168), (127, 640), (1000, 1152), (513, 128)])
def test_row_codes(R, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(R + K)
    x = (torch.randn((R, K), generator=g, device="cuda") * torch.exp(3 * torch.randn((R, 1), generator=g, device="cuda"))).to(dtype)
    x[0, :128] = 0
    x[R // 2, 5] = -0.0
    x[R - 1, :] *= 1e-36 if dtype == F32 else 1e-30
    big = torch.zeros((R, K + 16), device="cuda", dtype=dtype)
    big[:, :K] = x
    want, ws = reference_codes(x)
    for src in (x, big[:, :K]):
        codes, scales = Banded(R, K, torch.uint8, K + 32), Banded(R, K // 128, F32, K // 128 + 3)
        moe.quantize_rows(src, codes=codes.t, scales=scales.t)
        assert torch.equal(codes.t.cpu(), want) and torch.equal(scales.t.cpu(), ws)
        assert codes.intact() and scales.intact()


def test_row_codes_stop_at_the_rows_in_use():
    ix, R, seg = segments([5, 0, 70], 16, 9)
    x = torch.randn((R, 384), device="cuda").to(BF)
    codes, scales = torch.full((R, 384), 7, dtype=torch.uint8, device="cuda"), torch.full((R, 3), NAN, device="cuda")
    moe.quantize_rows(x, ix, codes=codes, scales=scales)
    n = int(ix["offsets"][-1])
    want, ws = moe.quantize_rows(x)
    assert torch.equal(codes[:n], want[:n]) and torch.equal(scales[:n], ws[:n])
    assert bool((codes[n:] == 7).all()) and bool(scales[n:].isnan().all())


def test_row_codes_of_infinities_and_nan():
    x = torch.randn((4, 256), device="cuda")
    x[1, 3], x[2, 200], x[3, 7] = float("inf"), NAN, float("-inf")
    codes, scales = moe.quantize_rows(x)
    clean, cs = moe.quantize_rows(torch.where(x.isfinite(), x, torch.zeros((), device="cuda")))
    assert bool(scales[1, 0].isinf()) and bool(scales[3, 0].isinf())
    assert int(codes[2, 200]) & 127 == 127 and torch.equal(codes[0], clean[0]) and torch.equal(codes[2, :128], clean[2, :128])
    assert torch.equal(codes[1, 128:], clean[1, 128:]) and torch.equal(scales[2], cs[2])


def test_row_codes_past_32_bits():
    x = torch.zeros((140000, 32768), device="cuda", dtype=BF)
    x[-3:] = torch.randn((3, 32768), device="cuda").to(BF)
    codes, scales = moe.quantize_rows(x)
    want, ws = reference_codes(x[-3:])
    assert torch.equal(codes[-3:].cpu(), want) and torch.equal(scales[-3:].cpu(), ws)
    assert bool((codes[:-3:1009] == 0).all()) and bool((scales[:-3] == 1).all())
