"""moe_add_rms_norm and its backward against the formulas in 64 bits.

Bounds count roundings (u = 2^-24 for fp32, half a step of the stored type on
top). A row's sum of squares is added in chains of at most H/128 + 144 fp32
operations, so rstd is off by at most half of that, plus the two ulp of the
reciprocal root; a normalised value carries three more roundings."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import U32, UNIT, Banded, assert_within, strided

pytestmark = pytest.mark.gpu

EPS = 1e-6
SHAPES = [(1, 1), (1, 7), (11, 15), (350, 17), (1, 7168), (3, 31), (5, 33), (4, 64), (130, 128), (129, 257), (7, 1001), (9, 1002), (33, 1024),
          (64, 2050), (300, 4096), (17, 7168), (5, 8192), (3, 12289), (4, 16384), (2, 32768), (2, 40000),
          (700, 96), (2000, 136), (2500, 131), (2600, 1023), (400, 4101), (3, 20001)]
DTYPES = [torch.float32, torch.bfloat16]


def chain(H):
    return H / 128 + 144


def rel32(H):
    return (chain(H) / 2 + 8) * U32


def inputs(rows, H, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(1000 * rows + H + seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    chan = torch.exp(r(H))
    return dict(x=(r(rows, H) * chan).to(dtype), r=(r(rows, H) * chan * 2).to(dtype), w=1 + 0.3 * r(H),
                dy=r(rows, H).to(dtype), dh=r(rows, H).to(dtype))


def reference(x, r, w, eps=EPS):
    s = x.double() + (0 if r is None else r.double())
    rstd = 1 / ((s * s).mean(1) + eps).sqrt()
    return s, rstd, s * rstd[:, None] * w.double()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", SHAPES)
def test_forward(rows, H, dtype, residual):
    i = inputs(rows, H, dtype)
    r = i["r"] if residual else None
    by, bh = Banded(rows, H, dtype), Banded(rows, H, dtype)
    out = moe.add_rms_norm(i["x"], i["w"], r, eps=EPS, want_rstd=True, y=by.t, h=bh.t if residual else None)
    s, rstd, y = reference(i["x"], r, i["w"])
    u = UNIT[dtype]
    assert_within(out["y"], y, y.abs() * (u + rel32(H)) + 1e-37, "y")
    assert_within(out["rstd"], rstd, rstd * rel32(H), "rstd")
    assert by.intact()
    if residual:
        # the fp32 sum, then the stored type
        assert_within(out["h"], s, s.abs() * (u + U32 * (1 + u)) + 1e-37, "h")
        assert bh.intact()
    else:
        assert "h" not in out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H,ld", [(5, 96, 104), (5, 96, 97), (6, 1002, 1004), (4, 1001, 1003), (3, 4096, 4104),
                                       (3, 4096, 4097), (2, 40000, 40002)])
def test_row_strides(rows, H, ld, dtype):
    i = inputs(rows, H, dtype)
    x, r, dy, dh = (strided(i[n], ld + 8 * k) for k, n in enumerate(("x", "r", "dy", "dh")))
    by, bh, bd = Banded(rows, H, dtype, ld), Banded(rows, H, dtype, ld + 16), Banded(rows, H, dtype, ld)
    out = moe.add_rms_norm(x, i["w"], r, eps=EPS, want_rstd=True, y=by.t, h=bh.t)
    flat = moe.add_rms_norm(i["x"], i["w"], i["r"], eps=EPS, want_rstd=True)
    s, rstd, y = reference(i["x"], i["r"], i["w"])
    assert_within(out["y"], y, y.abs() * (UNIT[dtype] + rel32(H)) + 1e-37, "y")
    assert torch.equal(out["h"], flat["h"])
    assert by.intact() and bh.intact()
    dx, dw = moe.add_rms_norm_backward(dy, out["h"], out["rstd"], i["w"], dh, dx=bd.t)
    check_backward(dx, dw, i["dy"], flat["h"], out["rstd"], i["w"], i["dh"])
    assert bd.intact()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", [(5, 97), (700, 96), (9, 1002), (400, 4099), (3, 16000), (2, 40001)])
def test_row_strides_that_differ(rows, H, dtype):
    """Every tensor's rows start on boundaries of their own."""
    i = inputs(rows, H, dtype)
    x, r, dy, dh = (strided(i[n], H + k) for n, k in (("x", 1), ("r", 2), ("dy", 3), ("dh", 6)))
    by, bh, bd = Banded(rows, H, dtype, H + 5), Banded(rows, H, dtype, H + 8), Banded(rows, H, dtype, H)
    out = moe.add_rms_norm(x, i["w"], r, eps=EPS, want_rstd=True, y=by.t, h=bh.t)
    s, rstd, y = reference(i["x"], i["r"], i["w"])
    assert_within(out["y"], y, y.abs() * (UNIT[dtype] + rel32(H)) + 1e-37, "y")
    assert_within(out["h"], s, s.abs() * (UNIT[dtype] + U32 * (1 + UNIT[dtype])) + 1e-37, "h")
    dx, dw = moe.add_rms_norm_backward(dy, out["h"], out["rstd"], i["w"], dh, dx=bd.t)
    check_backward(dx, dw, i["dy"], out["h"].contiguous(), out["rstd"], i["w"], i["dh"])
    assert by.intact() and bh.intact() and bd.intact()


def check_backward(dx, dw, dy, h, rstd, w, dh):
    rows, H = h.shape
    g, v, r, w = dy.double(), h.double(), rstd.double()[:, None], w.double()
    n = v * r
    m = (w * g * n).mean(1, keepdim=True)
    ref = r * (w * g - n * m) + (0 if dh is None else dh.double())
    mabs = (w * g * n).abs().mean(1, keepdim=True)
    bound = ref.abs() * UNIT[h.dtype] + U32 * (
        6 * ((r * w * g).abs() + (r * n * m).abs() + (0 if dh is None else dh.double().abs()))
        + (chain(H) + 6) * (r * n).abs() * mabs)
    assert_within(dx, ref, bound + 1e-37, "dx")
    if dw is not None:
        # a row's term carries two roundings; rows are added in chains of at most rows/152 + 64
        assert_within(dw, (g * n).sum(0), U32 * (rows / 152 + 64) * (g * n).abs().sum(0) + 1e-37, "dweight")


@pytest.mark.parametrize("dh", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", SHAPES)
def test_backward(rows, H, dtype, dh):
    i = inputs(rows, H, dtype)
    rstd = torch.rsqrt(i["x"].float().square().mean(1) + EPS)
    b = Banded(rows, H, dtype)
    dx, dw = moe.add_rms_norm_backward(i["dy"], i["x"], rstd, i["w"], i["dh"] if dh else None, dx=b.t)
    check_backward(dx, dw, i["dy"], i["x"], rstd, i["w"], i["dh"] if dh else None)
    assert b.intact()
    alone, none = moe.add_rms_norm_backward(i["dy"], i["x"], rstd, i["w"], i["dh"] if dh else None, want_dweight=False)
    assert none is None and torch.equal(alone, dx)


def test_gradient_against_differences():
    """d/dx and d/dw of sum(dy y) by central differences of the 64-bit formula."""
    rows, H = 3, 37
    i = inputs(rows, H, torch.float32, 5)
    out = moe.add_rms_norm(i["x"], i["w"], i["r"], eps=EPS, want_rstd=True)
    dx, dw = moe.add_rms_norm_backward(i["dy"], out["h"], out["rstd"], i["w"])
    loss = lambda x, w: (reference(x, i["r"], w)[2] * i["dy"].double()).sum()  # noqa: E731
    x, w = i["x"].double(), i["w"].double()
    d = 1e-6
    for at in [(0, 0), (1, 20), (2, 36)]:
        e = torch.zeros_like(x)
        e[at] = d
        num = (loss(x + e, w) - loss(x - e, w)) / (2 * d)
        # truncation d^2 and cancellation 1e-16/d of the differences, fp32 roundings of dx
        assert abs(num - dx[at].double()) <= 1e-5 * dx.double().abs().max()
    for c in (0, 19, 36):
        e = torch.zeros_like(w)
        e[c] = d
        num = (loss(x, w + e) - loss(x, w - e)) / (2 * d)
        assert abs(num - dw[c].double()) <= 1e-5 * dw.double().abs().max()


def e4m3_error(q):
    """Half an E4M3 step at |q| (2^-10 in the subnormal range)."""
    return (q.abs() * 2.0 ** -4).clamp_min(2.0 ** -10)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("quant", [moe.MOE_NORM_FP8_BLOCK, moe.MOE_NORM_MXFP8])
@pytest.mark.parametrize("rows,H", [(1, 128), (1, 7168), (8, 256), (127, 384), (128, 1024), (129, 4096), (260, 640),
                                    (3, 16384), (2, 32768), (2, 40960)])
@pytest.mark.parametrize("residual", [False, True])
def test_eight_bit_output(rows, H, dtype, quant, residual):
    i = inputs(rows, H, dtype)
    if rows > 1:
        i["x"][1] = 0
        i["r"][1] = 0
    i["w"][32:64] = 0           # blocks of zeros
    r = i["r"] if residual else None
    out = moe.add_rms_norm(i["x"], i["w"], r, eps=EPS, quant=quant, want_y=False)
    both = moe.add_rms_norm(i["x"], i["w"], r, eps=EPS, quant=quant, want_rstd=True)
    assert "y" not in out and torch.equal(out["codes"], both["codes"]) and torch.equal(out["scales"], both["scales"])
    s, rstd, y = reference(i["x"], r, i["w"])
    assert_within(both["y"], y, y.abs() * (UNIT[dtype] + rel32(H)) + 1e-37, "y")
    codes = out["codes"].view(torch.float8_e4m3fn).double()
    assert not bool(codes.isnan().any())
    rel = rel32(H)
    if quant == moe.MOE_NORM_FP8_BLOCK:
        amax = y.abs().view(rows, H // 128, 128).amax(2)
        ref = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        assert_within(out["scales"], ref, ref * (rel + U32), "scales")
        sc = out["scales"].double().repeat_interleave(128, 1)
    else:
        atoms = out["scales"].view(-1, H // 128, 32, 4, 4)     # [tile][k block][m % 32][m / 32][sub-block]
        e = atoms.permute(0, 3, 2, 1, 4).reshape(-1, H // 32).int()
        assert bool((e[rows:] == 0).all())                    # rows past the last one
        e = e[:rows] - 127
        amax = y.abs().view(rows, H // 32, 32).amax(2)
        up = lambda a: torch.where(a > 0, torch.ceil(torch.log2(a / 448)).clamp(-127, 127), torch.full_like(a, -127.0))  # noqa: E731
        assert bool(((e >= up(amax * (1 - rel))) & (e <= up(amax * (1 + rel)))).all())
        sc = torch.ldexp(torch.ones_like(amax), e).repeat_interleave(32, 1)
    q = y / sc
    assert_within(codes, q, e4m3_error(q) + q.abs() * 2 * (rel + 2 * U32), "codes")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", [100, 1001, 4096, 40000])
def test_in_place(H, dtype):
    i = inputs(6, H, dtype)
    ref = moe.add_rms_norm(i["x"], i["w"], i["r"], want_rstd=True)
    x, r = i["x"].clone(), i["r"].clone()
    out = moe.add_rms_norm(x, i["w"], r, h=r, y=x, want_rstd=True)
    assert out["h"] is r and out["y"] is x
    assert torch.equal(r, ref["h"]) and torch.equal(x, ref["y"])
    dx, dw = moe.add_rms_norm_backward(i["dy"], r, out["rstd"], i["w"], i["dh"])
    for k in ("dy", "dh"):
        j = {n: i[n].clone() for n in ("dy", "dh")}
        dx2, dw2 = moe.add_rms_norm_backward(j["dy"], r, out["rstd"], i["w"], j["dh"], dx=j[k])
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_no_rows():
    x = torch.empty((0, 256), device="cuda")
    w = torch.ones(256, device="cuda")
    for q in (moe.MOE_NORM_PLAIN, moe.MOE_NORM_FP8_BLOCK, moe.MOE_NORM_MXFP8):
        assert moe.add_rms_norm(x, w, x, quant=q)["y"].shape == (0, 256)
    dx, dw = moe.add_rms_norm_backward(x, x, torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 256) and bool((dw == 0).all())


def test_rows_that_are_not_finite_stay_in_their_row():
    i = inputs(6, 512, torch.bfloat16)
    x = i["x"].clone()
    x[2, 7] = float("inf")
    x[4, 9] = float("nan")
    ref = moe.add_rms_norm(i["x"], i["w"], quant=moe.MOE_NORM_MXFP8, want_rstd=True)
    out = moe.add_rms_norm(x, i["w"], quant=moe.MOE_NORM_MXFP8, want_rstd=True)
    keep = [0, 1, 3, 5]
    for n in ("y", "codes", "rstd"):
        assert torch.equal(out[n][keep], ref[n][keep])
    assert out["rstd"][2] == 0 and bool(out["rstd"][4].isnan()) and bool(out["y"][4].isnan().all())


def test_zero_eps_and_tiny_values():
    x = torch.full((2, 300), 1e-15, device="cuda")
    w = torch.ones(300, device="cuda")
    _, rstd, y = reference(x, None, w, 1e-6)
    out = moe.add_rms_norm(x, w, eps=1e-6, want_rstd=True)
    assert_within(out["y"], y, y.abs() * rel32(300), "y")
    out = moe.add_rms_norm(x, w, eps=0.0)
    _, rstd, y = reference(x, None, w, 0.0)
    assert_within(out["y"], y, y.abs() * rel32(300), "y")


def test_side_stream_graph_and_repeatability():
    i = inputs(37, 2050, torch.bfloat16)
    first = moe.add_rms_norm(i["x"], i["w"], i["r"], want_rstd=True)
    fdx, fdw = moe.add_rms_norm_backward(i["dy"], first["h"], first["rstd"], i["w"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x = i["x"].clone()
    with torch.cuda.stream(side):
        out = moe.add_rms_norm(x, i["w"], i["r"], want_rstd=True)
        dx, dw = moe.add_rms_norm_backward(i["dy"], out["h"], out["rstd"], i["w"])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in ((out["y"], first["y"]), (dx, fdx), (dw, fdw)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = moe.add_rms_norm(x, i["w"], i["r"], want_rstd=True)
        dx, dw = moe.add_rms_norm_backward(i["dy"], out["h"], out["rstd"], i["w"])
    x.copy_(i["dh"])
    g.replay()
    torch.cuda.synchronize()
    ref = moe.add_rms_norm(i["dh"], i["w"], i["r"], want_rstd=True)
    rdx, rdw = moe.add_rms_norm_backward(i["dy"], ref["h"], ref["rstd"], i["w"])
    assert all(torch.equal(a, b) for a, b in ((out["y"], ref["y"]), (dx, rdx), (dw, rdw)))


@pytest.mark.parametrize("H", [7168, 7167])
def test_far_rows(H):
    """More than 2^31 values: offsets past 32 bits, in every output."""
    rows = (1 << 31) // H + 1000
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((rows, H), generator=g, device="cuda", dtype=torch.bfloat16)
    w = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    at = [0, 1, rows // 2, rows - 2, rows - 1]
    quants = (moe.MOE_NORM_PLAIN,) if H % 128 else (moe.MOE_NORM_FP8_BLOCK, moe.MOE_NORM_MXFP8)
    _, rstd, y = reference(x[at], None, w)
    for q in quants:
        out = moe.add_rms_norm(x, w, eps=EPS, quant=q, want_rstd=True)
        assert_within(out["y"][at], y, y.abs() * (UNIT[torch.bfloat16] + rel32(H)) + 1e-37, "y")
        assert_within(out["rstd"][at], rstd, rstd * rel32(H), "rstd")
        if q != moe.MOE_NORM_PLAIN:
            few = moe.add_rms_norm(x[at], w, eps=EPS, quant=q)
            # the few rows go through another kernel: rstd may differ in its last bits
            assert float((out["codes"][at] != few["codes"]).float().mean()) < 1e-3
            if q == moe.MOE_NORM_FP8_BLOCK:
                assert_within(out["scales"][at], few["scales"].double(), few["scales"].double() * 2 * rel32(H), "scales")
    r = out["rstd"]
    del out
    dx, dw = moe.add_rms_norm_backward(x, x, r, w)
    check_backward(dx[at], None, x[at], x[at], r[at], w, None)
    # dw = sum of x^2 rstd, every row's terms positive
    ref = torch.zeros(H, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 20000):
        ref += (x[i:i + 20000].double().square() * r[i:i + 20000, None].double()).sum(0)
    assert_within(dw, ref, U32 * (rows / 152 + 64) * ref, "dweight")
