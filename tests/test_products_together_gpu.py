"""The products as a model uses them: an expert block between the token sort and
the way back, its gradients against autograd in 64 bits, on a layer's routing,
in captured graphs, on several streams, and with 8-bit weights."""
import os
import sys

import pytest
import torch

import moe_inputs as mi
import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import assert_within
from products import bound, product64, tile_values8, used_mask, values8, wgrad64

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from block_step import Blocks  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def routing(T, k, E, seed, drop=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    topk = torch.rand((T, E), generator=g, device="cuda").topk(k, 1).indices.int()
    if drop:
        topk[torch.rand((T, k), generator=g, device="cuda") < drop] = -1
    return topk.contiguous(), torch.rand((T, k), generator=g, device="cuda")


@pytest.mark.parametrize("align,drop", [(1, 0.0), (1, 0.2), (16, 0.1), (128, 0.0)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_an_expert_block_and_its_gradients(align, drop, layout):
    """y = sum_j g_j relu(x A_e)^2 B_e in fp32 against autograd of the same in 64 bits."""
    T, k, E, H, F = 150, 3, 7, 96, 160
    g = torch.Generator(device="cuda").manual_seed(align)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    topk, gates = routing(T, k, E, 5, drop)
    x, dout = r(T, H), r(T, H)
    w = lambda K, N: (r(E, K, N) if layout == "kn" else r(E, N, K).transpose(1, 2)).mul_(K ** -0.5)  # noqa: E731
    A, B = w(H, F), w(F, H)

    ix = moe.sort_index(topk, E, align)
    X = moe.sort_rows(x, ix)
    Z = moe.grouped_matmul(X, A, ix)
    R = Z.relu().square()
    Y = moe.grouped_matmul(R, B, ix)
    y = moe.unsort_rows(Y, ix, gates)
    dY, dg = moe.unsort_rows_backward(dout, Y, ix, gates)
    dR, dB = moe.grouped_matmul_backward(dY, R, B, ix)
    dX, dA = moe.grouped_matmul_backward(2 * Z.relu() * dR, X, A, ix)
    dx = moe.unsort_rows(dX, ix)
    assert moe.products_status() == moe.MOE_OK

    leaves = [v.double().requires_grad_() for v in (x, A, B, gates)]
    x6, A6, B6, g6 = leaves
    ref = torch.zeros_like(x6)
    for j in range(k):
        for e in range(E):
            ref = ref + (g6[:, j] * (topk[:, j] == e)).unsqueeze(1) * ((x6 @ A6[e]).relu().square() @ B6[e])
    ref.backward(dout.double())
    # sums of up to 160 fp32 products, four in a row (and, for weights, of about 65 rows): far below 1e-5
    for name, got, want in (("y", y, ref.detach()), ("dx", dx, x6.grad), ("dA", dA, A6.grad), ("dB", dB, B6.grad), ("dg", dg, g6.grad)):
        err = float((got.double() - want).norm() / want.norm())
        assert err < 1e-5, (name, err)


def test_on_a_layers_routing():
    """The offsets, counts and rows that a layer's forward returns (128-row segments)."""
    w = mi.scaled(mi.WORKLOADS["qwen3_235b"], T=300, H=256, E=16, k=4, F=128)
    g = {n: (None if v is None else v.cuda()) for n, v in mi.make_inputs(w, with_grad_out=False).items()}
    layer = moe.MoELayer(w.H, w.E, w.F, w.k, w.T, score=w.score)
    _, r = layer.forward(g["x"], g["Wr"], g["b"], g["Wg"], g["Wu"], g["Wd"], routing=True)
    ix = {n: r[n] for n in ("offsets", "counts", "row_of")}
    rows = moe.moe_sort_rows_cap(w.T, w.k, w.E, 128)
    X = moe.sort_rows(g["x"], ix, out=torch.full((rows, w.H), float("nan"), dtype=BF, device="cuda"))  # padding stays NaN
    Y = moe.grouped_matmul(X, g["Wg"], ix)
    dX, dW = moe.grouped_matmul_backward(Y, X, g["Wg"], ix)
    seg = list(zip(r["offsets"][:-1].tolist(), r["counts"].tolist()))
    m = used_mask(rows, seg)
    ref, mags = product64(X, g["Wg"], seg)
    assert_within(Y[m], ref[m], bound(ref, mags, w.H, BF)[m])
    ref, mags = wgrad64(X, Y, seg)
    assert_within(dW, ref, bound(ref, mags, max(n for _, n in seg), BF))
    used = int(r["offsets"][-1])
    pad = ~m
    pad[used:] = False
    assert bool((Y[pad] == 0).all()) and bool((dX[pad] == 0).all())


def test_a_captured_step_follows_its_inputs():
    """One graph of index, rows, products, gradients and codes; replays with other tokens and routing."""
    T, k, E, H, F, al = 130, 2, 9, 256, 384, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    A = (torch.randn((E, H, F), generator=g, device="cuda") / 16).to(BF)
    codes, scales = moe.quantize_tiles(A)
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    topk = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    rows = moe.moe_sort_rows_cap(T, k, E, al)
    bufs = lambda: dict(X=torch.zeros((rows, H), dtype=BF, device="cuda"), Y=torch.zeros((rows, F), dtype=BF, device="cuda"),  # noqa: E731
                        dX=torch.zeros((rows, H), dtype=BF, device="cuda"), Y8=torch.zeros((rows, F), dtype=BF, device="cuda"))

    def step(b):
        ix = moe.sort_index(topk, E, al)
        X = moe.sort_rows(x, ix, out=b["X"])
        Y = moe.grouped_matmul(X, A, ix, out=b["Y"])
        dX, dA = moe.grouped_matmul_backward(Y, X, A, ix, drows=b["dX"])
        c, s = moe.quantize_rows(X, ix)
        Y8 = moe.fp8_matmul(c, s, codes, scales, ix, out=b["Y8"])
        return ix["offsets"], X, Y, dX, dA, Y8

    step(bufs())                                         # the first call of each kernel is not captured
    b1, gr = bufs(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step(b1)
    for seed in range(4):
        t2, _ = routing(T, k, E, seed, 0.3 * seed)
        x.copy_(torch.randn((T, H), device="cuda"))
        topk.copy_(t2)
        gr.replay()
        want = step(bufs())
        n = int(want[0][-1])
        for a, b in zip(got, want):
            a, b = (a[:n], b[:n]) if a.shape[0] == rows else (a, b)
            assert torch.equal(a, b)
    assert moe.products_status() == moe.MOE_OK


def test_two_streams_at_once():
    """The same calls on two streams, together: nothing is shared between them."""
    sets = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        topk, _ = routing(700, 2, 6, seed)
        ix = moe.sort_index(topk, 6)
        x = torch.randn((1400, 520), generator=g, device="cuda").to(BF)
        w = torch.randn((6, 520, 264), generator=g, device="cuda").to(BF)
        wf, xf = w.float(), x.float()
        c, s = moe.quantize_rows(x[:, :512])
        q, t = moe.quantize_tiles(torch.randn((6, 512, 256), generator=g, device="cuda").to(BF))
        run = lambda ix=ix, x=x, w=w, c=c, s=s, q=q, t=t, xf=xf, wf=wf: (  # noqa: E731
            moe.grouped_matmul(x, w, ix), *moe.grouped_matmul_backward(moe.grouped_matmul(x, w, ix), x, w, ix),
            moe.fp8_matmul(c, s, q, t, ix), moe.grouped_matmul(xf, wf, ix))
        sets.append((run, [v.clone() for v in run()]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        outs = []
        for st, (run, _) in zip(streams, sets):
            with torch.cuda.stream(st):
                outs.append([run() for _ in range(3)])
        torch.cuda.synchronize()
        for got, (_, want) in zip(outs, sets):
            for one in got:
                assert all(torch.equal(a, b) for a, b in zip(one, want))


def test_two_graphs_replayed_in_turns():
    """Two captured products of different sizes that live side by side."""
    a, b = [], []
    for n, (T, E) in enumerate(((40, 5), (900, 3))):
        topk, _ = routing(T, 2, E, n)
        ix = moe.sort_index(topk, E)
        x, w = torch.randn((2 * T, 256), device="cuda").to(BF), torch.randn((E, 256, 320), device="cuda").to(BF)
        want = moe.grouped_matmul(x, w, ix)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = moe.grouped_matmul(x, w, ix)
        a.append((gr, out, want))
        b.append((ix, x, w))
    for _ in range(5):
        for gr, out, want in a:
            out.zero_()
            gr.replay()
            assert torch.equal(out, want)


def test_8bit_experts_decode_what_their_codes_say():
    m = Blocks(T=64, H=256, E=8, F=128, k=2)
    x = torch.randn((5, 256), device="cuda").to(m.dtype)
    codes = m.codes()
    y = m.decode_8bit(x, codes)
    n = moe.add_rms_norm(x, m.p["n2"], torch.zeros_like(x))
    topk, gates = m.route(n["y"], m.p["Wr2"])
    A, B = (tile_values8(*codes[c]) for c in "AB")
    xv = values8(*moe.quantize_rows(n["y"]))
    for t in range(5):
        out = n["h"][t].double()
        slack = 2.0 ** -8 * out.abs()
        for j in range(2):
            e = int(topk[t, j])
            z = (xv[t] @ A[e]).to(BF)
            r = moe.quantize_rows(z.relu().square()[None])
            v = values8(*r)[0]
            # z, rounded to bf16 from sums in another order, may fall a step away, its square two, and
            # the codes of those one step of E4M3; the outputs are bf16 again
            out = out + gates[t, j].double() * (v @ B[e])
            slack = slack + gates[t, j].double() * ((2.0 ** -3 + 2.0 ** -6) * (v.abs() @ B[e].abs()) + 2.0 ** -8 * (v @ B[e]).abs())
        assert bool(((y[t].double() - out).abs() <= slack + 1e-3).all())


def test_many_tokens_decoded_one_by_one_match_the_batch():
    m = Blocks(T=64, H=256, E=8, F=128, k=2, dtype=F32)
    x = torch.randn((9, 256), device="cuda")
    n = moe.add_rms_norm(x, m.p["n2"])["y"]
    topk, gates = m.route(n, m.p["Wr2"])
    ix = moe.sort_index(topk, m.E)
    whole = moe.unsort_rows(moe.grouped_matmul(moe.sort_rows(n, ix), m.p["A"], ix), ix, gates)
    for t in range(9):
        one = moe.sort_index(topk[t:t + 1].clone(), m.E)
        y = moe.unsort_rows(moe.grouped_matmul(moe.sort_rows(n[t:t + 1], one), m.p["A"], one), one, gates[t:t + 1].clone())
        assert torch.equal(y[0], whole[t])               # a row's sum does not depend on its neighbours


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_gradients_without_rows(dtype, layout):
    """An empty batch: zero weight gradients, and nothing else to write."""
    w = torch.randn((3, 64, 40) if layout == "kn" else (3, 40, 64), device="cuda").to(dtype)
    w = w if layout == "kn" else w.transpose(1, 2)
    ix = dict(offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    x, dy = torch.empty((0, 64), dtype=dtype, device="cuda"), torch.empty((0, 40), dtype=dtype, device="cuda")
    dx, dw = moe.grouped_matmul_backward(dy, x, w, ix, dw=torch.full_like(w, float("nan")))
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_one_expert_needs_no_index():
    x, w = torch.randn((77, 136), device="cuda").to(BF), torch.randn((1, 136, 200), device="cuda").to(BF)
    ix = dict(offsets=torch.tensor([0, 77], dtype=torch.int32, device="cuda"))
    assert torch.equal(moe.grouped_matmul(x, w, None), moe.grouped_matmul(x, w, ix))


def test_outputs_and_inputs_at_one_address_are_refused():
    x, w = torch.randn((8, 64), device="cuda"), torch.randn((1, 64, 64), device="cuda")
    with pytest.raises(moe.MoEError):
        moe.grouped_matmul(x, w, None, out=x)
    with pytest.raises(moe.MoEError):
        moe.grouped_matmul(x, w, None, out=w[0][:8])


def test_gradients_written_over_their_inputs_are_refused():
    """drows is written before dw reads the rows, and dw may not be the weights."""
    x, dy, w = (torch.randn(s, device="cuda") for s in ((8, 64), (8, 64), (1, 64, 64)))
    for kw in (dict(drows=x), dict(drows=dy), dict(dw=w)):
        with pytest.raises((moe.MoEError, ValueError)):
            moe.grouped_matmul_backward(dy, x, w, None, **kw)
    both = torch.empty((64, 64), device="cuda")
    with pytest.raises(ValueError):
        moe.grouped_matmul_backward(dy, x, w, None, drows=both[:8], dw=both[None])
    dx, _ = moe.grouped_matmul_backward(dy, x, w, None, want_dw=False, drows=x)   # nothing reads the rows
    assert dx is x


def test_eight_bit_decoding_follows_the_weights():
    m = Blocks(T=64, H=256, E=8, F=128, k=2)
    x = torch.randn((3, 256), device="cuda").to(m.dtype)
    before = m.decode_8bit(x, m.codes())
    m.p["B"].mul_(-1)
    h = moe.add_rms_norm(x, m.p["n2"], torch.zeros_like(x))["h"].float()
    after = m.decode_8bit(x, m.codes())
    # the experts' part changes its sign; each output is rounded once
    slack = 2.0 ** -8 * (before.float().abs() + after.float().abs()) + 1e-6
    assert bool((((before.float() - h) + (after.float() - h)).abs() <= slack).all())
    assert not torch.equal(before, after)
