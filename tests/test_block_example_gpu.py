"""The operators together, as examples/block_step.py uses them: the gradients
of two blocks against autograd of the same computation in 64 bits, a training
run, and one decoded token."""
import os
import sys

import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from block_step import Blocks  # noqa: E402

pytestmark = pytest.mark.gpu


def reference(m, x, topk1, topk2):
    """The blocks in float64 torch with the given routing."""
    p = {n: v.double().requires_grad_() for n, v in m.p.items()}
    x = x.double().requires_grad_()
    norm = lambda v, w: v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731

    def mix(y, Wr, topk, expert):
        s = torch.sigmoid((y @ Wr).gather(1, topk))
        g = s / s.sum(1, keepdim=True)
        out = torch.zeros_like(y)
        for e in range(m.E):
            w = (g * (topk == e)).sum(1, keepdim=True)
            out = out + w * expert(y, e)
        return out

    y1 = norm(x, p["n1"])
    m1 = mix(y1, p["Wr1"], topk1, lambda y, e: (torch.nn.functional.silu(y @ p["Wg"][e]) * (y @ p["Wu"][e])) @ p["Wd"][e])
    h2 = x + m1
    y2 = norm(h2, p["n2"])
    out = h2 + mix(y2, p["Wr2"], topk2, lambda y, e: (y @ p["A"][e]).relu().square() @ p["B"][e])
    return x, p, out


def test_gradients_of_two_blocks_match_autograd():
    m = Blocks(T=200, H=128, E=6, F=128, k=3, align=8, dtype=torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dout = (torch.randn((m.T, m.H), generator=g, device="cuda") for _ in range(2))
    out, s = m.forward(x)
    _, r1 = m.layer.forward(s["y1"], m.p["Wr1"], None, m.p["Wg"], m.p["Wu"], m.p["Wd"], routing=True)
    dx, d = m.backward(dout, s)
    rx, p, ref = reference(m, x, r1["topk_idx"].long(), s["topk"].long())
    ref.backward(dout.double())
    # fp32 matrix products (torch's and the layer's) of length 128 in a row of eight: relative L2 far below 1e-4
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, ref.detach()) < 1e-4
    assert rel(dx, rx.grad) < 1e-4
    for n in m.p:
        assert rel(d[n], p[n].grad) < 1e-4, n


def test_training_lowers_the_loss_and_clips():
    m = Blocks(T=300, H=256, E=8, F=128, k=2)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, t = (torch.randn((m.T, m.H), generator=g, device="cuda").to(m.dtype) for _ in range(2))
    m.max_norm = 1e-2
    losses = []
    for _ in range(8):
        before = {n: v.clone() for n, v in m.p.items()}
        loss, norm = m.step(x, t, lr=4.0)
        losses.append(float(loss))
        assert float(norm) > m.max_norm
        # fp32 parameters move by lr times a part of a clipped gradient
        moved = sum(float((m.p[n] - before[n]).double().square().sum()) for n in ("n1", "n2", "Wr1", "Wr2")) ** 0.5
        assert moved <= 4.0 * m.max_norm * 1.01
    assert losses[-1] < losses[0]


def test_one_token_is_decoded():
    m = Blocks(T=64, H=256, E=8, F=128, k=2)
    x = torch.randn((1, 256), device="cuda").to(m.dtype)
    y, codes, scales = m.decode(x)
    assert y.shape == x.shape and bool(y.isfinite().all())
    assert codes.shape == (1, 256) and scales.numel() == 2 * 512
    codes2, scales2 = torch.empty((128, 256), dtype=torch.uint8, device="cuda"), torch.empty(1024, dtype=torch.uint8, device="cuda")
    n = moe.add_rms_norm(x, m.p["n2"], torch.zeros_like(x))["y"]
    pad = torch.cat([n, torch.zeros((127, 256), dtype=m.dtype, device="cuda")])
    moe.moe_mx_quantize(128, 256, pad.data_ptr(), codes2.data_ptr(), scales2.data_ptr(), None, None, 0,
                        torch.cuda.current_stream().cuda_stream)
    # the layer's quantiser reads the norm after its rounding to bf16: the same scales but for block
    # maxima next to 448 2^e, and codes within a step
    at = torch.arange(1024, device="cuda").view(2, 32, 4, 4)[:, 0, 0]
    assert bool(((scales[at].int() - scales2[at].int()).abs() <= 1).all())
