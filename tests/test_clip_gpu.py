"""moe_clip_grad_norm against 64-bit sums.

A thread adds at most 256 squares in fp32 before going on in 64 bits, so the
norm is off by at most half of 256 + 4 roundings; a clipped value by that, the
coefficient's and the product's rounding and half a step of its type."""
import math

import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import U32, UNIT, assert_within

pytestmark = pytest.mark.gpu

REL = (256 / 2 + 4) * U32
DTYPES = [torch.float32, torch.bfloat16]


def make(sizes, seed=0, std=1.0, offset=0):
    """Tensors as views of one flat buffer, `offset` values apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, (n, dt) in enumerate(sizes):
        flat = torch.randn(n + offset + 8, generator=g, device="cuda").mul_(std * (1 + i % 3)).to(dt)
        out.append(flat[offset:offset + n])
    return out


def exact_norm(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads if g.numel()))


def check(grads, max_norm, outs, norm):
    ref = exact_norm(grads)
    assert abs(float(norm) - ref) <= ref * (REL + U32)
    c = min(1.0, max_norm / ref) if ref > 0 else 1.0
    for g, o in zip(grads, outs):
        r = g.double() * c
        if c == 1.0:
            assert torch.equal(o, g)
        else:
            assert_within(o, r, r.abs() * (UNIT[g.dtype] + (REL + 3 * U32)) + 1e-37, "out")


SETS = {
    "one_value": [(1, torch.float32)],
    "small": [(1, torch.bfloat16), (3, torch.float32), (255, torch.bfloat16), (0, torch.float32), (1000, torch.float32)],
    "chunk_edges": [(n, dt) for dt in DTYPES for n in (16383, 16384, 16385, 32767, 32768, 32769, 100001)],
    "many": [(17 * i + 1, DTYPES[i % 2]) for i in range(1500)],
    "large": [(3000001, torch.bfloat16), (5, torch.float32), (2500000, torch.float32), (20000000, torch.bfloat16)],
}


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("clipped", [True, False])
@pytest.mark.parametrize("name", list(SETS))
def test_norm_and_clip(name, clipped, offset):
    grads = make(SETS[name], offset=offset)
    max_norm = exact_norm(grads) * (0.25 if clipped else 4.0)
    keep = [g.clone() for g in grads]
    outs = [torch.full((g.numel() + 16,), 7.0, dtype=g.dtype, device="cuda") for g in grads]
    views = [o[8:8 + g.numel()] for o, g in zip(outs, grads)]
    norm = moe.clip_grad_norm(grads, max_norm, views)
    check(grads, max_norm, views, norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    assert all(bool((o[:8] == 7).all()) and bool((o[8 + g.numel():] == 7).all()) for o, g in zip(outs, grads))
    # a destination of another alignment, in place, and the norm alone
    shifted = [o[3:3 + g.numel()] for o, g in zip(outs, grads)]
    n2 = moe.clip_grad_norm(grads, max_norm, shifted)
    assert torch.equal(n2, norm)
    check(grads, max_norm, shifted, n2)
    assert torch.equal(moe.clip_grad_norm(grads, max_norm, clip=False), norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    n3 = moe.clip_grad_norm(grads, max_norm)
    assert torch.equal(n3, norm)
    check(keep, max_norm, grads, n3)


@pytest.mark.parametrize("std", [1e-30, 1e-20, 1e-12, 1e12, 1e18])
@pytest.mark.parametrize("dtype", DTYPES)
def test_ranges_whose_squares_leave_fp32(dtype, std):
    grads = make([(50001, dtype), (70, dtype)], seed=3, std=std)
    n = exact_norm(grads)
    outs = [torch.empty_like(g) for g in grads]
    check(grads, n / 3, outs, moe.clip_grad_norm(grads, n / 3, outs))


def test_one_large_value_among_tiny_ones():
    g = make([(40000, torch.float32)], std=1e-22)[0]
    g[12345] = 2e19
    out = torch.empty_like(g)
    check([g], 1.0, [out], moe.clip_grad_norm([g], 1.0, [out]))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_the_values(bad):
    grads = make([(5000, torch.float32), (700, torch.bfloat16)])
    grads[1][33] = bad
    keep = [g.clone() for g in grads]
    outs = [torch.empty_like(g) for g in grads]
    norm = moe.clip_grad_norm(grads, 0.5, outs)
    assert not math.isfinite(float(norm)) and math.isnan(float(norm)) == math.isnan(bad)
    for o, k in zip(outs, keep):
        assert torch.equal(o.view(torch.uint8), k.view(torch.uint8))


def test_zeros_and_infinite_limit():
    grads = [torch.zeros(1000, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(moe.clip_grad_norm(grads, 1.0)) == 0.0 and bool((grads[0] == 0).all())
    grads = make([(5000, torch.float32)])
    keep = grads[0].clone()
    assert abs(float(moe.clip_grad_norm(grads, float("inf"))) - exact_norm([keep])) <= exact_norm([keep]) * (REL + U32)
    assert torch.equal(grads[0], keep)
    assert float(moe.clip_grad_norm([torch.empty(0, device="cuda")], 1.0)) == 0.0


def test_repeatable_side_stream_and_graph():
    sizes = [(100003, torch.bfloat16), (777, torch.float32)]
    grads, other = make(sizes), make(sizes, seed=9)
    first = moe.clip_grad_norm([g.clone() for g in grads], 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [torch.empty_like(g) for g in grads]
        again = moe.clip_grad_norm(grads, 1.0, outs)
    side.synchronize()
    assert torch.equal(again, first)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        norm = moe.clip_grad_norm(grads, 1.0, outs)
    for g, o in zip(grads, other):
        g.copy_(o)
    gr.replay()
    torch.cuda.synchronize()
    check(other, 1.0, outs, norm)


def test_a_tensor_of_more_than_32_bits():
    """More than 2^31 values and 2^32 bytes in one tensor."""
    n = (1 << 31) + 12345
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.randn(n, device="cuda", dtype=torch.bfloat16)
    out = torch.empty_like(g)
    norm = moe.clip_grad_norm([g], 100.0, [out])
    ref = math.sqrt(math.fsum(float(p.double().square().sum()) for p in g.split(1 << 28)))
    assert abs(float(norm) - ref) <= ref * (REL + U32)
    for s in (slice(0, 70000), slice(1 << 30, (1 << 30) + 70000), slice(n - 70000, n)):
        r = g[s].double() * (100.0 / ref)
        assert_within(out[s], r, r.abs() * (UNIT[torch.bfloat16] + REL + 3 * U32) + 1e-37, "out")
