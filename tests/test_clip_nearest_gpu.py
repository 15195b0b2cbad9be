"""The norm of moe_clip_grad_norm is the fp32 value nearest to the exact one, and
its coefficient the one nearest to max_norm / norm.

Squares of fp32 values are exact in 64 bits and math.fsum rounds their sum once,
so the reference norm is off by 2^-53 of itself. The call's sum is off by some
2^-46 of it for few values and by less than 2^-35 for whole chunks: only a norm that
close to the middle of two fp32 numbers could come out as the other one, less than one
in 2^10 sets; the sets here are fixed. A clipped value
is the fp32 product with the coefficient, rounded once more to its type."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
SIZES = [1, 2, 3, 7, 8, 33, 100, 1000, 5001, 16384, 70001, 300007]


def exact(grads):
    return math.sqrt(math.fsum(v for g in grads for v in g.cpu().double().square().tolist()))


def check(grads, share):
    """Clips to `share` of the norm (not in place) and compares every bit."""
    n = exact(grads)
    max_norm = np.float32(n * share) if n else np.float32(1)     # values too small for their type are zeros
    outs = [torch.full_like(g, 7.0) for g in grads]
    norm = moe.clip_grad_norm(grads, float(max_norm), outs)
    wrong = float(norm) != float(np.float32(n))
    f = np.float32(min(1.0, float(max_norm) / n) if n else 1)
    for g, o in zip(grads, outs):
        want = (g.float() * torch.tensor(f, device="cuda")).to(g.dtype) if f < 1 else g
        wrong = wrong or not torch.equal(o, want)
    alone = moe.clip_grad_norm(grads, 1.0, clip=False)
    assert torch.equal(alone, norm)
    return wrong


def tensor(n, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda", dtype=torch.float64) * std).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", SIZES)
def test_nearest(n, dtype):
    seeds = range(40 if n < 10000 else 12)
    wrong = [s for s in seeds if check([tensor(n, dtype, 100 * n + s, std=0.02)], 0.3)]
    assert not wrong, f"{len(wrong)} of {len(seeds)} sets"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("std", [1e-42, 1e-38, 1e-30, 1e-20, 1e-12, 1e-10, 1e12, 1e18, 1e30])
def test_nearest_at_any_size_of_the_values(std, dtype):
    wrong = [s for s in range(12) if check([tensor(3001 + s, dtype, 7 * s, std=std)], 0.4)]
    assert not wrong, f"{len(wrong)} of 12 sets"


def test_nearest_over_many_tensors():
    """Two batches of the table, both types, values of very different sizes."""
    for seed in range(4):
        grads = [tensor(37 + i % 50, DTYPES[i % 2], 1000 * seed + i, std=10.0 ** (i % 7 - 3)) for i in range(1000)]
        assert not check(grads, 0.5)


def test_a_limit_next_to_the_norm():
    """Limits one step around the norm: the coefficient is 1 or the number below it."""
    for seed in range(8):
        g = tensor(1234, torch.float32, seed)
        n = np.float32(exact([g]))
        for m in (np.nextafter(n, np.float32(0)), n, np.nextafter(n, np.float32(np.inf))):
            out = torch.empty_like(g)
            moe.clip_grad_norm([g], float(m), [out])
            f = np.float32(min(1.0, float(m) / exact([g])))
            assert torch.equal(out, g * torch.tensor(f, device="cuda"))
