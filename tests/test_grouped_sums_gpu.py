"""fp32 products over long contractions: sums of many terms, with a bound that does not grow
as their number does."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import U32, assert_within

pytestmark = pytest.mark.gpu


def piecewise(n, mags):
    """fp32 sums of at most 256 products in a row, and the sum of those: each addition is off
    by half a step of at most the sum of the magnitudes (a term goes through 256 + n / 256)."""
    return (256 + n / 256 + 4) * U32 * mags


@pytest.mark.parametrize("rows", [1, 40, 9000])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_fp32_rows_over_a_long_contraction(rows, layout):
    """One term of 1 and 8191 of 2^-25, which one running sum loses one by one."""
    K, N = 8192, 1100 if rows == 9000 else 70
    x = torch.full((rows, K), 2.0 ** -25, device="cuda")
    x[:, 0] = 1
    w = torch.ones((1, K, N) if layout == "kn" else (1, N, K), device="cuda")
    w = w if layout == "kn" else w.transpose(1, 2)
    y = moe.grouped_matmul(x, w, None)
    want = torch.full((), 1 + 8191 * 2.0 ** -25, dtype=torch.float64, device="cuda")
    assert_within(y, want.expand_as(y), piecewise(K, want).expand_as(y))


@pytest.mark.parametrize("M,N,E", [(64, 96, 1), (1200, 1200, 8)])
def test_fp32_weight_gradient_over_many_rows(M, N, E):
    R = 30000
    ix = dict(offsets=torch.arange(E + 1, dtype=torch.int32, device="cuda") * R)
    x, dy = torch.full((E * R, M), 2.0 ** -25, device="cuda"), torch.ones((E * R, N), device="cuda")
    x[::R] = 1
    w = torch.empty((E, M, N), device="cuda")
    _, dw = moe.grouped_matmul_backward(dy, x, w, ix, want_drows=False)
    want = torch.full((), 1 + (R - 1) * 2.0 ** -25, dtype=torch.float64, device="cuda")
    assert_within(dw, want.expand_as(dw), piecewise(R, want).expand_as(dw))


@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("K", [255, 256, 257, 511, 512, 513, 8192, 8199])
def test_fp32_rows_of_random_values(K, rows):
    """Lengths at the pieces' borders, aligned and odd."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x, w = torch.randn((rows, K), generator=g, device="cuda"), torch.randn((1, K, 96), generator=g, device="cuda")
    y = moe.grouped_matmul(x, w, None)
    ref, mags = x.double() @ w[0].double(), x.double().abs() @ w[0].double().abs()
    assert_within(y, ref, piecewise(K, mags) + U32 * ref.abs())


@pytest.mark.parametrize("R", [256, 300, 513, 30000])
def test_fp32_weight_gradients_of_random_values(R):
    g = torch.Generator(device="cuda").manual_seed(R)
    x, dy = torch.randn((R, 65), generator=g, device="cuda"), torch.randn((R, 72), generator=g, device="cuda")
    _, dw = moe.grouped_matmul_backward(dy, x, torch.empty((1, 65, 72), device="cuda"), None, want_drows=False)
    ref, mags = x.double().T @ dy.double(), x.double().abs().T @ dy.double().abs()
    assert_within(dw[0], ref, piecewise(R, mags) + U32 * ref.abs())
