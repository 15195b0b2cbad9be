"""A dense weight gradient from 8-bit codes: X's codes along the tokens (moe_fp8_quantize with
MOE_Q_COLS_T, one scale for 128 tokens of a column) times dY's tile codes, tokens a multiple of 128."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import assert_within
from products import bound, tile_values8, values8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N", [(128, 128, 128), (640, 256, 384), (4096, 512, 1024)])
def test_codes_along_the_tokens(T, K, N):
    g = torch.Generator(device="cuda").manual_seed(T)
    x, dy = (torch.randn((T, n), generator=g, device="cuda").to(torch.bfloat16) for n in (K, N))
    ct, st = torch.empty((K, T), dtype=torch.uint8, device="cuda"), torch.empty((K, T // 128), device="cuda")
    moe.moe_fp8_quantize(T, K, moe.MOE_Q_COLS_T, x.data_ptr(), None, None, ct.data_ptr(), st.data_ptr(),
                         torch.cuda.current_stream().cuda_stream)
    c, s = moe.quantize_tiles(dy)
    dw = moe.fp8_matmul(ct, st, c, s, dtype=torch.float32)
    a, b = values8(ct, st), tile_values8(c, s)
    assert_within(dw, a @ b, bound(a @ b, a.abs() @ b.abs(), T + 2, torch.float32))
    # and the codes are those of the values: half a step of E4M3 each, or of its smallest one
    full, mags = x.double().T @ dy.double(), x.double().abs().T @ dy.double().abs()
    small = 2.0 ** -10 * (st.double().amax() * dy.double().abs().sum(0) + s.double().amax() * x.double().abs().sum(0)[:, None])
    assert_within(dw, full, (2 * 2.0 ** -4 + 2.0 ** -8) * mags + small + 1e-3)
