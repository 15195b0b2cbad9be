"""The norm at sizes between those of test_norm_gpu.py: 8-bit output and plain rows
for each number of rows and width that takes another number of pieces per thread.
Bounds as there; the 8-bit codes are also those of a division, bit for bit."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import UNIT, assert_within
from test_norm_gpu import EPS, check_backward, e4m3_error, inputs, reference, rel32

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
# rows off the 128-row tile: up to 152 rows, up to 1215, and more; every limit of the width from both sides
EIGHT_BIT = [(1300, 640), (1217, 1920), (1217, 2048), (1250, 4096), (1217, 3968), (1217, 2176), (1217, 4224), (200, 128), (1217, 384),
             (200, 640), (200, 1152), (200, 1536), (200, 2176), (200, 4096), (200, 4224), (200, 7168), (200, 8192), (153, 8320),
             (200, 16384), (152, 7168), (152, 1024), (160, 16512), (300, 30080)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("quant", [moe.MOE_NORM_FP8_BLOCK, moe.MOE_NORM_MXFP8])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,H", EIGHT_BIT)
def test_eight_bit_output(rows, H, residual, quant, dtype):
    i = inputs(rows, H, dtype)
    i["x"][1] = 0
    i["r"][1] = 0
    i["w"][32:64] = 0
    r = i["r"] if residual else None
    out = moe.add_rms_norm(i["x"], i["w"], r, eps=EPS, quant=quant, want_y=False)
    both = moe.add_rms_norm(i["x"], i["w"], r, eps=EPS, quant=quant, want_rstd=True)
    assert torch.equal(out["codes"], both["codes"]) and torch.equal(out["scales"], both["scales"])
    s, rstd, y = reference(i["x"], r, i["w"])
    rel = rel32(H)
    assert_within(both["rstd"], rstd, rstd * rel, "rstd")
    assert_within(both["y"], y, y.abs() * (UNIT[dtype] + rel) + 1e-37, "y")
    codes = out["codes"].view(torch.float8_e4m3fn)
    if quant == moe.MOE_NORM_FP8_BLOCK:
        amax = y.abs().view(rows, H // 128, 128).amax(2)
        ref = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        assert_within(out["scales"], ref, ref * (rel + 2.0 ** -24), "scales")
        sc = out["scales"].repeat_interleave(128, 1)
    else:
        e = out["scales"].view(-1, H // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, H // 32).int()
        assert bool((e[rows:] == 0).all())
        e = e[:rows] - 127
        amax = y.abs().view(rows, H // 32, 32).amax(2)
        up = lambda a: torch.where(a > 0, torch.ceil(torch.log2(a / 448)).clamp(-127, 127), torch.full_like(a, -127.0))  # noqa: E731
        assert bool(((e >= up(amax * (1 - rel))) & (e <= up(amax * (1 + rel)))).all())
        sc = torch.ldexp(torch.ones_like(amax, dtype=torch.float32), e).repeat_interleave(32, 1)
    q = y / sc.double()
    assert_within(codes.double(), q, e4m3_error(q) + q.abs() * 2 * (rel + 2.0 ** -23), "codes")
    if dtype == torch.float32:
        # y is the norm that the codes were taken from: its fp32 quotient, nearest even
        want = (both["y"] / sc).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(out["codes"], want.view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,H", [(400, 1536), (400, 2048), (400, 8192), (160, 8200), (200, 513), (200, 1030), (200, 3001), (200, 6001),
                                    (153, 16000), (153, 15999), (1300, 520), (1300, 300)])
def test_plain_rows_and_gradient(rows, H, dtype):
    i = inputs(rows, H, dtype)
    for r in (None, i["r"]):
        out = moe.add_rms_norm(i["x"], i["w"], r, eps=EPS, want_rstd=True)
        s, rstd, y = reference(i["x"], r, i["w"])
        assert_within(out["rstd"], rstd, rstd * rel32(H), "rstd")
        assert_within(out["y"], y, y.abs() * (UNIT[dtype] + rel32(H)) + 1e-37, "y")
    dx, dw = moe.add_rms_norm_backward(i["dy"], out["h"], out["rstd"], i["w"], i["dh"])
    check_backward(dx, dw, i["dy"], out["h"], out["rstd"], i["w"], i["dh"])


def test_codes_of_many_rows_are_a_divisions():
    """Whole training-size outputs against the division, by both kernels that take few and many rows."""
    i = inputs(4097, 4096, torch.float32)
    out = moe.add_rms_norm(i["x"], i["w"], eps=EPS, quant=moe.MOE_NORM_FP8_BLOCK)
    sc = out["scales"].repeat_interleave(128, 1)
    want = (out["y"] / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(out["codes"], want)
    amax = out["y"].abs().view(4097, 32, 128).amax(2)
    assert np.array_equal(out["scales"].cpu().numpy(), amax.cpu().numpy() / np.float32(448))
