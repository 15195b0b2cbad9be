"""The codes of the decoded token in examples/block_step.py: each set of codes
times its own scales against the norm in 64 bits."""
import os
import sys

import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from opcheck import UNIT
from test_norm_gpu import e4m3_error, reference, rel32

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from block_step import Blocks  # noqa: E402

pytestmark = pytest.mark.gpu


def scales_of(atoms, H):
    """Scales of row 0 of the first tile, one per value."""
    e = atoms.view(-1, H // 128, 32, 4, 4)[0, :, 0, 0].reshape(-1).int() - 127
    return torch.ldexp(torch.ones(H // 32, dtype=torch.float64, device="cuda"), e).repeat_interleave(32)


def test_decoded_tokens_codes():
    m = Blocks(T=64, H=256, E=8, F=128, k=2)
    for seed in range(20):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn((1, 256), generator=g, device="cuda").to(m.dtype)
        _, codes, scales = m.decode(x)
        y = reference(x, None, m.p["n2"])[2][0]
        sc = scales_of(scales, 256)
        got = codes[0].view(torch.float8_e4m3fn).double()
        q = y / sc
        assert bool(((got - q).abs() <= e4m3_error(q) + q.abs() * 2 * rel32(256)).all())
        # the layer's quantiser takes the norm after its rounding to bf16: half a step of that more
        rows = torch.zeros((128, 256), dtype=m.dtype, device="cuda")
        rows[:1] = moe.add_rms_norm(x, m.p["n2"], torch.zeros_like(x))["y"]
        codes2 = torch.empty((128, 256), dtype=torch.uint8, device="cuda")
        scales2 = torch.empty(1024, dtype=torch.uint8, device="cuda")
        moe.moe_mx_quantize(128, 256, rows.data_ptr(), codes2.data_ptr(), scales2.data_ptr(), None, None, 0,
                            torch.cuda.current_stream().cuda_stream)
        sc2 = scales_of(scales2, 256)
        got2 = codes2[0].view(torch.float8_e4m3fn).double()
        q2 = y / sc2
        assert bool(((got2 - q2).abs() <= e4m3_error(q2) + q2.abs() * 2 * (UNIT[m.dtype] + rel32(256))).all())
        # at the same scale the two differ by one step at most
        same = sc == sc2
        assert int(same.sum()) > 128
        a, b = codes[0][same].int(), codes2[0][same].int()
        assert bool(((a - b).abs() <= 1).all())
