"""Blockwise codes of the norm are those of a division, whatever the scale.

tests/e4m3_quotient_fp32_check.c walks every pair of fp32 value and scale at
which the kernel's corrected product could give another code than the fp32
quotient, from the smallest scale that the kernel uses it for (norm.cu's
kQuotientMin); on the GPU such pairs, from the smallest scales to the largest,
go through the norm itself."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mixture_experts_layer_sigmoid_gb300", "csrc")


def test_corrected_product_gives_the_divisions_codes(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = open(os.path.join(CSRC, "norm.cu")).read()
    border = re.search(r"constexpr float kQuotientMin = 0x1p(-\d+)f", src)
    assert border, "norm.cu: kQuotientMin"
    exe = str(tmp_path / "check")
    subprocess.run([cc, "-O2", "-ffp-contract=off", "-o", exe, os.path.join(HERE, "e4m3_quotient_fp32_check.c"), "-lm"],
                   check=True)
    r = subprocess.run([exe, border.group(1)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "E4M3 differences 0" in r.stdout, r.stdout


def beside_ties():
    """Pairs (value, scale) of significands whose quotient lies next to a tie of
    two codes: V 2^j - S N = d for small d, N the half steps beside the tie."""
    out = []
    for odd in range(1, 32, 2):
        tie = odd << (24 - odd.bit_length())
        for N in [2 * tie + 1, 2 * tie - 1] + ([4 * tie - 1] if odd == 1 else []):
            for j in (23, 24, 25, 26):
                inv = pow(N, -1, 1 << j)
                for d in [*range(-32, 0), *range(1, 33)]:
                    S = -d * inv % (1 << j)
                    V = (S * N + d) >> j
                    if 1 << 23 <= S < 1 << 24 and 1 << 23 <= V < 1 << 24:
                        out.append((V, S))
    return out


def maximum_of(s):
    """fp32 maxima with RN(maximum / 448) = s, or 0 where no maximum gives it."""
    a = s * np.float32(448)
    for c in (a, np.nextafter(a, np.float32(0)), np.nextafter(a, np.float32(np.inf))):
        a = np.where(c / np.float32(448) == s, c, a)
    return np.where(a / np.float32(448) == s, a, np.float32(0))


def blocks_beside_ties(low, high):
    """128-value blocks: one value per block sets the scale, the others lie
    next to ties of that scale. Scales in [2^low, 2^high)."""
    pairs = beside_ties()
    V, S = (np.array([p[i] for p in pairs], dtype=np.float64) for i in (0, 1))
    rows = []
    for b in range(low, high):
        s = np.ldexp(S, b - 23).astype(np.float32)
        top = maximum_of(s)
        blk = np.zeros((len(s), 128), dtype=np.float32)
        for i, q in enumerate(range(-12, 9)):
            v = np.ldexp(V, b - 23 + q).astype(np.float32)
            blk[:, 1 + i] = np.where(v <= top, v, 0)
            blk[:, 40 + i] = -blk[:, 1 + i]
        blk[:, 0] = top
        rows.append(blk[top > 0])
    return np.concatenate(rows)


def division_codes(blocks):
    """E4M3 codes of the fp32 quotients, nearest even, by torch's conversion."""
    amax = np.abs(blocks).max(1, keepdims=True)
    s = (amax / np.float32(448)).astype(np.float32)
    q = np.clip(blocks / s, -448, 448).astype(np.float32)
    return s[:, 0], torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("low,high", [(-125, -110), (-111, -92), (-93, -80), (-10, 10), (90, 110)])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_beside_ties(low, high, residual):
    """Rows of ones with eps = 0 are their own norm, so y is the weight itself."""
    blocks = blocks_beside_ties(low, high)
    want_s, want = division_codes(blocks)
    per = 64                                              # blocks of a row
    for at in range(0, len(blocks), per):
        w = blocks[at:at + per]
        H = w.size
        x = torch.ones((3, H), device="cuda")
        r = torch.zeros_like(x) if residual else None
        out = moe.add_rms_norm(x, torch.from_numpy(w.reshape(-1)).cuda(), r, eps=0.0, quant=moe.MOE_NORM_FP8_BLOCK)
        assert torch.equal(out["y"][1].cpu(), torch.from_numpy(w.reshape(-1)))
        for row in (0, 2):
            assert np.array_equal(out["scales"][row].cpu().numpy(), want_s[at:at + per])
            assert torch.equal(out["codes"][row].cpu().view(-1, 128), want[at:at + per])
