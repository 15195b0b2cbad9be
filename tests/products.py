"""Helpers of the tests of the products over sorted rows: segments of chosen
lengths, the products in 64 bits, and the bounds they are held to."""
import torch

from opcheck import UNIT

#: one ulp of an fp32 value, the most an addition that truncates is off by
ULP32 = 2.0 ** -23


def segments(lengths, align=1, behind=0, counts=True, device="cuda"):
    """An index of segments of these lengths, each padded to a multiple of
    ``align``, with ``behind`` rows after the last: (index, rows, [(first, rows)])."""
    offsets, at, seg = [0], 0, []
    for n in lengths:
        seg.append((at, n))
        at += -(-n // align) * align
        offsets.append(at)
    ix = dict(offsets=torch.tensor(offsets, dtype=torch.int32, device=device))
    if counts:
        ix["counts"] = torch.tensor(lengths, dtype=torch.int32, device=device)
    return ix, at + behind, seg


def used_mask(rows, seg, device="cuda"):
    m = torch.zeros(rows, dtype=torch.bool, device=device)
    for o, n in seg:
        m[o:o + n] = True
    return m


def product64(x, w, seg):
    """(Y, sum of the terms' magnitudes) of rows times their expert's weights; zeros elsewhere."""
    y = torch.zeros((x.shape[0], w.shape[2]), dtype=torch.float64, device=x.device)
    a = torch.zeros_like(y)
    for e, (o, n) in enumerate(seg):
        xe, we = x[o:o + n].double(), w[e].double()
        y[o:o + n] = xe @ we
        a[o:o + n] = xe.abs() @ we.abs()
    return y, a


def wgrad64(x, dy, seg):
    d = torch.zeros((len(seg), x.shape[1], dy.shape[1]), dtype=torch.float64, device=x.device)
    a = torch.zeros_like(d)
    for e, (o, n) in enumerate(seg):
        xe, ye = x[o:o + n].double(), dy[o:o + n].double()
        d[e] = xe.T @ ye
        a[e] = xe.abs().T @ ye.abs()
    return d, a


def bound(ref, mags, terms, dtype):
    """Rounding to the output's type, and a sum of ``terms`` fp32 products: each of the
    additions (and for fp32 values each product) is off by an ulp of at most the sum
    of the magnitudes."""
    return UNIT[dtype] * ref.abs() + (terms + 4) * ULP32 * (mags + UNIT[dtype] * mags) + 1e-40


def values8(codes, scales):
    """64-bit values of codes with 1x128 blocks."""
    v = codes.view(torch.float8_e4m3fn).double()
    return v * scales.double().repeat_interleave(128, -1)


def tile_values8(codes, scales):
    """64-bit values of E x K x N codes with 128x128 tiles (either layout)."""
    K, N = codes.shape[-2:]
    s = scales.double().repeat_interleave(128, -2)[..., :K, :].repeat_interleave(128, -1)[..., :N]
    return codes.contiguous().view(torch.float8_e4m3fn).double() * s
