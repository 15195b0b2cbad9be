"""Helpers of the operator tests: outputs between canary bands, rounding
units, and buffers with padded row strides."""
import torch

CANARY = 0x5A
GUARD = 1024

#: half a step of rounding to a type, relative to the value
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U32 = 2.0 ** -24


class Banded:
    """A rows x H view with row stride ld inside an allocation whose other
    bytes (bands before and after, gaps between rows) hold a canary; the view
    itself starts as NaN."""

    def __init__(self, rows, H, dtype, ld=None):
        self.rows, self.H, self.ld = rows, H, ld or H
        size = torch.finfo(dtype).bits // 8 if dtype.is_floating_point else torch.iinfo(dtype).bits // 8
        n = (max(rows - 1, 0) * self.ld + (H if rows else 0)) * size
        pad = -n % 16
        self.raw = torch.full((GUARD + n + pad + GUARD,), CANARY, dtype=torch.uint8, device="cuda")
        flat = self.raw[GUARD:GUARD + n].view(dtype)
        self.t = flat.as_strided((rows, H), (self.ld, 1), flat.storage_offset())
        if dtype.is_floating_point:
            self.t.fill_(float("nan"))
        self.dtype = dtype

    def intact(self):
        """Whether every byte outside the view still holds the canary."""
        keep = self.raw.clone()
        n = keep.numel() - 2 * GUARD
        inner = keep[GUARD:GUARD + n]
        size = self.t.element_size()
        for_view = inner[:(n // size) * size].view(self.dtype)
        v = for_view.as_strided((self.rows, self.H), (self.ld, 1), for_view.storage_offset())
        mark = torch.full((size,), CANARY, dtype=torch.uint8, device="cuda").view(self.dtype)[0]
        v.copy_(mark.expand_as(v))
        return bool((keep == CANARY).all())


def strided(t, ld):
    """The same matrix with row stride ld."""
    b = torch.zeros((t.shape[0], ld), dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


def assert_within(got, ref, bound, what=""):
    """|got - ref| <= bound elementwise, in 64 bits; reports the worst ratio."""
    d = (got.double() - ref).abs()
    bad = ~(d <= bound)
    if bool(bad.any()):
        i = int((d / bound.clamp_min(1e-300)).nan_to_num(float("inf")).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off; worst at {i}: "
                             f"{got.flatten()[i].item()} for {ref.flatten()[i].item()}, bound {bound.flatten()[i].item()}")
