"""Rows moved by the routing tables of a plan with a capacity: the tables name a
row for every slot, and with the slots past the capacity marked as moe_sorted_t
says, own experts give what the layer gives."""
import math

import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cf", [0.5, 0.9, 4.0])
def test_own_experts_follow_the_layers_drops(cf):
    T, H, E, F, k = 200, 128, 6, 128, 2
    g = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std  # noqa: E731
    x, Wr = r(T, H), r(H, E, std=0.2)
    Wg, Wu, Wd = r(E, H, F, std=H ** -0.5), r(E, H, F, std=H ** -0.5), r(E, F, H, std=F ** -0.5)
    layer = moe.MoELayer(H, E, F, k, T, score=moe.MOE_SCORE_SIGMOID, dtype=moe.MOE_FP32, capacity_factor=cf)
    y, t = layer.forward(x, Wr, None, Wg, Wu, Wd, routing=True)
    row_of, offsets, expert = t["row_of"], t["offsets"], t["topk_idx"].long()
    rows = int(offsets[-1])
    # every slot has a row of its own
    assert bool((row_of >= 0).all()) and row_of.unique().numel() == T * k
    C = math.ceil(cf * T * k / E)
    place = row_of - offsets[expert]
    kept = torch.where(place < C, row_of, torch.full_like(row_of, -1))
    dropped = int((kept < 0).sum())
    assert dropped == int((t["counts"] - C).clamp_min(0).sum()) and (dropped > 0) == (cf < 1)

    def by(table):
        index = {"row_of": table}
        X = moe.sort_rows(x, index, out=torch.zeros((rows, H), device="cuda")).double()
        Y = torch.zeros((rows, H), dtype=torch.float64, device="cuda")
        for e in range(E):
            s = slice(int(offsets[e]), int(offsets[e + 1]))
            Y[s] = (torch.nn.functional.silu(X[s] @ Wg[e].double()) * (X[s] @ Wu[e].double())) @ Wd[e].double()
        return moe.unsort_rows(Y.float(), index, t["gates"])

    rel = lambda a: float((a - y).norm() / y.norm())  # noqa: E731
    # fp32 products of 128 terms in the layer: 128 roundings of 2^-24 at most, three products deep
    assert rel(by(kept)) < 3 * 128 * 2.0 ** -24
    assert rel(by(row_of)) > 0.05 or not dropped
