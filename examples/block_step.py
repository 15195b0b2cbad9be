"""Two pre-norm expert blocks, trained for a few steps, then one token decoded.

Block 1 has this library's expert layer (MoELayer); block 2 has experts of its
own (here squared-ReLU FFNs), which the library's routing, token sort and grouped
products serve:

    h1, y1 = add_rms_norm(x)            m1  = MoELayer(y1)
    h2, y2 = add_rms_norm(m1, h1)       out = h2 + sum_j g_j expert_j(y2)

with the backward of each part, and every gradient clipped by the global norm
before the update.

    python examples/block_step.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixture_experts_layer_sigmoid_gb300 as moe  # noqa: E402


class Blocks:
    def __init__(self, T=512, H=256, E=8, F=256, k=2, align=16, dtype=torch.bfloat16, seed=0, max_norm=1.0):
        self.T, self.H, self.E, self.F, self.k, self.align, self.max_norm = T, H, E, F, k, align, max_norm
        self.dtype = dtype
        self.layer = moe.MoELayer(H, E, F, k, T, score=moe.MOE_SCORE_SIGMOID,
                                  dtype=moe.MOE_FP32 if dtype == torch.float32 else moe.MOE_BF16)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, std=1.0, dt=torch.float32: (torch.randn(s, generator=g, device="cuda") * std).to(dt)  # noqa: E731
        self.p = dict(
            n1=torch.ones(H, device="cuda"), n2=torch.ones(H, device="cuda"),
            Wr1=rand(H, E, std=0.1), Wg=rand(E, H, F, std=H ** -0.5, dt=dtype), Wu=rand(E, H, F, std=H ** -0.5, dt=dtype),
            Wd=rand(E, F, H, std=F ** -0.5, dt=dtype),
            Wr2=rand(H, E, std=0.1), A=rand(E, H, F, std=H ** -0.5, dt=dtype), B=rand(E, F, H, std=F ** -0.5, dt=dtype))

    # ---- block 2: routing, sort, experts of the caller's own, back
    def route(self, y, Wr):
        """Top-k experts and gates of each token (moe_route_static)."""
        T, k, E = y.shape[0], self.k, self.E
        topk = torch.empty((T, k), dtype=torch.int32, device="cuda")
        gates = torch.empty((T, k), device="cuda")
        counts, offsets = (torch.empty(E + 4, dtype=torch.int32, device="cuda") for _ in range(2))
        row_of = torch.empty_like(topk)
        st = moe.load_library().moe_route_static(
            self.layer.plan, T, y.data_ptr(), Wr.data_ptr(), None, topk.data_ptr(), gates.data_ptr(), counts.data_ptr(),
            offsets.data_ptr(), row_of.data_ptr(), torch.cuda.current_stream().cuda_stream)
        if st != moe.MOE_OK:
            raise moe.MoEError(st, "moe_route_static")
        return topk, gates

    def forward(self, x):
        p, s = self.p, {}
        s["x"] = x
        n = moe.add_rms_norm(x, p["n1"], want_rstd=True)
        s["y1"], s["r1"] = n["y"], n["rstd"]
        s["m1"] = self.layer.forward(s["y1"], p["Wr1"], None, p["Wg"], p["Wu"], p["Wd"])
        n = moe.add_rms_norm(s["m1"], p["n2"], x, want_rstd=True)
        s["h2"], s["y2"], s["r2"] = n["h"], n["y"], n["rstd"]
        s["topk"], s["gates"] = self.route(s["y2"], p["Wr2"])
        ix = s["index"] = moe.sort_index(s["topk"], self.E, self.align)
        s["X"] = moe.sort_rows(s["y2"], ix)
        s["Z"] = moe.grouped_matmul(s["X"], p["A"], ix)
        s["R"] = s["Z"].relu().square()
        s["Y"] = moe.grouped_matmul(s["R"], p["B"], ix)
        return moe.unsort_rows(s["Y"], ix, s["gates"], s["h2"]), s

    def backward(self, dout, s):
        p, ix = self.p, s["index"]
        d = {}
        dY, dg = moe.unsort_rows_backward(dout, s["Y"], ix, s["gates"])
        dR, d["B"] = moe.grouped_matmul_backward(dY, s["R"], p["B"], ix)
        dX, d["A"] = moe.grouped_matmul_backward(2 * s["Z"].relu() * dR, s["X"], p["A"], ix)
        # the router's share: sigmoid scores over their sum
        chosen = s["topk"].long()
        score = torch.sigmoid((s["y2"].float() @ p["Wr2"]).gather(1, chosen))
        dl = score * (1 - score) * (dg - (dg * s["gates"]).sum(1, keepdim=True)) / score.sum(1, keepdim=True)
        dlogits = torch.zeros((len(dl), self.E), device="cuda").scatter_(1, chosen, dl)
        d["Wr2"] = s["y2"].float().T @ dlogits
        dy2 = moe.unsort_rows(dX, ix, None, (dlogits @ p["Wr2"].T).to(self.dtype))
        dm1, d["n2"] = moe.add_rms_norm_backward(dy2, s["h2"], s["r2"], p["n2"], dout)
        g = self.layer.backward(dm1, s["y1"], p["Wr1"], p["Wg"], p["Wu"], p["Wd"])
        d.update(Wr1=g["dWr"], Wg=g["dW_gate"], Wu=g["dW_up"], Wd=g["dW_down"])
        dx, d["n1"] = moe.add_rms_norm_backward(g["dX"], s["x"], s["r1"], p["n1"], dm1)
        return dx, d

    def step(self, x, target, lr):
        out, s = self.forward(x)
        err = out.float() - target.float()
        _, d = self.backward((err * (2 / err.numel())).to(self.dtype), s)
        norm = moe.clip_grad_norm([d[n] for n in self.p], self.max_norm)
        for n, v in self.p.items():
            v.sub_(d[n], alpha=lr)
        return err.square().mean(), norm

    def decode(self, x):
        """One token through block 2, its experts' input as MXFP8 codes as well."""
        n = moe.add_rms_norm(x, self.p["n2"], torch.zeros_like(x), quant=moe.MOE_NORM_MXFP8)
        topk, gates = self.route(n["y"], self.p["Wr2"])
        ix = moe.sort_index(topk, self.E)
        X = moe.sort_rows(n["y"], ix)
        Y = moe.grouped_matmul(moe.grouped_matmul(X, self.p["A"], ix).relu().square(), self.p["B"], ix)
        return moe.unsort_rows(Y, ix, gates, n["h"]), n["codes"], n["scales"]

    def codes(self):
        """Block 2's weights as they are now, as E4M3 codes and scales of 128 x 128 tiles."""
        return {n: moe.quantize_tiles(self.p[n]) for n in ("A", "B")}

    def decode_8bit(self, x, codes):
        """Tokens through block 2 with the experts' weights in these codes."""
        n = moe.add_rms_norm(x, self.p["n2"], torch.zeros_like(x))
        topk, gates = self.route(n["y"], self.p["Wr2"])
        ix = moe.sort_index(topk, self.E)
        X = moe.quantize_rows(moe.sort_rows(n["y"], ix), ix)
        R = moe.quantize_rows(moe.fp8_matmul(*X, *codes["A"], ix).relu().square(), ix)
        return moe.unsort_rows(moe.fp8_matmul(*R, *codes["B"], ix), ix, gates, n["h"])


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    m = Blocks()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((m.T, m.H), generator=g, device="cuda").to(m.dtype)
    target = torch.randn((m.T, m.H), generator=g, device="cuda").to(m.dtype)
    for i in range(a.steps):
        loss, norm = m.step(x, target, lr=0.5)
        print(f"step {i}: loss {loss.item():.4f}, gradient norm {norm.item():.4f}")
    y, codes, scales = m.decode(x[:1])
    print(f"decoded one token: |y| {y.float().norm().item():.3f}, {codes.numel()} codes, {scales.numel()} scale bytes")
    y8 = m.decode_8bit(x[:1], m.codes())
    print(f"with 8-bit experts: |y| {y8.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
