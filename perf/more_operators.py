"""Timed cases of the experts' matrix products: rows sorted by expert times each
expert's weights, with the gradients of both (bf16, fp32); the same product, and
the dense one, on E4M3 codes with a scale for each block of 128; and the codes
of activation rows.

``own`` selects the framework's calls; otherwise ``run`` computes the same in
elementary fp32 torch operations, rounded once at the end.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
MAX_FLOPS = {"bf16": 1.6e12, "fp32": 2.5e11, "fp8": 1.6e12}
MAX_WEIGHTS = 9e8      # values of the experts' weights
MAX_ROWS = 5e8         # values of the rows on either side


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of four sequences: few rows for each of the chosen experts, the weights are read once
        dict(name="gmm_decode", op="gmm", T=4, k=8, E=128, K=4096, N=1536, dtype="bf16", align=1, skew=0.0, drop=0.0, layout="kn"),
        # a training step's up projection at the Qwen3-shaped layer, 128-row segments, skewed routing
        dict(name="gmm_train", op="gmm", T=16384, k=8, E=128, K=4096, N=1536, dtype="bf16", align=128, skew=0.5, drop=0.0, layout="kn"),
        # odd widths, unpadded segments, dropped assignments, weights stored out x in
        dict(name="gmm_odd", op="gmm", T=1777, k=3, E=11, K=1001, N=771, dtype="bf16", align=1, skew=0.5, drop=0.1, layout="nk"),
        # a small fp32 model's experts
        dict(name="gmm_fp32", op="gmm", T=1021, k=2, E=5, K=1024, N=640, dtype="fp32", align=1, skew=0.5, drop=0.0, layout="kn"),
        # gradients of the Mixtral-shaped layer's up projection
        dict(name="gmm_bwd_train", op="gmm_bwd", T=4096, k=2, E=8, K=4096, N=14336, dtype="bf16", align=128, skew=0.0, drop=0.0, layout="kn"),
        # gradients for many experts of about 256 rows each, segments of any length (a quarter of the DeepSeek-V3-shaped experts)
        dict(name="gmm_bwd_many", op="gmm_bwd", T=2048, k=8, E=64, K=7168, N=2048, dtype="bf16", align=1, skew=0.5, drop=0.0, layout="kn"),
        # the fp32 test layer's gradients
        dict(name="gmm_bwd_fp32", op="gmm_bwd", T=256, k=2, E=4, K=128, N=256, dtype="fp32", align=1, skew=0.0, drop=0.0, layout="kn"),
        # sixteen sequences decoded by 8-bit experts
        dict(name="fp8_decode", op="fp8", T=16, k=8, E=128, K=7168, N=2048, dtype="bf16", align=1, skew=0.0, drop=0.0, layout="kn"),
        # a training step's dense projection on 8-bit operands, or the gradient of one: weights stored out x in
        dict(name="fp8_dense", op="fp8", T=8192, k=1, E=0, K=7168, N=4096, dtype="bf16", align=1, skew=0.0, drop=0.0, layout="nk"),
        # the Qwen3-shaped step on 8-bit operands
        dict(name="fp8_train", op="fp8", T=16384, k=8, E=128, K=4096, N=1536, dtype="bf16", align=128, skew=0.5, drop=0.0, layout="kn"),
        # a decode batch's activations to codes
        dict(name="quant_decode", op="quant", T=33, k=1, E=0, K=7168, dtype="bf16", align=1, skew=0.0, drop=0.0),
        # a training step's sorted rows to codes, up to the last row in use
        dict(name="quant_train", op="quant", T=16384, k=8, E=128, K=4096, dtype="bf16", align=128, skew=0.5, drop=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gmm", "gmm", "gmm_bwd", "gmm_bwd", "fp8", "fp8", "quant"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    E = _log(rng, 1, 256)
    if op in ("fp8", "quant") and rng.random() < 0.3:
        E = 0                                     # dense
    K, N = _log(rng, 64, 8192), _log(rng, 64, 8192)
    if op in ("fp8", "quant"):
        K = -(-K // 128) * 128
        N = -(-N // 16) * 16
    elif rng.random() < 0.6:
        K, N = -(-K // 8) * 8, -(-N // 8) * 8
    k = rng.randint(1, min(8, max(1, E))) if E else 1
    align = rng.choice([1, 16, 128]) if E else 1
    if E:
        E = max(1, min(E, int(MAX_WEIGHTS // (K * N))))
        k = min(k, E)
    most = MAX_ROWS / max(K, N)
    if op != "quant":
        most = min(most, MAX_FLOPS["fp8" if op == "fp8" else dtype] / (2.0 * K * N * (2 if op == "gmm_bwd" else 1)))
    T = max(1, min(_log(rng, 1, 16384), int(most) // k))
    if align > 1 and T * k < 4 * E:
        align = 1
    c = dict(op=op, T=T, k=k, E=E, K=K, dtype=dtype, align=align, skew=rng.choice([0.0, 0.5, 1.0]) if E else 0.0,
             drop=rng.choice([0.0, 0.05, 0.3]) if E else 0.0)
    if op != "quant":
        c["N"], c["layout"] = N, rng.choice(["kn", "nk"])
    return c


# ------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def rows_cap(T, k, E, align):
    n = T * k
    return -(-(n + min(E, n) * (align - 1)) // align) * align


def _route(case, g):
    """The index of a skewed random routing: counts, padded offsets, each slot's
    row (-1: dropped) and each row's slot (-1: padding), and on the host the
    segments (expert, first row, rows) that hold rows."""
    T, k, E, align = case["T"], case["k"], case["E"], case["align"]
    rank = torch.randperm(E, generator=g, device="cuda").float() + 1
    noise = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    topk = torch.topk(-case["skew"] * torch.log(rank) - torch.log(-torch.log(noise)), k, dim=1).indices
    if case["drop"]:
        topk = torch.where(torch.rand((T, k), generator=g, device="cuda") < case["drop"], torch.full_like(topk, E), topk)
    ids = topk.reshape(-1)
    counts = torch.bincount(ids, minlength=E + 1)
    offsets = torch.zeros(E + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum((counts[:E] + align - 1) // align * align, 0)
    order = torch.sort(ids, stable=True).indices
    by = ids[order]
    place = torch.arange(T * k, device="cuda") - (torch.cumsum(counts, 0) - counts)[by]
    row = torch.where(by < E, offsets[by.clamp(max=E - 1)] + place, torch.full_like(place, -1))
    row_of = torch.empty_like(row)
    row_of[order] = row
    cap = rows_cap(T, k, E, align)
    slot_of = torch.full((cap + 1,), -1, dtype=torch.long, device="cuda")
    slot_of[torch.where(row >= 0, row, torch.full_like(row, cap))] = order
    index = dict(counts=counts[:E].int(), offsets=offsets.int(), row_of=row_of.view(T, k).int(), slot_of=slot_of[:cap].int())
    seg = [(e, o, c) for e, (o, c) in enumerate(zip(offsets.tolist(), counts[:E].tolist())) if c]
    return index, seg, cap


def _rows(g, index, n, H, dtype, std=1.0):
    """n rows of activations; the padding rows (and those behind the last segment) are zeros."""
    x = torch.empty((n, H), device="cuda", dtype=dtype).normal_(0.0, std, generator=g)
    if index is not None:
        x.mul_((index["slot_of"] >= 0)[:, None])
    return x


def _weights(g, E, K, N, layout, dtype):
    """E x K x N weights; layout "nk" stores each expert's transpose."""
    shape = (E, K, N) if layout == "kn" else (E, N, K)
    w = torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, K ** -0.5, generator=g)
    return w if layout == "kn" else w.transpose(1, 2)


def _codes_of(x):
    """E4M3 codes (as bytes) and fp32 scales of 1x128 blocks. (A tensor of 448s divides;
    a number would be multiplied by its reciprocal on the GPU.)"""
    M, K = x.shape
    codes = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    scales = torch.empty((M, K // 128), device=x.device)
    for r in range(0, M, 16384):
        b = x[r:r + 16384].float().view(-1, K // 128, 128)
        amax = b.abs().amax(2)
        sc = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))
        scales[r:r + 16384] = sc
        codes[r:r + 16384] = (b / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, K)
    return codes, scales


def _tile_codes(w):
    """Codes and one scale for each 128x128 tile of a matrix (the last tiles may be partial)."""
    R, C = w.shape
    v = torch.zeros((-(-R // 128) * 128, -(-C // 128) * 128), device=w.device)
    v[:R, :C] = w
    amax = v.abs().view(v.shape[0] // 128, 128, v.shape[1] // 128, 128).amax((1, 3))
    sc = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))
    q = (v / sc.repeat_interleave(128, 0).repeat_interleave(128, 1)).to(torch.float8_e4m3fn)
    return q[:R, :C].contiguous().view(torch.uint8), sc


def prepare(case, seed):
    op, g, s = case["op"], _gen(seed), dict(case=case)
    K, dt = case["K"], DT[case["dtype"]]
    index, seg, cap = _route(case, g) if case["E"] else (None, [(0, 0, case["T"])], case["T"])
    s["index"], s["seg"] = index, seg
    chan = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))  # a few channels are far larger
    if op in ("quant", "fp8"):
        x = _rows(g, index, cap, K, dt if op == "quant" else torch.bfloat16)
        x.mul_(chan)
        if op == "quant":
            s["x"] = x
            s["codes"] = torch.zeros((cap, K), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.zeros((cap, K // 128), device="cuda")
            return s
        N, E = case["N"], max(1, case["E"])
        s["a"], s["sa"] = _codes_of(x)
        shape = (K, N) if case["layout"] == "kn" else (N, K)
        w = torch.empty((E,) + shape, dtype=torch.uint8, device="cuda")
        sw = torch.empty((E,) + tuple(-(-n // 128) for n in shape), device="cuda")
        for e in range(E):
            w[e], sw[e] = _tile_codes(torch.empty(shape, device="cuda").normal_(0.0, K ** -0.5, generator=g))
        if case["layout"] == "nk":
            w, sw = w.transpose(1, 2), sw.transpose(1, 2)
        s["w"], s["sw"] = (w, sw) if case["E"] else (w[0], sw[0])
        s["y"] = torch.zeros((cap, N), device="cuda", dtype=dt)
        return s
    E, N = case["E"], case["N"]
    s["w"] = _weights(g, E, K, N, case["layout"], dt)
    s["x"] = _rows(g, index, cap, K, dt)
    s["x"].mul_(chan)
    if op == "gmm":
        s["y"] = torch.zeros((cap, N), device="cuda", dtype=dt)  # the program's buffer
        return s
    s["dy"] = _rows(g, index, cap, N, dt, 0.1)
    s["dx"] = torch.zeros((cap, K), device="cuda", dtype=dt)
    s["dw"] = torch.zeros_like(s["w"])  # the gradient's buffer, laid out as the weights
    return s


# ------------------------------------------------------------------- plain forms
def _value(codes, scales):
    """The fp32 values of codes with 1x128 blocks."""
    M, K = codes.shape
    return (codes.view(torch.float8_e4m3fn).float().view(M, K // 128, 128) * scales[..., None]).view(M, K)


def _tile_value(w, sw):
    """The fp32 values of K x N codes with 128x128 tiles."""
    K, N = w.shape
    if w.stride(1) != 1:
        return _tile_value(w.t(), sw.t()).t()
    s = sw.repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :N]
    return w.view(torch.float8_e4m3fn).float() * s


def _run_plain(s, case):
    op = case["op"]
    if op == "quant":
        n, K, a = s["x"].shape[0], case["K"], case["align"]
        if s["index"] is not None:               # up to the last segment's end
            n = max((o + -(-c // a) * a for _, o, c in s["seg"]), default=0)
        b = s["x"][:n].float().view(n, K // 128, 128)
        amax = b.abs().amax(2)
        sc = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, 448.0))
        s["scales"][:n] = sc
        s["codes"][:n] = (b / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(n, K)
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    if op == "fp8":
        for e, o, c in s["seg"]:
            w, sw = (s["w"][e], s["sw"][e]) if case["E"] else (s["w"], s["sw"])
            s["y"][o:o + c] = _value(s["a"][o:o + c], s["sa"][o:o + c]) @ _tile_value(w, sw)
        return {"y": s["y"]}
    if op == "gmm":
        for e, o, c in s["seg"]:
            s["y"][o:o + c] = s["x"][o:o + c].float() @ s["w"][e].float()
        return {"y": s["y"]}
    live = {e: (o, c) for e, o, c in s["seg"]}
    for e in range(case["E"]):
        o, c = live.get(e, (0, 0))
        dy = s["dy"][o:o + c].float()
        if c:
            s["dx"][o:o + c] = dy @ s["w"][e].float().t()
        s["dw"][e] = s["x"][o:o + c].float().t() @ dy
    return {"dx": s["dx"], "dw": s["dw"]}


# ------------------------------------------------------------------- the framework's calls
def _run_own(s, case):
    import mixture_experts_layer_sigmoid_gb300 as moe
    op = case["op"]
    if op == "quant":
        codes, scales = moe.quantize_rows(s["x"], s["index"], codes=s["codes"], scales=s["scales"])
        return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
    if op == "fp8":
        return {"y": moe.fp8_matmul(s["a"], s["sa"], s["w"], s["sw"], s["index"], out=s["y"])}
    if op == "gmm":
        return {"y": moe.grouped_matmul(s["x"], s["w"], s["index"], out=s["y"])}
    dx, dw = moe.grouped_matmul_backward(s["dy"], s["x"], s["w"], s["index"], drows=s["dx"], dw=s["dw"])
    return {"dx": dx, "dw": dw}


def run(state):
    return _run_own(state, state["case"]) if own else _run_plain(state, state["case"])


# ------------------------------------------------------------------- what a pass has to move
def work(case):
    op, b, K = case["op"], SIZE[case["dtype"]], case["K"]
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k * (1 - case["drop"])                                    # rows that reach an expert
    used = E * (1 - (1 - k / E) ** (T * (1 - case["drop"]))) if E else 1  # experts that an even routing reaches
    if op == "quant":
        return {"bytes": R * K * (b + 1) + R * K / 128 * 4, "flops": 3 * R * K}
    N = case["N"]
    if op == "fp8":
        return {"bytes": R * K * (1 + 4 / 128) + used * K * N + R * N * b, "flops": 2 * R * K * N}
    if op == "gmm":
        return {"bytes": b * (R * (K + N) + used * K * N), "flops": 2 * R * K * N}
    return {"bytes": b * (R * (2 * K + N) + (used + E) * K * N), "flops": 4 * R * K * N}


# ------------------------------------------------------------------- the definitions in 64 bits
def _e4m3(v):
    """Nearest E4M3 value (ties to even), saturating at 448."""
    a = v.abs()
    e = torch.frexp(a).exponent - 1
    e = torch.where(a == 0, torch.full_like(e, -6), e).clamp(min=-6)
    step = torch.ldexp(torch.ones_like(a), e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)


def _spread(s, n, dim, size):
    """Block scales to one for each of `size` values along a dimension."""
    at = torch.arange(size, device=s.device) // n
    return s.double().index_select(dim, at)


def exact(case, seed):
    s = prepare(case, seed)
    op, K = case["op"], case["K"]
    index = s["index"]
    if op == "quant":
        M = s["x"].shape[0]
        codes = torch.zeros((M, K), dtype=torch.float64, device="cuda")
        scales = torch.zeros((M, K // 128), dtype=torch.float64, device="cuda")
        n = M if index is None else int(index["offsets"][-1])
        for r in range(0, n, 8192):
            q = min(n, r + 8192)
            x = s["x"][r:q].double()
            amax = x.abs().reshape(q - r, -1, 128).max(2).values
            scales[r:q] = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
            # the codes belong to the scales as they are stored, in fp32
            codes[r:q] = _e4m3(x / _spread(scales[r:q].float(), 128, 1, K))
        return {"codes": codes, "scales": scales}
    if index is None:
        bounds = torch.tensor([0, case["T"]])
        counts = [case["T"]]
    else:
        bounds, counts = index["offsets"].cpu(), index["counts"].tolist()
    E = len(counts)
    if op in ("gmm", "fp8"):
        y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        for e in range(E):
            rows = torch.arange(int(bounds[e]), int(bounds[e]) + counts[e], device="cuda")
            if op == "gmm":
                y[rows] = torch.einsum("rk,kn->rn", s["x"][rows].double(), s["w"][e].double())
            elif counts[e]:
                w, sw = (s["w"][e], s["sw"][e]) if case["E"] else (s["w"], s["sw"])
                wv = w.contiguous().view(torch.float8_e4m3fn).double()
                wv = wv * _spread(_spread(sw, 128, 0, K), 128, 1, case["N"])
                av = s["a"][rows].view(torch.float8_e4m3fn).double() * _spread(s["sa"][rows], 128, 1, K)
                y[rows] = torch.einsum("rk,kn->rn", av, wv)
        return {"y": y}
    dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = torch.arange(int(bounds[e]), int(bounds[e]) + counts[e], device="cuda")
        dy = s["dy"][rows].double()
        dx[rows] = torch.einsum("rn,kn->rk", dy, s["w"][e].double())
        dw[e] = torch.einsum("rk,rn->kn", s["x"][rows].double(), dy)
    return {"dx": dx, "dw": dw}
