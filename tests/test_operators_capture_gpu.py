"""Operators captured where a launch that may start early has something else than
one kernel in front of it: nothing, a copy, a memset, or two streams that meet."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


def setup(T=60, k=4, E=9, H=264):
    g = torch.Generator(device="cuda").manual_seed(5)
    topk = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((T, H), generator=g, device="cuda")
    ix = moe.sort_index(topk, E, 8)
    return ix, x, torch.zeros((ix["slot_of"].numel(), H), device="cuda")


@pytest.mark.parametrize("before", ["nothing", "copy", "memset", "join"])
def test_rows_out_behind(before):
    ix, x, buf = setup()
    want = moe.sort_rows(x, ix, out=buf.clone())
    src, out = x.clone(), buf.clone()
    feed, side = x.clone(), torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        if before == "copy":
            src.copy_(feed)
        elif before == "memset":
            out.zero_()
        elif before == "join":
            here = torch.cuda.current_stream()
            side.wait_stream(here)
            with torch.cuda.stream(side):
                out.mul_(2)
            src.mul_(1.5)
            here.wait_stream(side)
        moe.sort_rows(src, ix, out=out)
    if before == "join":
        src.copy_(x / 1.5)
    gr.replay()
    torch.cuda.synchronize()
    used = int(ix["offsets"][-1])
    ref = moe.sort_rows(src, ix, out=buf.clone()) if before == "join" else want
    assert torch.equal(out[:used], ref[:used])


def test_a_step_in_one_graph():
    """Norm, index, rows, gradients and clipping in one capture, on two streams."""
    ix, x, buf = setup()
    topk = torch.randint(0, 9, (60, 4), device="cuda", dtype=torch.int32)
    w, gates = torch.ones(264, device="cuda"), torch.rand((60, 4), device="cuda")
    side = torch.cuda.Stream()

    def step():
        n = moe.add_rms_norm(x, w, x, want_rstd=True)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            dx, dw = moe.add_rms_norm_backward(x, n["h"], n["rstd"], w)
        i = moe.sort_index(topk, 9, 8)
        X = moe.sort_rows(n["y"], i, out=torch.zeros_like(buf))
        here.wait_stream(side)
        dY, dg = moe.unsort_rows_backward(dx, X, i, gates, out=torch.zeros_like(buf))
        norm = moe.clip_grad_norm([dw, dg], 0.1)
        y = moe.unsort_rows(X, i, gates, n["h"])
        return X, dY, dg, dw, norm, y

    ref = [t.clone() for t in step()]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    for _ in range(3):
        gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
