"""Products that run for seconds: waits that last as long as the work they wait for."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_products_that_run_for_seconds():
    """A product of more than three seconds in CTA pairs: nothing in it waits for the whole
    of it with a limit. Zeros but for some columns of one row and one weight."""
    n = 147456
    x = torch.zeros((n, n), dtype=BF, device="cuda")
    w = torch.zeros((1, n, n), dtype=BF, device="cuda")
    y = torch.full((n, n), float("nan"), dtype=BF, device="cuda")
    x[n - 3, 7::1000], w[0, 7::1000, n - 5] = 2, 3
    moe.products_status()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    moe.grouped_matmul(x, w, None, out=y)
    b.record()
    assert moe.products_status() == moe.MOE_OK
    assert a.elapsed_time(b) > 2000
    # 148 products of 6: 888, a bf16 value
    assert float(y[n - 3, n - 5]) == 888 and float(y[n - 3].float().sum()) == 888
    y[n - 3, n - 5] = 0
    assert not any(bool(y[r:r + 8192].any()) for r in range(0, n, 8192))


def check_gradient_of_many_rows(lengths, M, N):
    """Zeros but for one row in a million (and the first and last) of the long segments."""
    E, R = len(lengths), sum(lengths)
    ix = dict(offsets=torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), dtype=torch.int32, device="cuda"))
    x, dy = torch.zeros((R, M), dtype=BF, device="cuda"), torch.zeros((R, N), dtype=BF, device="cuda")
    w = torch.empty((E, M, N), dtype=BF, device="cuda")
    want, at = torch.zeros((E, M, N), device="cuda"), 0
    for e, n in enumerate(lengths):
        rows = sorted({*range(at, at + n, 1000003), at + n - 1} if n else ())
        x[rows, 1], dy[rows, 2] = 1, 0.5
        want[e, 1, 2] = 0.5 * len(rows)
        at += n
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    moe.products_status()
    a.record()
    _, dw = moe.grouped_matmul_backward(dy, x, w, ix, want_drows=False)
    b.record()
    assert moe.products_status() == moe.MOE_OK
    assert a.elapsed_time(b) > 2000
    assert torch.equal(dw.float(), want.to(BF).float())


@pytest.mark.parametrize("M,N,rows", [(3, 5, 180000000), (8, 8, 700000000)])
def test_a_gradient_whose_only_tile_takes_seconds(M, N, rows):
    """The outputs' wait for a tile lasts as long as its contraction."""
    check_gradient_of_many_rows([rows], M, N)


def test_a_short_segment_behind_a_long_one():
    """The last, partial block of a short segment comes after all of a long one in the same block."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    check_gradient_of_many_rows([700000000 // 64 * 64] + [0] * (sms - 1) + [10], 8, 8)
