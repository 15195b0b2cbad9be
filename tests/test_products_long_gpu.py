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
