"""The wait of the products' kernels on a barrier that nothing signals: it gives up after its
limit, another one with the flag that the first raises, and products_status says so once."""
import time

import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_stalled_wait_is_reported_once(which):
    lib, stream = moe.load_library(), torch.cuda.current_stream().cuda_stream
    x, w = torch.ones((40, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((1, 64, 32), dtype=torch.bfloat16, device="cuda")
    want = moe.grouped_matmul(x, w, None)
    assert moe.products_status() == moe.MOE_OK
    t0 = time.time()
    assert lib.moe_diag_products_wait(which, stream) == moe.MOE_OK
    assert moe.products_status() == moe.MOE_ERR_DEVICE_TIMEOUT
    # 10 ms, and not the two seconds of the other wait
    assert 0.01 <= time.time() - t0 < 1.0
    assert moe.products_status() == moe.MOE_OK
    assert torch.equal(moe.grouped_matmul(x, w, None), want) and bool((want == 64).all())
    assert moe.products_status() == moe.MOE_OK


def test_two_stalled_waits_are_one_report():
    lib, stream = moe.load_library(), torch.cuda.current_stream().cuda_stream
    for which in (2, 0, 1):
        assert lib.moe_diag_products_wait(which, stream) == moe.MOE_OK
    assert moe.products_status() == moe.MOE_ERR_DEVICE_TIMEOUT
    assert moe.products_status() == moe.MOE_OK
