"""The largest numbers of rows that the products take. Next to 2^31 the numbers of rows
behind a tile, or of a block of a contraction behind the last, would leave 32 bits."""
import ctypes

import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe
from mixture_experts_layer_sigmoid_gb300 import _build

MOST = 2 ** 31 - 1024
P, Q, R = 4096, 8192, 12288          # aligned addresses that nothing dereferences


def calls(lib, rows):
    g = ctypes.byref(moe.moe_groups_t(E=1, dtype=0, rows=rows, offsets=None, counts=None))
    a = moe.moe_fp8_matmul_args_t(A=P, lda=128, SA=Q, ldsa=1, B=P, ldb=16, sb=128 * 16, SB=Q, ldsb=1, ssb=1, b_nk=0, Y=R, ldy=16)
    return (lib.moe_grouped_matmul(g, 4, 4, P, 4, Q, 4, 16, 0, R, 4, None),
            lib.moe_grouped_wgrad(g, 4, 4, P, 4, Q, 4, R, 4, 16, None),
            lib.moe_fp8_matmul(g, 128, 16, ctypes.byref(a), None))


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: for a machine without a GPU only")
def test_more_rows_are_refused():
    _build.build()
    lib = moe.load_library()
    for rows in (MOST + 1, 2 ** 31 - 33, 2 ** 31 - 2):
        assert calls(lib, rows) == (moe.MOE_ERR_INVALID_ARG,) * 3
    assert moe.MOE_ERR_INVALID_ARG not in calls(lib, MOST)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,width", [(torch.float32, 1), (torch.bfloat16, 1), (torch.bfloat16, 8)])
def test_segments_at_the_end_of_the_most_rows(dtype, width):
    """The last forty of 2^31 - 1024 rows, whose sums are small whole numbers."""
    x = torch.zeros((MOST, width), dtype=dtype, device="cuda")
    y = torch.full((MOST, width), 7.0, dtype=dtype, device="cuda")
    four = (torch.arange(40, device="cuda") % 4)[:, None].to(dtype)
    x[-40:] = four
    w = torch.full((2, width, width), 2.0, dtype=dtype, device="cuda")
    ix = dict(offsets=torch.tensor([MOST - 40, MOST - 3, MOST], dtype=torch.int32, device="cuda"))
    moe.grouped_matmul(x, w, ix, out=y)
    assert bool((y[-40:] == 2 * width * four).all())
    assert bool((y[-41 - 1024:-40] == 7).all()) and bool((y[:1024] == 7).all())
    y[-40:] = 1
    _, dw = moe.grouped_matmul_backward(y, x, w, ix, want_drows=False)
    assert bool((dw[0] == 9 * (1 + 2 + 3)).all()) and bool((dw[1] == 1 + 2 + 3).all())
    assert moe.products_status() == moe.MOE_OK
