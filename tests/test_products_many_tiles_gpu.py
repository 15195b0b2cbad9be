"""Products whose blocks take several tiles with products each (some hundred tiles
of every kernel): what a block carries from tile to tile, stages and phases,
accumulators, slots of scales, and full tiles of the larger fp32 kernels."""
import pytest
import torch

import mixture_experts_layer_sigmoid_gb300 as moe  # noqa: F401
import test_fp8_matmul_gpu as fp8
import test_grouped_gpu as grouped

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
#: segments of any length, empty ones between: 7033 rows, 61 tiles of 128
RAGGED = [700, 0, 1111, 513, 128, 0, 0, 2049, 300, 127, 1500, 1, 64, 540]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("K", [128, 384, 640, 896])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_codes(K, dtype, layout):
    """61 x 7 tiles of 1, 3, 5 and 7 blocks: odd counts, part groups of scales."""
    fp8.run(RAGGED, K, 1680, dtype, layout=layout, seed=K)


@pytest.mark.parametrize("align,counts", [(300, True), (128, True), (128, False)])
def test_codes_with_padding(align, counts):
    """Tiles without products between those that have some."""
    fp8.run(RAGGED, 640, 1200, BF, align=align, counts=counts)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("K,N", [(136, 2600), (320, 2608), (2600, 328)])
def test_rows_of_short_segments(K, N, layout):
    """40 experts of up to 127 rows, 11 column tiles: the kernel of single CTAs."""
    grouped.run_all([(37 * i) % 128 for i in range(1, 41)], K, N, BF, layout=layout, seed=K)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("K,N", [(320, 1032), (1032, 136)])
def test_rows_of_few(K, N, layout):
    """90 experts of up to 40 rows, 17 column tiles of 64."""
    grouped.run_all([(11 * i) % 41 for i in range(1, 91)], K, N, BF, layout=layout, seed=K)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("align", [1, 300])
def test_rows_and_gradients_in_pairs(align, layout):
    """Units of 256 rows and of 128, five or more column tiles; weight gradients of 14 experts."""
    grouped.run_all(RAGGED, 1096, 1304, BF, align=align, layout=layout)


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_gradients_of_narrow_weights(layout):
    """72 outputs of a weight gradient in one CTA's rows: 60 experts, four column tiles."""
    grouped.run_all([(53 * i) % 300 for i in range(60)], 72, 808, BF, layout=layout)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("K,N", [(1001, 2051), (333, 1537)])
def test_off_the_16_byte_boundaries(K, N, layout):
    grouped.run_all([900, 0, 1111, 513, 127, 0, 1049, 300, 1500, 1, 499], K, N, BF, layout=layout, seed=K)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("K,N", [(200, 1100), (203, 1101), (1100, 200), (1101, 203)])
def test_fp32_rows_in_the_larger_tiles(K, N, layout):
    """About 9000 rows: 71 x 9 tiles of 128 x 128."""
    grouped.run_all([2000, 0, 1111, 2513, 128, 0, 2049, 1300, 127], K, N, F32, layout=layout, seed=K)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M", [1200, 1203])
def test_fp32_weight_gradients_in_the_larger_tiles(M, layout):
    """8 experts of some hundred rows, 10 x 10 tiles of 128 x 128 each."""
    grouped.run_all([500, 0, 311, 513, 128, 64, 349, 33], M, M, F32, layout=layout, seed=M)
