"""moe_diag_products_wait refuses what it does not know (CPU)."""
import mixture_experts_layer_sigmoid_gb300 as moe
from mixture_experts_layer_sigmoid_gb300 import _build


def test_an_unknown_word_is_refused():
    _build.build()
    lib = moe.load_library()
    assert lib.moe_diag_products_wait(-1, None) == lib.moe_diag_products_wait(3, None) == moe.MOE_ERR_INVALID_ARG
