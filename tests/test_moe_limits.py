"""Sizes the mixture-of-experts products refuse because of how they work; on the
CPU, nothing is launched."""
import gguf_quant_dequant_q4k_b200 as q4k
from test_moe_abi import product_status


def test_gated_gemm_refuses_rows_its_waits_do_not_cover():
    """q4k_moe_gemm_swiglu_f16 keeps one sum for a whole row, for which its epilogue
    waits a second at most. The plain form, which takes sums of 768 products, has no
    such limit."""
    k = 1 << 24
    far = dict(w=1 << 40, w2=1 << 41, x=1 << 42)
    assert product_status("q4k_moe_gemm_swiglu_f16", k=k + 256, n_pairs=0, **far) == q4k.Q4K_ERR_SHAPE
    assert product_status("q4k_moe_gemm_swiglu_f16", k=k, n_pairs=0, **far) == q4k.Q4K_OK
    assert product_status("q4k_moe_gemm_f16", k=k + 256, n_pairs=0, **far) == q4k.Q4K_OK
    assert k == q4k.Q4K_MOE_GEMM_SWIGLU_MAX_K
