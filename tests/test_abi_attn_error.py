"""qmm_take_attn_error refuses a missing result pointer before it touches a GPU."""
import block_quantized_matmul_q8_gb300 as qmm


def test_refuses_null():
    qmm.build()
    assert qmm.lib().qmm_take_attn_error(None, None) == 1
