"""Pages that do not exist, down to the bits: what rows read from them hold."""
import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
from test_gpu_kv import BF, DEV, FP, QMM_ERR_IDS, _errors, _lib, filled, gen, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
@pytest.mark.parametrize("dt", [BF, FP])
def test_rows_of_no_page_are_positive_zeros(qtype, dt):
    lens, hk, d, page = [40, 20], 3, 96, 16
    cache, table, _, _ = filled(gen(1), lens, qtype, page, hk, d)
    table[0, 1] = cache.pages.shape[0]
    table[1, 0] = -1
    for out in qmm.qmm_kv_read(cache, table, ints([0, 40, 60]), 60, out_dtype=dt):
        bits = out.view(torch.int16)
        assert not bits[16:32].any() and not bits[40:56].any()
        assert out[:16].any() and out[32:40].any() and out[56:].any()
    assert qmm.qmm_take_attn_error() == QMM_ERR_IDS
