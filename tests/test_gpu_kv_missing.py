"""Pages that do not exist, down to the bits: rows read from them, and a cache that has no pages."""
import math

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
from test_gpu_kv import BF, DEV, FP, QMM_ERR_IDS, _errors, _lib, filled, gen, ints, normal, query  # noqa: F401

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


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
@pytest.mark.parametrize("page", [16, 64])
def test_a_cache_without_pages(qtype, page):
    """Reading it gives zeros in the sequences' rows and leaves the others; attending gives zeros."""
    hk, d = 2, 64
    cache = qmm.KVPages.empty(0, qtype, page, hk, d, device=DEV)
    table, g = torch.zeros((2, 6), dtype=torch.int32, device=DEV), gen(2)
    k, v = (torch.full((120, hk, d), 7.0, dtype=BF, device=DEV) for _ in range(2))
    qmm.qmm_kv_read(cache, table, ints([3, 73, 110]), 120, k_out=k, v_out=v)
    for out in (k, v):
        assert not out.view(torch.int16)[3:110].any() and bool((out[:3] == 7).all()) and bool((out[110:] == 7).all())
    assert qmm.qmm_take_attn_error() == QMM_ERR_IDS
    lse = torch.zeros(2, 4, device=DEV)
    out = qmm.qmm_attn_decode_kv(query(g, 2, 4, d, BF), cache, table, ints([70, 20]), lse=lse)
    assert not out.any() and bool((lse == -math.inf).all()) and qmm.qmm_take_attn_error() == QMM_ERR_IDS
    x = normal(g, 5, hk, d)
    _, ko, vo = qmm.qmm_kv_append(None, x, x, None, None, cache, ints([0, 1, 2, 3, 4]), values=True)
    assert torch.equal(ko, vo) and ko.any() and qmm.qmm_take_attn_error() == 0
