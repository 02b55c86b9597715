"""The paged attention layer of examples/attention_layer.py: chunks of prompts and decode steps, the attention
rows against fp64 over the bytes that the cache holds."""
import importlib.util
import os

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
import kv_ref
from attn_ref import check_prompt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    qmm.build()
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
def test_chunks_and_steps(example, qtype):
    layer = example.PagedAttentionLayer(hidden=512, heads=8, kv_heads=2, dim=64, seed=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    cache = qmm.KVPages.empty(12, qtype, 16, 2, 64, device=DEV)
    table = torch.randperm(12, generator=g, device=DEV).to(torch.int32).view(2, 6)
    have = [0, 0]

    def held(i):
        j = torch.arange(have[i], device=DEV)
        return kv_ref.load(cache.pages, qtype, 16, 2, 64, table[i].long()[j // 16] * 16 + j % 16)

    for new in ([30, 7], [1, 40]):
        have = [a + n for a, n in zip(have, new)]
        cu_q, cu_k = (torch.tensor([0] + x, device=DEV).cumsum(0).to(torch.int32) for x in (new, have))
        x = torch.randn(sum(new), 512, generator=g, device=DEV)
        y, attended, q = layer.chunk(x, cache, table, cu_q, cu_k)
        k, v = (torch.cat([kv_ref.values(c[i], s[i]) for c, s in (held(0), held(1))]).float().to(layer.dtype) for i in range(2))
        check_prompt(q, k, v, new, have, True, 64 ** -0.5, attended)
        assert y.shape == (sum(new), 512) and bool(torch.isfinite(y).all())
    lens = torch.tensor(have, dtype=torch.int32, device=DEV)
    for _ in range(4):
        x = torch.randn(2, 512, generator=g, device=DEV)
        y, attended, q, lens = layer.step(x, cache, table, lens, 96)
        have = [a + 1 for a in have]
        both = [held(i) for i in range(2)]
        kv_ref.check_decode_kv(q, [[c[i] for c, _ in both] for i in range(2)], [[s[i] for _, s in both] for i in range(2)],
                               have, 64 ** -0.5, qtype, attended)
        assert bool(torch.isfinite(y).all())
    assert lens.tolist() == have and qmm.qmm_take_attn_error() == 0
