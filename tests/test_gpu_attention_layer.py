"""The attention layer of examples/attention_layer.py: the attention rows of a prefill and of decode
steps against fp64 over what the layer holds in its caches, and the layer's calls on both sides of
the attention against the library's own products."""
import importlib.util
import os

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
from attn_ref import check_decode, check_prompt

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


def test_prefill_and_steps(example):
    layer = example.AttentionLayer(hidden=512, heads=8, kv_heads=2, dim=64, seed=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    lens = [130, 7]
    x = torch.randn(sum(lens), 512, generator=g, device=DEV)
    cu = torch.tensor([0, 130, 137], dtype=torch.int32, device=DEV)
    y, attended, (q, k, v) = layer.prefill(x, cu)
    check_prompt(q, k, v, lens, lens, True, 64 ** -0.5, attended)
    assert y.shape == (137, 512) and bool(torch.isfinite(y).all())
    # the first prompt becomes the prefix of three requests
    prefix = (k[:130], v[:130])
    caches = tuple(torch.full((3, 9, 2, 64), float("nan"), dtype=layer.dtype, device=DEV) for _ in range(2))
    n = torch.zeros(3, dtype=torch.int32, device=DEV)
    for _ in range(4):
        token = torch.randn(3, 512, generator=g, device=DEV)
        y, attended, q, n = layer.step(token, prefix, caches, n)
        check_decode(q, caches[0], caches[1], n, *prefix, 64 ** -0.5, attended)
        assert bool(torch.isfinite(y).all())
    assert n.tolist() == [4, 4, 4]


def test_a_step_continues_a_prefill(example):
    """The step's query, key and value are those of the next row of a longer prefill, to the rounding
    of a product whose fp32 sums run in another order (1e-5 of its terms) and one 16-bit rounding."""
    layer = example.AttentionLayer(hidden=512, heads=4, kv_heads=4, dim=64, seed=5)
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(66, 512, generator=g, device=DEV)
    _, _, (q, k, v) = layer.prefill(x, torch.tensor([0, 66], dtype=torch.int32, device=DEV))
    caches = tuple(torch.zeros(1, 2, 4, 64, dtype=layer.dtype, device=DEV) for _ in range(2))
    _, _, q1, n = layer.step(x[65:], (k[:65], v[:65]), caches, torch.zeros(1, dtype=torch.int32, device=DEV))
    for a, b in ((q1[0], q[65]), (caches[0][0, 0], k[65]), (caches[1][0, 0], v[65])):
        a, b = a.double(), b.double()
        assert float((a - b).norm() / b.norm()) <= 2 * 2.0 ** -8
