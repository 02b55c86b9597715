"""The hand-over of cleaned value tiles to the tensor cores: prompts whose only key tile ends inside the
tile, so that the zeroed rows of the first piece of work are all that stands between NaN and the output."""
import math

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
from attn_ref import check_prompt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 7, 64, 101, 127])
def test_one_ragged_key_tile(n, d, dt):
    qmm.build()
    hq, hk = 8, 2
    g = torch.Generator(device=DEV).manual_seed(n + d)
    q = torch.randn(n, hq, d, generator=g, device=DEV).to(dt)
    k, v = (torch.full((n + 128, hk, d), math.nan, dtype=dt, device=DEV) for _ in range(2))
    k[:n], v[:n] = (torch.randn(n, hk, d, generator=g, device=DEV).to(dt) for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    first = qmm.qmm_attn_prompt(q, k, v, cu, cu)
    check_prompt(q, k, v, [n], [n], True, d ** -0.5, first)
    outs = [qmm.qmm_attn_prompt(q, k, v, cu, cu) for _ in range(200)]
    assert all(torch.equal(o, first) for o in outs)
