"""The attention kernels' bounded waits are made to run out: with the test switch set no copy is
issued, the first wait for one gives up (after about 10^5 cycles), the kernel leaves and reports
QMM_ERR_DEVICE, and the next call on the same stream and workspace is right."""
import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
from attn_ref import check_decode, check_prompt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
QMM_ERR_DEVICE = 8


@pytest.fixture(autouse=True)
def _switch_off():
    qmm.build()
    yield
    qmm.qmm_set_test_fault(0)


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).half()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk", [(200, 200), (20, 4000)])  # one key range, and split keys with their join
def test_prompt_wait_runs_out_then_recovers(d, lq, lk):
    q, k, v = normal(1, lq, 4, d), normal(2, lk, 2, d), normal(3, lk, 2, d)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (lq, lk))
    ws = torch.empty(qmm.qmm_workspace_bytes_attn_prompt(lq, lk, 1, 4, 2, d), dtype=torch.uint8, device=DEV)
    qmm.qmm_set_test_fault(1)
    qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k, workspace=ws)
    assert qmm.qmm_read_device_status(ws) == QMM_ERR_DEVICE
    assert qmm.qmm_get_device_status(ws) == QMM_ERR_DEVICE
    qmm.qmm_set_test_fault(0)
    out = qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k, workspace=ws)
    assert qmm.qmm_get_device_status(ws) == 0
    check_prompt(q, k, v, [lq], [lk], True, d ** -0.5, out)


@pytest.mark.parametrize("p,b", [(0, 3), (500, 3), (9000, 20)])  # caches; a prefix read inline; one read once
def test_decode_wait_runs_out_then_recovers(p, b):
    d = 128
    q, k, v = normal(4, b, 8, d), normal(5, b, 200, 2, d), normal(6, b, 200, 2, d)
    pk, pv = (normal(7, p, 2, d), normal(8, p, 2, d)) if p else (None, None)
    lens = torch.arange(200, 200 - b, -1, dtype=torch.int32, device=DEV)
    ws = torch.empty(qmm.qmm_workspace_bytes_attn_decode(b, 200, p, 8, 2, d), dtype=torch.uint8, device=DEV)
    qmm.qmm_set_test_fault(1)
    qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, workspace=ws)
    assert qmm.qmm_read_device_status(ws) == QMM_ERR_DEVICE
    qmm.qmm_set_test_fault(0)
    out = qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, workspace=ws)
    assert qmm.qmm_get_device_status(ws) == 0
    check_decode(q, k, v, lens, pk, pv, d ** -0.5, out)
