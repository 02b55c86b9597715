"""A wait of the attention kernels gives up while copies are in flight (test switch 2: the copies are
issued, the first wait for one gives up at once): the call reports QMM_ERR_DEVICE, and the calls
queued right behind it, which take the same shared memory, are right."""
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


def fail_then_run(call, ws):
    for _ in range(20):
        qmm.qmm_set_test_fault(2)
        call()
        qmm.qmm_set_test_fault(0)
        out = call()  # queued behind the call that gave up
    assert qmm.qmm_get_device_status(ws) == 0
    qmm.qmm_set_test_fault(2)
    call()
    assert qmm.qmm_read_device_status(ws) == QMM_ERR_DEVICE
    qmm.qmm_set_test_fault(0)
    assert torch.equal(call(), out)
    assert qmm.qmm_get_device_status(ws) == 0
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk,hq,hk", [
    (60, 60, 4, 2),        # one key tile: every copy is issued before any wait of the copy warp
    (200, 900, 4, 2),      # more key tiles than the ring holds
    (20, 4000, 4, 2),      # split keys and their join
    (3000, 3000, 16, 8),   # more pieces than SMs
])
def test_prompt_copies_in_flight(d, lq, lk, hq, hk):
    q, k, v = normal(1, lq, hq, d), normal(2, lk, hk, d), normal(3, lk, hk, d)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (lq, lk))
    ws = torch.empty(qmm.qmm_workspace_bytes_attn_prompt(lq, lk, 1, hq, hk, d), dtype=torch.uint8, device=DEV)
    out = fail_then_run(lambda: qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k, workspace=ws), ws)
    check_prompt(q, k, v, [lq], [lk], True, d ** -0.5, out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b,room,p", [
    (3, 40, 0),       # one tile
    (2, 5000, 0),     # clusters, more tiles than the ring holds
    (200, 300, 0),    # more CTAs than fit at once
    (3, 200, 500),    # a prefix read inline
    (20, 200, 16500), # a prefix read once
])
def test_decode_copies_in_flight(d, b, room, p):
    q, k, v = normal(4, b, 8, d), normal(5, b, room, 2, d), normal(6, b, room, 2, d)
    pk, pv = (normal(7, p, 2, d), normal(8, p, 2, d)) if p else (None, None)
    lens = torch.full((b,), room, dtype=torch.int32, device=DEV)
    ws = torch.empty(qmm.qmm_workspace_bytes_attn_decode(b, room, p, 8, 2, d), dtype=torch.uint8, device=DEV)
    assert (ws.numel() > 256) == (p > 1000)
    out = fail_then_run(lambda: qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, workspace=ws), ws)
    check_decode(q, k, v, lens, pk, pv, d ** -0.5, out)
