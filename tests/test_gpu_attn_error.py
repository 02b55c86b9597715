"""Device errors of attention calls that were given no workspace: a wait is made to run out (nothing
is copied), and qmm_take_attn_error says so once, however many calls succeed in between."""
import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
QMM_ERR_DEVICE = 8


@pytest.fixture(autouse=True)
def _switch_off():
    qmm.build()
    qmm.qmm_take_attn_error()
    yield
    qmm.qmm_set_test_fault(0)
    qmm.qmm_take_attn_error()


def half(*shape):
    return torch.randn(*shape, device=DEV).half()


def prompt(lq, lk):
    q, k = half(lq, 4, 64), half(lk, 2, 64)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (lq, lk))
    return lambda **kw: qmm.qmm_attn_prompt(q, k, k, cu_q, cu_k, **kw)


def decode(b, room, p):
    q, k = half(b, 8, 128), half(b, room, 2, 128)
    pk = half(p, 2, 128) if p else None
    lens = torch.full((b,), room, dtype=torch.int32, device=DEV)
    return lambda **kw: qmm.qmm_attn_decode(q, k, k, lens, prefix_k=pk, prefix_v=pk, **kw)


@pytest.mark.parametrize("make", [lambda: prompt(100, 100), lambda: prompt(20, 4000), lambda: decode(3, 100, 0),
                                  lambda: decode(3, 100, 300), lambda: decode(20, 100, 9000)],
                         ids=["prompt", "prompt_split", "decode", "decode_inline", "decode_prefix"])
@pytest.mark.parametrize("mode", [1, 2])
def test_an_error_without_a_workspace_is_kept(make, mode):
    call = make()
    call()
    assert qmm.qmm_take_attn_error() == 0
    qmm.qmm_set_test_fault(mode)
    call()
    qmm.qmm_set_test_fault(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):  # later calls, here and on another stream, do not hide it
        call()
        prompt(5, 5)()
        decode(1, 4, 0)()
        call(stream=side)
    torch.cuda.synchronize()
    assert qmm.qmm_take_attn_error() == QMM_ERR_DEVICE
    call()
    assert qmm.qmm_take_attn_error() == 0


def test_an_error_on_another_stream():
    call, side = decode(2, 50, 0), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmm.qmm_set_test_fault(1)
    call(stream=side)
    qmm.qmm_set_test_fault(0)
    assert qmm.qmm_take_attn_error(stream=side) == QMM_ERR_DEVICE
    assert qmm.qmm_take_attn_error() == 0
