"""The attention calls of the C ABI refuse bad arguments before anything touches a GPU."""
import ctypes

import pytest

import block_quantized_matmul_q8_gb300 as qmm

P = ctypes.c_void_p
F16, BF16, F32 = 1, 30, 0


@pytest.fixture(scope="module")
def L():
    qmm.build()
    return qmm.lib()


def H(data=4096, token=512, head=64):
    return qmm.Heads(data, token, head)


def prompt(L, q=H(), k=H(), v=H(), t=BF16, tq=10, tk=10, hq=8, hk=2, d=64, cu_q=4096, cu_k=4096, n=1, scale=1.0,
           out=H(), lse=0, ws=1 << 20, wsb=1 << 40):
    return L.qmm_attn_prompt(q, k, v, t, tq, tk, hq, hk, d, P(cu_q), P(cu_k), n, 1, scale, out, P(lse), P(ws), wsb,
                             None)


def decode(L, q=H(), k=H(), v=H(), kb=1 << 16, vb=1 << 16, lens=4096, b=4, room=16, pk=None, pv=None, p=0, t=F16, hq=8,
           hk=2, d=64, scale=1.0, out=H(), lse=0, ws=1 << 20, wsb=1 << 40):
    return L.qmm_attn_decode(q, k, v, kb, vb, P(lens), b, room, pk, pv, p, t, hq, hk, d, scale, out, P(lse), P(ws),
                             wsb, None)


def rope(L, q=H(), k=H(), v=H(), t=F32, m=4, hq=8, hk=2, d=64, wq=4096, wk=4096, eps=1e-6, pos=4096, inv=4096, r=64,
         qo=H(), ko=H(), vo=H(), to=BF16):
    return L.qmm_qk_norm_rope(q, k, v, t, m, hq, hk, d, P(wq), P(wk), eps, P(pos), P(inv), r, 0, qo, ko, vo, to, None)


def test_prompt_refuses(L):
    assert prompt(L, t=F32) == 3 and prompt(L, t=7) == 3
    assert prompt(L, tq=-1) == 1 and prompt(L, n=-1) == 1 and prompt(L, hk=0) == 1 and prompt(L, d=0) == 1
    assert prompt(L, hq=7) == 2 and prompt(L, d=60) == 2 and prompt(L, d=136) == 2
    assert prompt(L, hq=129 * 2) == 2                                    # 129 query heads of one kv head
    assert prompt(L, tq=1 << 31) == 2 and prompt(L, n=(1 << 20) + 1) == 2
    assert prompt(L, scale=float("inf")) == 1 and prompt(L, scale=float("nan")) == 1
    assert prompt(L, q=None) == 1 and prompt(L, out=H(data=0)) == 1 and prompt(L, cu_k=0) == 1
    assert prompt(L, v=H(data=4104)) == 4 and prompt(L, k=H(token=516)) == 4 and prompt(L, q=H(head=68)) == 4
    assert prompt(L, k=H(token=32)) == 2 and prompt(L, q=H(head=0)) == 2   # views that overlap themselves
    assert prompt(L, q=H(token=1 << 40)) == 2
    assert prompt(L, cu_q=4098) == 4 and prompt(L, lse=4098) == 4
    need = L.qmm_workspace_bytes_attn_prompt(10, 10, 1, 8, 2, 64)
    assert need >= 16
    assert prompt(L, ws=0) == 5 and prompt(L, wsb=need - 1) == 5 and prompt(L, ws=(1 << 20) + 16) == 4


def test_decode_refuses(L):
    assert decode(L, t=F32) == 3
    assert decode(L, b=-1) == 1 and decode(L, room=-1) == 1 and decode(L, p=-1) == 1
    assert decode(L, hq=9) == 2 and decode(L, d=4) == 2 and decode(L, b=1 << 31) == 2 and decode(L, p=1 << 31) == 2
    assert decode(L, lens=0) == 1 and decode(L, k=None) == 1 and decode(L, p=5) == 1 and decode(L, q=None) == 1
    assert decode(L, kb=(1 << 16) + 4) == 4 and decode(L, vb=0) == 2 and decode(L, lens=4098) == 4
    assert decode(L, p=5, pk=H(), pv=H(data=4100)) == 4
    assert decode(L, scale=float("nan")) == 1
    need = L.qmm_workspace_bytes_attn_decode(4, 16, 0, 8, 2, 64)
    assert decode(L, ws=0) == 5 and decode(L, wsb=need - 1) == 5 and decode(L, ws=(1 << 20) + 64) == 4


def test_rope_refuses(L):
    assert rope(L, t=9) == 3 and rope(L, to=F32) == 3
    assert rope(L, m=-1) == 1 and rope(L, eps=-1.0) == 1 and rope(L, eps=float("nan")) == 1 and rope(L, r=-8) == 1
    assert rope(L, d=68) == 2 and rope(L, d=136) == 2 and rope(L, r=72) == 2 and rope(L, r=12) == 2
    assert rope(L, q=None) == 1 and rope(L, vo=None) == 1 and rope(L, v=None) == 1 and rope(L, pos=0) == 1
    assert rope(L, q=H(token=514)) == 4 and rope(L, ko=H(token=516)) == 4 and rope(L, qo=H(data=4098)) == 4
    assert rope(L, inv=4097) == 4
    assert rope(L, m=0) == 0


def test_workspace_bytes_zero_for_rejected_sizes(L):
    w = L.qmm_workspace_bytes_attn_prompt
    assert w(10, 10, 1, 8, 2, 64) > 0 and w(0, 0, 0, 8, 2, 64) > 0
    assert w(-1, 10, 1, 8, 2, 64) == 0 and w(10, 10, 1, 7, 2, 64) == 0 and w(10, 10, 1, 8, 2, 129) == 0
    w = L.qmm_workspace_bytes_attn_decode
    assert w(4, 16, 100, 8, 2, 64) > 0
    assert w(4, -1, 0, 8, 2, 64) == 0 and w(1 << 40, 16, 0, 8, 2, 64) == 0 and w(4, 16, 0, 8, 0, 64) == 0
