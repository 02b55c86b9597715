"""Attention calls on a stream of the caller's choice that make their outputs and workspaces
themselves: those never come from memory that the current stream still has work queued on."""
import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qmm.build()


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(BF)


def rope():
    q, k, v = normal(1, 300, 8, 128), normal(2, 300, 2, 128), normal(3, 300, 2, 128)
    pos, inv = torch.arange(300, device=DEV, dtype=torch.int32), torch.linspace(1, 1e-3, 64, device=DEV)
    return lambda **kw: qmm.qmm_qk_norm_rope(q, k, v, pos, inv, **kw), 0


def prompt(lq, lk):
    q, k, v = normal(4, lq, 8, 128), normal(5, lk, 2, 128), normal(6, lk, 2, 128)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=DEV) for n in (lq, lk))
    return (lambda **kw: qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k, **kw),
            qmm.qmm_workspace_bytes_attn_prompt(lq, lk, 1, 8, 2, 128))


def decode(b, room, p):
    q, k, v = normal(7, b, 8, 128), normal(8, b, room, 2, 128), normal(9, b, room, 2, 128)
    pk, pv = (normal(10, p, 2, 128), normal(11, p, 2, 128)) if p else (None, None)
    lens = torch.full((b,), room, dtype=torch.int32, device=DEV)
    return (lambda **kw: qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, **kw),
            qmm.qmm_workspace_bytes_attn_decode(b, room, p, 8, 2, 128))


def tensors(x):
    return x if isinstance(x, tuple) else (x,)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("make", [rope, lambda: prompt(300, 300), lambda: prompt(20, 4000),
                                  lambda: decode(5, 64, 0), lambda: decode(20, 100, 9000)],
                         ids=["rope", "prompt", "prompt_split", "decode", "decode_prefix"])
def test_tensors_a_call_makes_belong_to_its_stream(make, handle):
    call, ws_bytes = make()
    want = [t.clone() for t in tensors(call())]
    sizes = [t.numel() * t.element_size() for t in want] + ([ws_bytes] if ws_bytes > 256 else [])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the call's own sizes: freed, with work of the current stream on them still to run
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda._sleep(40_000_000)
    kept = [b.clone() for b in blocks]
    for b in blocks:
        b.fill_(9)
    ranges = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
    del b, blocks
    got = tensors(call(stream=side.cuda_stream if handle else side))
    for t in got:
        assert not any(a <= t.data_ptr() < z for a, z in ranges)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_outputs_given_stay_the_callers():
    call, _ = rope()
    want = tensors(call())
    mine = [torch.empty_like(t) for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side, q_out=mine[0], k_out=mine[1])
    side.synchronize()
    assert got[0] is mine[0] and got[1] is mine[1]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.cuda.current_stream() != side


def test_a_refusal_leaves_the_current_stream():
    call, _ = prompt(30, 30)
    before, side = torch.cuda.current_stream(), torch.cuda.Stream()
    with pytest.raises(qmm.QMMError):
        call(stream=side, scale=float("nan"))
    assert torch.cuda.current_stream() == before
    call(stream=0)
    call(stream=before)
    torch.cuda.synchronize()
