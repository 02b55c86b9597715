"""Packed prompts of thousands of sequences: right in every row, and the search for pieces of work grows
with the number of sequences, not with its square."""
import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
from attn_ref import check_prompt

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qmm.build()


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(BF)


def milliseconds(q, k, cu):
    out = torch.empty_like(q)
    times = []
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        qmm.qmm_attn_prompt(q, k, k, cu, out=out)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return sorted(times)[1]


def test_time_grows_with_the_sequences():
    def run(n):  # n sequences of 4 tokens
        cu = (torch.arange(n + 1, device=DEV) * 4).to(torch.int32)
        return milliseconds(normal(1, 4 * n, 4, 64), normal(2, 4 * n, 2, 64), cu)

    assert run(16384) <= 16 * run(2048)  # 8 times the work; the square would be 64


@pytest.mark.parametrize("front", [True, False])
def test_time_grows_with_empty_sequences(front):
    def run(n):  # 8 sequences of 4096 tokens and n empty ones, each of which the grid counts a tile for
        cu = torch.arange(9, device=DEV) * 4096
        cu = torch.cat((torch.zeros(n, dtype=cu.dtype, device=DEV), cu) if front else (cu, cu[-1:].expand(n)))
        return milliseconds(normal(3, 32768, 2, 64), normal(4, 32768, 1, 64), cu.to(torch.int32))

    assert run(32768) <= 16 * run(2048)


def padded(x, lens, most):
    at = torch.arange(most, device=DEV) < torch.tensor(lens, device=DEV)[:, None]
    p = torch.zeros((len(lens), most, *x.shape[1:]), dtype=x.dtype, device=DEV)
    p[at] = x
    return p, at


def test_every_row_of_many_short_sequences():
    """16000 sequences of 0 to 6 tokens against fp64, as one padded batch.  Bound: the two roundings to 16
    bits, 2^-8 of the output and of the largest value, and 2^-12 of it for fp32 sums of 64 and 6 terms."""
    lens = [(i * i * 7 + i) % 7 for i in range(16000)]
    n = sum(lens)
    q, k, v = normal(5, n, 4, 64), normal(6, n, 2, 64), normal(7, n, 2, 64)
    cu = torch.tensor([0, *lens]).cumsum(0).to(torch.int32).to(DEV)
    lse = torch.full((n, 4), 7.0, device=DEV)
    out = qmm.qmm_attn_prompt(q, k, v, cu, lse=lse)
    (qp, at), (kp, _), (vp, _) = (padded(x, lens, 6) for x in (q, k, v))
    kd, vd = (x.double().repeat_interleave(2, 2) for x in (kp, vp))
    s = torch.einsum("nihd,njhd->nhij", qp.double(), kd) / 8
    s = s.masked_fill(torch.ones(6, 6, dtype=torch.bool, device=DEV).triu(1), -float("inf"))
    want = torch.einsum("nhij,njhd->nihd", s.softmax(-1), vd)[at]
    most = vd.abs().amax((1, 2), keepdim=True).expand(-1, 6, 4, -1)[at].amax(-1, keepdim=True)
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * most).all())
    assert float((lse.double() - s.logsumexp(-1).transpose(1, 2)[at]).abs().max()) <= 2.0 ** -12


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hq,hk,d", [(8, 4, 64), (8, 4, 128), (10, 2, 80)])
@pytest.mark.parametrize("lens,lk,causal", [
    ([(97 * i) % 411 for i in range(60)], None, True),                                # more than 32 sequences, 1-4 key tiles
    ([(61 * i) % 300 for i in range(45)], [(61 * i) % 300 + (i % 5) * 150 for i in range(45)], True),
    ([(61 * i) % 300 for i in range(45)], [(83 * i) % 700 for i in range(45)], False),
    ([1500, 900, 1300, 5, 0, 2100], None, True),                                      # up to 32: longest pieces first
    ([1500, 900, 1800, 1300, 2000], [2000, 3000, 100, 700, 1], False),
])
def test_pieces_that_follow_one_another(lens, lk, causal, hq, hk, d, dt):
    """More pieces of work than SMs, of one to 24 key tiles each and with one half or both, so that a
    CTA's later pieces start in the middle of the ring, on every parity."""
    lk = lens if lk is None else lk
    q, k, v = normal(8, sum(lens), hq, d).to(dt), normal(9, sum(lk), hk, d).to(dt), normal(10, sum(lk), hk, d).to(dt)
    cu_q, cu_k = (torch.tensor([0, *x]).cumsum(0).to(torch.int32).to(DEV) for x in (lens, lk))
    span = 2 * (128 // (hq // hk))
    pieces = sum((n + span - 1) // span for n in lens) * hk
    assert pieces > torch.cuda.get_device_properties(0).multi_processor_count
    lse = torch.full((sum(lens), hq), 7.0, device=DEV)
    out = qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k, causal=causal, lse=lse)
    check_prompt(q, k, v, lens, lk, causal, d ** -0.5, out, lse)
    again = [qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k, causal=causal) for _ in range(20)]
    assert all(torch.equal(x, out) for x in again)
