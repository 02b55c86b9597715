"""Decoding over pages with values of any size: the error follows the values' size.

The bound, with u the output's unit, v_j = d_j code_j and p normalised, per element:
  * the output is rounded once: u |out|;
  * the weight p 2^x is rounded to fp16 (bf16 heads) and so is its product with the value scale, w = 2 2^-11;
    f16 heads the product alone, w = 2^-11, of the weight's two halves;
  * x is 15 as long as the scales are below 2, else 15 - E for scales from 2^E on, so 2^-x is at most
    r = 2^-15 max(1, max |d|).  Below fp16's normal range a rounding is off by 2^-25: of the weight (times d code), of
    the product (times code), for f16 heads of two products: 2^-24 r sum_j (|v_j| + |code_j|) / sum_j exp(s_j - max);
  * codes enter with their bias, which comes off in the same fp32 sums: the two products of 16 keys are each
    rounded at 2^-23 of at most sum p |d| (15 + 8) or (255 + 128), together 2^-22 of it.  The codes are fp16 subnormals, code
    2^-24, and the matrix unit lines its products up as if they began at the smallest normal, 2^-14, keeping 25 bits
    below that: a product of 16 keys is off by 2^-25 2^-14 / 2^-24 = 2^-15 of the largest p |d| among them, the two by
    2^-14, over all keys at most 2^-14 sum p |d| (three tokens whose first has the code 0 and all the weight
    but 1e-4 come out as multiples of 2^-17 where their scale is 0.35: 2^-26 of 2^-24 times 2^15);
  * scores, exponentials and sums in fp32 as in kv_ref.check_decode_kv: (2 ds + (64 + n^(1/2)) 2^-23) A, A = sum_j p_j |v_j|.
"""
import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
import kv_ref
from attn_ref import TINY, U, check
from test_gpu_kv import BF, DEV, FP, _errors, _lib, filled, gen, ints, normal, query  # noqa: F401

pytestmark = pytest.mark.gpu


def check_values(q, codes, scales, lens, qtype, out):
    d = q.shape[-1]
    w = 2.0 ** -10 if q.dtype == BF else 2.0 ** -11
    wide = 23 if qtype == "q4_0" else 383
    g = q.shape[1] // codes[0][0].shape[1]
    for b in sorted({*range(min(len(lens), 6)), len(lens) - 1}):
        n = lens[b]
        for h in range(codes[0][b].shape[1]):
            heads = slice(h * g, (h + 1) * g)
            k, v = (kv_ref.values(c[b][:n, h], s[b][:n, h]) for c, s in zip(codes, scales))
            kd, vd = (s[b][:n, h].double().abs() for s in scales)
            qd = q[b, heads].double()
            s = qd @ k.t() * d ** -0.5
            reach = qd.abs().unflatten(-1, (-1, 32)).sum(-1) @ kd.t() * wide * d ** -0.5
            ds = ((d + 5) * 2.0 ** -23 * (reach + s.abs())).amax(1, keepdim=True)
            p = torch.exp(s - s.amax(1, keepdim=True))
            total = p.sum(1, keepdim=True)
            p = p / total
            want, A = p @ v, p @ v.abs()
            r = 2.0 ** -15 * max(1.0, float(vd.max()))
            lost = 2.0 ** -24 * r * (v.abs().sum(0) + codes[1][b][:n, h].double().abs().sum(0)) / total
            bias = (2.0 ** -14 + 2.0 ** -22 * wide) * (p @ vd.repeat_interleave(32, -1))
            bound = U[q.dtype] * want.abs() + A * (w + 2 * ds + (64 + n ** 0.5) * 2.0 ** -23) + TINY[q.dtype] + lost + bias
            check(out[b, heads], want, bound, f"request {b} kv head {h}")


def with_values(cache, table, lens, qtype, page, codes, scales, make):
    """Other values in the same places: make(n, hk, d)."""
    for i, n in enumerate(lens):
        _, hk, d = codes[1][i].shape
        codes[1][i], scales[1][i] = kv_ref.quantize(qtype, make(n, hk, d))
        j = torch.arange(n, device=DEV)
        kv_ref.store(cache.pages, qtype, page, hk, d, table[i].long()[j // page] * page + j % page,
                     [c[i] for c in codes], [s[i] for s in scales])


FORMS = [  # lens, most, query heads, kv heads, head size, page
    ([1000, 33], 1000, 8, 2, 128, 16),                      # clusters
    ([3] * 3 + [60] * 150, 60, 8, 4, 64, 32),               # a warp each
    ([20000, 300], 20000, 8, 1, 96, 64),                    # parts in the workspace
]


@pytest.mark.parametrize("qtype,dt", [("q4_0", BF), ("q4_0", FP), ("q8_0", BF), ("q8_0", FP)])
@pytest.mark.parametrize("size", [1.0, 2e-2, 5e-3, 1e-3, 1e-4, 1e-6, 300.0, 2e4])
@pytest.mark.parametrize("lens,most,hq,hk,d,page", FORMS)
def test_sizes(lens, most, hq, hk, d, page, size, qtype, dt):
    """Values of one size; the first token is one that all heads look at more than at others."""
    if dt == FP:
        size = min(size, 5000.0)  # outputs in fp16's range
    g = gen(sum(lens) + d)
    cache, table, codes, scales = filled(g, lens, qtype, page, hk, d)
    with_values(cache, table, lens, qtype, page, codes, scales, lambda *n: normal(g, *n) * size)
    q = query(g, len(lens), hq, d, dt)
    first = kv_ref.values(codes[0][0][0], scales[0][0][0])  # of the first request, a direction for each kv head
    q[0] += (first / first.pow(2).sum(-1, keepdim=True) * (9 * d ** 0.5)).repeat_interleave(hq // hk, 0).to(dt)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=most)
    check_values(q, codes, scales, lens, qtype, out)
    assert torch.equal(qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=most), out)


@pytest.mark.parametrize("qtype,dt", [("q4_0", BF), ("q4_0", FP), ("q8_0", BF), ("q8_0", FP)])
@pytest.mark.parametrize("lens,most,hq,hk,d,page", FORMS + [([257], 257, 8, 1, 32, 16), ([500], 500, 18, 2, 64, 16)])
@pytest.mark.parametrize("order", [1, -1, 0])
def test_sizes_that_change_along_a_request(lens, most, hq, hk, d, page, order, qtype, dt):
    """Sizes over 2^-20 to 2^12 that rise along the tokens, fall, or come in any order; a block of 32 without values, and
    an element that is zero in every token."""
    g = gen(sum(lens) + d + 1)
    cache, table, codes, scales = filled(g, lens, qtype, page, hk, d)

    def make(n, hk, d):
        e = torch.linspace(-20, 12, n, device=DEV)
        e = e if order > 0 else e.flip(0) if order < 0 else e[torch.randperm(n, generator=g, device=DEV)]
        v = normal(g, n, hk, d) * e.exp2()[:, None, None]
        v[..., 5] = 0
        v[1::3, :, :32] = 0
        return v

    with_values(cache, table, lens, qtype, page, codes, scales, make)
    q = query(g, len(lens), hq, d, dt)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=most)
    check_values(q, codes, scales, lens, qtype, out)


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
def test_the_largest_scales(qtype):
    """Scales of 65504, of one sign and of both, and a page that is gone between them."""
    n, hq, hk, d, page = 200, 8, 1, 64, 16
    g = gen(9)
    cache, table, codes, scales = filled(g, [n], qtype, page, hk, d)
    with_values(cache, table, [n], qtype, page, codes, scales, lambda *s: normal(g, *s) * 1e7)
    assert float(scales[1][0].abs().max()) == 65504
    q = query(g, 1, hq, d, BF)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints([n]), max_len=n)
    check_values(q, codes, scales, [n], qtype, out)
    table[0, 3] = -1
    keep = torch.arange(n, device=DEV) // page != 3
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints([n]), max_len=n)
    check_values(q, [[c[0][keep]] for c in codes], [[s[0][keep]] for s in scales], [int(keep.sum())], qtype, out)
