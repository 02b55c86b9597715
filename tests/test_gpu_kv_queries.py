"""Decoding over pages with queries at the ends of their type: very large ones, infinities and NaN."""
import math

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
import kv_ref
from attn_ref import U, check
from test_gpu_kv import BF, DEV, FP, _errors, _lib, filled, gen, ints, query  # noqa: F401

pytestmark = pytest.mark.gpu
FORMS = [  # lens, most, query heads, kv heads, head size, page
    ([700, 40], 700, 8, 2, 128, 16),                        # clusters
    ([31] * 30, 31, 4, 2, 64, 32),                          # a warp each
    ([20000], 20000, 8, 1, 64, 64),                         # parts in the workspace
]


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
@pytest.mark.parametrize("dt,power,kpower,scale", [
    (BF, 100, 0, None), (BF, 115, 0, None), (BF, 117, -8, None), (BF, 120, -10, -0.125), (BF, 124, -12, None),
    (BF, 110, 3, 2.0), (BF, 20, 0, None), (FP, 13, 6, None), (FP, 13, 0, 1e30),
])
@pytest.mark.parametrize("lens,most,hq,hk,d,page", FORMS)
def test_scores_so_far_apart_that_one_key_counts(lens, most, hq, hk, d, page, dt, power, kpower, scale, qtype):
    """Finite scores up to fp32's range: the output is the value of the key with the largest, where it leads by more
    than a score's error and the 2^7 that make the others' weights vanish."""
    g = gen(power + d)
    cache, table, codes, scales = filled(g, lens, qtype, page, hk, d, 2.0 ** kpower)
    q = query(g, len(lens), hq, d, dt, 2.0 ** power)
    assert bool(torch.isfinite(q).all())
    lse = torch.zeros(len(lens), hq, device=DEV)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=most, scale=scale, lse=lse)
    scale, counted = d ** -0.5 if scale is None else scale, 0
    for b, n in enumerate(lens):
        for h in range(hq):
            kh = h // (hq // hk)
            k, v = (kv_ref.values(c[b][:, kh], s[b][:, kh]) for c, s in zip(codes, scales))
            s = k @ q[b, h].double() * scale
            assert float(s.abs().max()) < 2.0 ** 127
            reach = scales[0][b][:, kh].double().abs() @ q[b, h].double().abs().unflatten(-1, (-1, 32)).sum(-1)
            ds = float((reach * (abs(scale) * (23 if qtype == "q4_0" else 383) * (d + 5) * 2.0 ** -23)).max())
            top = s.topk(2)
            if float(top.values[0] - top.values[1]) < 4 * ds + 128:
                continue
            counted += 1
            want = v[top.indices[0]]
            check(out[b, h], want, want.abs() * (U[dt] + 2.0 ** -10), f"request {b} head {h}")
            check(lse[b, h], top.values[0], torch.tensor(2 * ds, device=DEV, dtype=torch.float64), f"lse of request {b} head {h}")
    assert counted >= len(lens) * hq // 2


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("lens,most,hq,hk,d,page", FORMS)
def test_infinities_and_nan_stay_in_their_head(lens, most, hq, hk, d, page, value, dt):
    """An infinite or NaN element makes every score of its head NaN or infinite of either sign, so its row NaN; a
    request without tokens gives zeros all the same, and the other heads keep their bits."""
    lens = list(lens)
    if len(lens) > 1:
        lens[-1] = 0
    g = gen(3)
    cache, table, _, _ = filled(g, lens, "q4_0", page, hk, d)
    q = query(g, len(lens), hq, d, dt)
    plain = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=most)
    q[:, 1, 7] = value
    lse = torch.zeros(len(lens), hq, device=DEV)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=most, lse=lse)
    some = ints(lens) > 0
    assert bool(out[some, 1].isnan().all()) and bool(lse[some, 1].isnan().all())
    assert not out[~some].any() and bool((lse[~some] == -math.inf).all())
    others = [h for h in range(hq) if h != 1]
    assert torch.equal(out[:, others], plain[:, others]) and bool(torch.isfinite(lse[some][:, others]).all())
