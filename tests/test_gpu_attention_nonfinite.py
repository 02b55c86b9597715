"""Rows that see infinities and NaN, element for element: an element is the sum of the non-finite values
that its row sees (infinities of both signs give NaN), a row that sees a NaN key is NaN, and every
other element keeps the bound of attn_ref.  Where the reference is not finite nothing but the same
infinity, or NaN, passes."""
import math

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
from attn_ref import attend, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qmm.build()


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def strict(got, want, bound, what):
    fin = torch.isfinite(want)
    g = got.double()
    same = (g == want) | (g.isnan() & want.isnan())
    wrong = ~fin & ~same
    assert not wrong.any(), (f"{what}: {int(wrong.sum())} non-finite elements differ, first at {wrong.nonzero()[0].tolist()}: "
                             f"got {g[wrong][0].item()} want {want[wrong][0].item()}")
    zero = torch.zeros_like(want)
    check(torch.where(fin, g, zero), torch.where(fin, want, zero), torch.where(fin, bound, zero), what)


def test_strict_refuses_what_it_should():
    w = torch.tensor([INF, -INF, NAN, 1.0], dtype=torch.float64)
    b = torch.tensor([INF, INF, NAN, 0.1], dtype=torch.float64)
    strict(w.clone(), w, b, "same")
    for i, x in ((0, 0.0), (0, -INF), (0, NAN), (1, INF), (2, 1.0), (2, INF), (3, 1.2), (3, NAN)):
        g = w.clone()
        g[i] = x
        with pytest.raises(AssertionError):
            strict(g, w, b, "differs")


def check_rows(q, k, v, lq, lk, causal, out, at_q=0, at_k=0):
    g = q.shape[1] // k.shape[1]
    hidden = torch.ones(lq, lk, dtype=torch.bool, device=DEV).triu(lk - lq + 1) if causal else None
    for h in range(q.shape[1]):
        a, b = slice(at_q, at_q + lq), slice(at_k, at_k + lk)
        o, bound, _, _ = attend(q[a, h], k[b, h // g], v[b, h // g], q.shape[2] ** -0.5, hidden)
        strict(out[a, h], o, bound, f"head {h}")


def bounds(*lens):
    return torch.tensor([0, *lens]).cumsum(0).to(torch.int32).to(DEV)


def plant(k, v, at, d):
    """Non-finite values in head 0 around the keys of `at` (early, middle, late): one element each for a sole
    infinity, both signs at the same key distance, an infinity before and after the other sign, and NaN."""
    early, mid, late = at
    v[late, 0, 0] = INF
    v[late, 0, 1] = -INF
    v[late, 0, 2] = NAN
    v[mid, 0, 3], v[late, 0, 3] = INF, -INF       # both signs, both late
    v[early, 0, 4], v[late, 0, 4] = INF, -INF     # the first in a tile that every row sees
    v[early, 0, 5], v[late, 0, 5] = NAN, INF      # a NaN before an infinity
    v[early, 0, d - 1], v[mid, 0, d - 1] = -INF, -INF
    v[mid, 0, 6] = INF


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("lq,lk,hq,hk,causal", [
    (200, 200, 4, 2, True),
    (300, 700, 2, 2, True),        # two halves, six key tiles
    (600, 600, 8, 1, True),        # several pieces, each with its own diagonal tile
    (150, 333, 4, 2, False),
    (20, 3000, 4, 1, True),        # split keys
])
def test_prompt_rows_that_see_them(lq, lk, hq, hk, causal, d, dt):
    g = torch.Generator(device=DEV).manual_seed(lq + d)
    q, k, v = (normal(g, n, h, d).to(dt) for n, h in ((lq, hq), (lk, hk), (lk, hk)))
    plant(k, v, (min(5, lk - lq), lk - lq // 2 - 1, lk - max(lq // 4, 2)), d)
    out = qmm.qmm_attn_prompt(q, k, v, bounds(lq), bounds(lk), causal=causal)
    check_rows(q, k, v, lq, lk, causal, out)
    # a NaN key before a late infinity: the rows that see it are NaN as a whole
    k[max(lk - lq, 0) + lq // 3, 0, 7] = NAN
    out = qmm.qmm_attn_prompt(q, k, v, bounds(lq), bounds(lk), causal=causal)
    check_rows(q, k, v, lq, lk, causal, out)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b,room,p", [(3, 200, 0), (3, 200, 300), (40, 70, 9000)])  # caches; inline; read once
def test_decode_rows_that_see_them(b, room, p, d, dt):
    hq, hk = 8, 4
    g = torch.Generator(device=DEV).manual_seed(b + d)
    q = normal(g, b, hq, d).to(dt)
    k, v = (normal(g, b, room, hk, d).to(dt) for _ in range(2))
    pk, pv = (normal(g, p, hk, d).to(dt) for _ in range(2)) if p else (None, None)
    lens = torch.randint(40, room + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
    v[0, 3, 0, 0], v[0, 39, 0, 1], v[0, 20, 0, 2] = INF, -INF, NAN
    v[1, 2, 1, 3], v[1, 30, 1, 3] = INF, -INF
    k[2, 17, 3, 5] = NAN
    if p:
        pv[p // 2, 2, d - 1] = INF
        v[0, 9, 2, d - 1] = -INF
    out = qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv)
    for i, n in enumerate(lens.tolist()):
        kk, vv = (k[i, :n], v[i, :n]) if not p else (torch.cat((pk, k[i, :n])), torch.cat((pv, v[i, :n])))
        for h in range(hq):
            o, bound, _, _ = attend(q[i:i + 1, h], kk[:, h // 2], vv[:, h // 2], d ** -0.5)
            strict(out[i:i + 1, h], o, bound, f"request {i} head {h}")
