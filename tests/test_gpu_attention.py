"""The attention calls on the GPU against fp64 references, elementwise within bounds derived
from the formulas (attn_ref.py)."""
import math

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
from attn_ref import TINY, U, attend, check, check_decode, check_prompt, norm_rope

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qmm.build()
    qmm.lib()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def bounds(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)


# ------------------------------------------------------------------------------ norm and rotation
def check_rope(x, got, w, eps, pos, inv, interleaved, what):
    want, bound = norm_rope(x, w, eps, pos, inv, interleaved)
    check(got, want, bound + U[got.dtype] * (want.abs() + bound) + TINY[got.dtype], what)


@pytest.mark.parametrize("m,hq,hk,d,rot,interleaved,src,dst,norm", [
    (1, 32, 8, 128, 128, False, torch.float32, BF, True),
    (1, 1, 1, 8, 8, False, torch.float32, FP, True),
    (3, 5, 5, 40, 24, False, torch.float32, FP, True),      # partner lanes inside a group of 16
    (17, 28, 4, 80, 80, True, torch.float32, BF, True),
    (257, 12, 2, 64, 32, False, FP, FP, True),
    (5, 7, 1, 24, 16, True, BF, BF, True),
    (1000, 16, 16, 128, 64, False, BF, BF, False),          # rotation only
    (33, 16, 4, 96, 0, False, torch.float32, BF, True),     # norm only
    (9, 3, 3, 72, 72, False, BF, FP, False),
])
def test_norm_rope(m, hq, hk, d, rot, interleaved, src, dst, norm):
    g = gen(m + d)
    qkv = (normal(g, m, (hq + 2 * hk) * d) * 3).to(src)
    q, k, v = (x.view(m, -1, d) for x in qkv.split((hq * d, hk * d, hk * d), 1))
    pos = torch.randint(0, 100000, (m,), generator=g, device=DEV, dtype=torch.int32)
    inv = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV) / max(rot, 1))).float() if rot else None
    wq, wk = (1 + 0.2 * normal(g, d), 1 + 0.2 * normal(g, d)) if norm else (None, None)
    qo, ko, vo = qmm.qmm_qk_norm_rope(q, k, v, pos, inv, w_q=wq, w_k=wk, eps=1e-5, interleaved=interleaved,
                                      out_dtype=dst)
    check_rope(q, qo, wq, 1e-5, pos, inv, interleaved, "q")
    check_rope(k, ko, wk, 1e-5, pos, inv, interleaved, "k")
    assert torch.equal(vo, v.to(dst))


def test_norm_rope_far_positions_and_one_sided_norm():
    m, h, d = 6, 4, 64
    g = gen(1)
    q, k = normal(g, m, h, d), normal(g, m, h, d)
    pos = torch.tensor([2 ** 31 - 1, -1, -(2 ** 31), 0, 1234567891, 65537], dtype=torch.int32, device=DEV)
    inv = torch.linspace(1.0, 1e-4, d // 2, device=DEV)
    w = 1 + normal(g, d)
    qo, ko, vo = qmm.qmm_qk_norm_rope(q, k, None, pos, inv, w_q=w, w_k=None, out_dtype=FP)
    assert vo is None
    check_rope(q, qo, w, 1e-6, pos, inv, False, "q")
    check_rope(k, ko, None, 1e-6, pos, inv, False, "k")


def test_norm_rope_into_a_cache_and_in_place():
    """Outputs as strided views (the rows of one request in a [batch, room, heads, d] cache, and a
    heads-first layout); the rest of the buffers stays; in place gives the same bits."""
    m, hq, hk, d = 37, 6, 2, 64
    g = gen(2)
    q, k, v = (normal(g, m, h, d).to(BF) for h in (hq, hk, hk))
    pos = torch.arange(m, device=DEV, dtype=torch.int32)
    inv = torch.linspace(1.0, 1e-3, d // 2, device=DEV)
    w = 1 + normal(g, d)
    want = qmm.qmm_qk_norm_rope(q, k, v, pos, inv, w_q=w, w_k=w)
    cache = torch.full((2, 3, 64, hk, d), 7.0, dtype=BF, device=DEV)
    qo = torch.full((hq, m + 3, d), 7.0, dtype=BF, device=DEV)
    qmm.qmm_qk_norm_rope(q, k, v, pos, inv, w_q=w, w_k=w, q_out=qo.transpose(0, 1)[:m], k_out=cache[0, 1, 5:5 + m],
                         v_out=cache[1, 1, 5:5 + m])
    assert torch.equal(qo.transpose(0, 1)[:m], want[0])
    assert torch.equal(cache[0, 1, 5:5 + m], want[1]) and torch.equal(cache[1, 1, 5:5 + m], want[2])
    cache[:, 1, 5:5 + m] = 7.0
    assert bool((cache == 7.0).all()) and bool((qo[:, m:] == 7.0).all())
    qmm.qmm_qk_norm_rope(q, k, v, pos, inv, w_q=w, w_k=w, q_out=q, k_out=k, v_out=v)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, want[2])


def test_norm_rope_empty_and_zero_rows():
    e = torch.empty((0, 4, 64), device=DEV)
    inv = torch.ones(32, device=DEV)
    out = qmm.qmm_qk_norm_rope(e, e, e, torch.empty(0, dtype=torch.int32, device=DEV), inv)
    assert [tuple(x.shape) for x in out] == [(0, 4, 64)] * 3
    z = torch.zeros((2, 4, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    for x in qmm.qmm_qk_norm_rope(z, z, z, torch.ones(2, dtype=torch.int32, device=DEV), inv, w_q=w, w_k=w):
        assert not x.any()


# ------------------------------------------------------------------------------ packed prompts
def make_prompt(g, lq, lk, hq, hk, d, dt, spread=1.0):
    q, k, v = normal(g, sum(lq), hq, d), normal(g, sum(lk), hk, d), normal(g, sum(lk), hk, d)
    return (q * spread).to(dt), k.to(dt), v.to(dt)


@pytest.mark.parametrize("lq,lk,hq,hk,d,causal,dt", [
    ([1], None, 1, 1, 64, True, BF),
    ([1], [1], 4, 1, 8, False, FP),
    ([37], None, 32, 8, 128, True, BF),
    ([127, 128, 129], None, 4, 4, 64, True, FP),
    ([255, 257, 256], None, 2, 2, 128, True, BF),
    ([63, 64, 65, 1, 0, 33], None, 8, 2, 128, True, BF),          # an empty sequence between
    ([0, 0, 300, 0], None, 4, 2, 64, True, FP),
    ([700], None, 5, 1, 128, True, BF),                            # 5 heads of one kv head
    ([411, 90], None, 14, 2, 80, True, FP),                        # 7 heads of one kv head
    ([333], None, 6, 2, 96, True, BF),
    ([200, 5], None, 16, 1, 40, True, BF),
    ([50, 3], None, 128, 1, 64, True, FP),                         # as many heads of one kv head as allowed
    ([600, 130], None, 4, 2, 128, False, BF),
    ([100, 1, 65], [400, 777, 66], 8, 4, 128, True, BF),           # chunks after a history
    ([1, 1, 1], [1, 1000, 129], 32, 32, 64, True, FP),             # single tokens
    ([130, 40, 9], [10, 0, 8], 4, 2, 64, True, BF),                # rows that see no key, a sequence without keys
    ([130, 40], [10, 0], 4, 2, 128, False, FP),
    ([16, 16], [5000, 3], 4, 1, 128, True, BF),                    # a long key axis for few rows
    ([1100], None, 4, 2, 24, True, BF),
    ([1030, 1025], None, 2, 1, 128, True, FP),
])
def test_prompt(lq, lk, hq, hk, d, causal, dt):
    lk = lq if lk is None else lk
    g = gen(sum(lq) + d)
    q, k, v = make_prompt(g, lq, lk, hq, hk, d, dt)
    lse = torch.full((sum(lq), hq), 7.0, device=DEV)
    out = qmm.qmm_attn_prompt(q, k, v, bounds(lq), bounds(lk), causal=causal, lse=lse)
    check_prompt(q, k, v, lq, lk, causal, d ** -0.5, out, lse)


@pytest.mark.parametrize("lq,lk,hq,hk,d,causal,dt", [
    ([1], [8192], 8, 2, 128, True, BF),                 # one row over many keys
    ([37, 12], [5000, 900], 8, 1, 64, True, FP),        # sequences with more and with fewer key tiles than splits
    ([64], [2000], 4, 4, 128, False, BF),
    ([100, 0, 3], [3000, 2500, 2], 4, 2, 80, True, FP), # a sequence without queries, rows with hardly any key
    ([30, 20], [4000, 0], 4, 1, 128, True, BF),         # a sequence without keys
    ([500], [500 * 8 + 1], 8, 1, 64, True, BF),
])
def test_prompt_few_rows_many_keys(lq, lk, hq, hk, d, causal, dt):
    """Calls whose keys are split among SMs and joined: the workspace holds the parts."""
    assert qmm.qmm_workspace_bytes_attn_prompt(sum(lq), sum(lk), len(lq), hq, hk, d) > 256
    g = gen(sum(lk) + d)
    q, k, v = make_prompt(g, lq, lk, hq, hk, d, dt)
    lse = torch.full((sum(lq), hq), 7.0, device=DEV)
    out = qmm.qmm_attn_prompt(q, k, v, bounds(lq), bounds(lk), causal=causal, lse=lse)
    check_prompt(q, k, v, lq, lk, causal, d ** -0.5, out, lse)
    # the same bits again, with a workspace that holds NaN
    ws = torch.full((qmm.qmm_workspace_bytes_attn_prompt(sum(lq), sum(lk), len(lq), hq, hk, d),), 255,
                    dtype=torch.uint8, device=DEV)
    again = qmm.qmm_attn_prompt(q, k, v, bounds(lq), bounds(lk), causal=causal, workspace=ws)
    assert torch.equal(again, out) and qmm.qmm_read_device_status(ws) == 0


def test_prompt_few_rows_unseen_places():
    """Split keys: rows outside the sequences are not written, what a row does not see may be NaN."""
    hq, hk, d, dt = 4, 1, 64, BF
    g = gen(20)
    q, k, v = normal(g, 60, hq, d).to(dt), normal(g, 6000, hk, d).to(dt), normal(g, 6000, hk, d).to(dt)
    cu_q, cu_k = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([5, 25, 45], [100, 3000, 5800]))
    k[:100], v[:100], k[5800:], v[5800:], q[:5], q[45:] = (math.nan,) * 6
    k[3000 - 4:3000], v[3000 - 4:3000] = math.inf, math.nan  # the first sequence's last 4 keys: its last 4 rows see them
    assert qmm.qmm_workspace_bytes_attn_prompt(60, 6000, 2, hq, hk, d) > 256
    out = torch.full((60, hq, d), 7.0, dtype=dt, device=DEV)
    lse = torch.full((60, hq), 7.0, device=DEV)
    qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k, out=out, lse=lse)
    for x in (out, lse):
        assert bool((x[:5] == 7.0).all()) and bool((x[45:] == 7.0).all())
    check_prompt(q, k, v, [16], [2896], True, d ** -0.5, out, at_q=[5], at_k=[100])
    assert not torch.isfinite(out[21:25]).any()
    check_prompt(q, k, v, [20], [2800], True, d ** -0.5, out, lse, at_q=[25], at_k=[3000])


def test_prompt_many_short_sequences():
    lens = [(7 * i) % 11 for i in range(700)]
    g = gen(5)
    q, k, v = make_prompt(g, lens, lens, 2, 1, 64, BF)
    out = qmm.qmm_attn_prompt(q, k, v, bounds(lens))
    pad = torch.zeros((700, 11), dtype=torch.bool, device=DEV)
    for i, n in enumerate(lens):
        pad[i, :n] = True
    qp, kp, vp = (torch.zeros((700, 11, x.shape[1], 64), dtype=BF, device=DEV) for x in (q, k, v))
    qp[pad], kp[pad], vp[pad] = q, k, v
    op = torch.zeros_like(qp)
    op[pad] = out
    for i in range(0, 700, 37):
        check_prompt(qp[i, :lens[i]], kp[i, :lens[i]], vp[i, :lens[i]], [lens[i]], [lens[i]], True, 0.125,
                     op[i, :lens[i]])
    s = torch.einsum("nihd,njxd->nhij", qp.double(), kp.double()) * 0.125
    see = torch.ones(11, 11, dtype=torch.bool, device=DEV).tril() & pad[:, None, None, :]
    p = torch.where(see, s, torch.full_like(s, -1e30)).softmax(-1)
    want = torch.einsum("nhij,njxd->nihd", p, vp.double())
    assert float((op.double() - want)[pad].abs().max()) < 2 ** -6


@pytest.mark.parametrize("spread,scale", [(30.0, None), (1.0, -0.3), (1.0, 0.0), (8.0, 2.0)])
def test_prompt_sharp_and_other_scales(spread, scale):
    """Scores far apart (most weights vanish, the maximum moves late), a negative and a zero scale."""
    lens, d = [515, 130], 64
    g = gen(6)
    q, k, v = make_prompt(g, lens, lens, 4, 2, d, BF, spread)
    k[300] *= 4  # a late key that takes over rows that were settled
    out = qmm.qmm_attn_prompt(q, k, v, bounds(lens), scale=scale)
    check_prompt(q, k, v, lens, lens, True, d ** -0.5 if scale is None else scale, out)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_rising_maximum(d):
    """Scores that rise key by key, so that the running maximum moves at every tile."""
    n = 900
    q = torch.zeros((n, 2, d), dtype=FP, device=DEV)
    q[..., 0] = 8.0
    k = torch.zeros((n, 1, d), dtype=FP, device=DEV)
    k[:, 0, 0] = torch.arange(n, device=DEV) / 10
    v = normal(gen(7), n, 1, d).to(FP)
    for causal in (True, False):
        out = qmm.qmm_attn_prompt(q, k, v, bounds([n]), causal=causal, scale=1.0)
        check_prompt(q, k, v, [n], [n], causal, 1.0, out)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("g_", [1, 4])
def test_prompt_unseen_places_have_no_influence(bad, g_):
    """Rows outside the sequences and keys after a row's last one hold NaN or infinities; the
    buffers' rows outside the sequences are not written."""
    hk, d, dt = 2, 64, BF
    hq = hk * g_
    g = gen(8)
    q, k, v = (normal(g, 900, h, d).to(dt) for h in (hq, hk, hk))
    cu_q = torch.tensor([10, 210, 210, 500], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([30, 230, 300, 590], dtype=torch.int32, device=DEV)
    inside = torch.zeros(900, dtype=torch.bool, device=DEV)
    inside[30:590] = True
    k[~inside], v[~inside], q[:10], q[500:] = bad, bad, bad, bad
    out = torch.full((900, hq, d), 7.0, dtype=dt, device=DEV)
    qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k, out=out)
    check_prompt(q, k, v, [200, 0, 290], [200, 70, 290], True, d ** -0.5, out, at_q=[10, 210, 210], at_k=[30, 230, 300])
    assert bool((out[:10] == 7.0).all()) and bool((out[500:] == 7.0).all())
    # one late key of the first sequence, in its own diagonal tile: later rows see it, earlier ones do not
    k2, v2 = k.clone(), v.clone()
    v2[30 + 150, 0, 3] = bad
    k2[30 + 180, 1, 5] = bad
    out2 = qmm.qmm_attn_prompt(q, k2, v2, cu_q, cu_k, out=torch.full_like(out, 7.0))
    assert torch.equal(out2[10:160], out[10:160]) and torch.equal(out2[210:500], out[210:500])
    assert torch.equal(out2[10:190, g_:], out[10:190, g_:])
    seen = out2[160:210, :g_, 3]
    assert not torch.isfinite(seen).any()
    keep = [x for x in range(d) if x != 3]
    assert torch.equal(out2[10:210, :g_][..., keep], out[10:210, :g_][..., keep])
    if math.isnan(bad):
        assert out2[190:210, g_:].isnan().all()


def test_prompt_strides_streams_and_bits():
    """Heads-first q and out, k and v as slices of one wide buffer; another stream; the same bits twice,
    from a caller's workspace that holds garbage, and from a graph replay."""
    lens, hq, hk, d = [300, 77], 4, 2, 128
    n = sum(lens)
    g = gen(9)
    qs, kv = normal(g, hq, n, d).to(BF), normal(g, n, 3, hk, d).to(BF)
    q, k, v = qs.transpose(0, 1), kv[:, 0], kv[:, 2]
    cu = bounds(lens)
    first = qmm.qmm_attn_prompt(q, k, v, cu)
    check_prompt(q, k, v, lens, lens, True, d ** -0.5, first)
    out = torch.empty((hq, n, d), dtype=BF, device=DEV)
    ws = torch.full((qmm.qmm_workspace_bytes_attn_prompt(n, n, 2, hq, hk, d),), 255, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmm.qmm_attn_prompt(q, k, v, cu, out=out.transpose(0, 1), workspace=ws, stream=side)
    assert qmm.qmm_read_device_status(ws, stream=side) == 0
    side.synchronize()
    assert torch.equal(out.transpose(0, 1), first)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_attn_prompt(q, k, v, cu, out=out.transpose(0, 1), workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.transpose(0, 1), first)


def test_prompt_bounds_outside_the_buffers_are_clamped():
    g = gen(10)
    q, k, v = make_prompt(g, [100], [100], 2, 1, 64, BF)
    cu = torch.tensor([-5, 60, 1000], dtype=torch.int32, device=DEV)
    out = qmm.qmm_attn_prompt(q, k, v, cu)
    check_prompt(q, k, v, [60, 40], [60, 40], True, 0.125, out)
    # bounds that fall: no row is read or written outside the buffers
    cu = torch.tensor([50, 20, 100], dtype=torch.int32, device=DEV)
    out = qmm.qmm_attn_prompt(q, k, v, cu, out=torch.full_like(q, 7.0))
    check_prompt(q, k, v, [80], [80], True, 0.125, out, at_q=[20], at_k=[20])
    assert bool((out[:20] == 7.0).all())


def test_prompt_empty():
    e = torch.empty((0, 4, 64), dtype=BF, device=DEV)
    assert qmm.qmm_attn_prompt(e, e, e, bounds([0, 0])).shape == (0, 4, 64)
    q = torch.full((3, 4, 64), 7.0, dtype=BF, device=DEV)
    lse = torch.full((3, 4), 7.0, device=DEV)
    out = qmm.qmm_attn_prompt(q, e, e, bounds([2, 1]), bounds([0, 0]), lse=lse)  # queries without any key
    assert not out.any() and bool((lse == -math.inf).all())


# ------------------------------------------------------------------------------ decoding
def make_decode(g, b, room, p, hq, hk, d, dt):
    q = normal(g, b, hq, d).to(dt)
    k, v = (normal(g, b, room, hk, d).to(dt) for _ in range(2)) if room else (None, None)
    pk, pv = (normal(g, p, hk, d).to(dt) for _ in range(2)) if p else (None, None)
    return q, k, v, pk, pv


@pytest.mark.parametrize("b,room,p,hq,hk,d,dt", [
    (1, 1, 0, 1, 1, 8, FP),
    (1, 640, 0, 32, 8, 128, BF),
    (1, 5000, 0, 8, 1, 64, BF),          # one request with a long cache
    (3, 129, 0, 4, 4, 64, FP),
    (48, 300, 0, 8, 2, 128, BF),
    (5, 200, 0, 10, 2, 80, FP),          # 5 heads of one kv head
    (2, 100, 0, 28, 4, 96, BF),
    (3, 300, 0, 48, 2, 40, FP),          # 24 heads of one kv head
    (2, 70, 0, 128, 1, 64, BF),          # as many heads of one kv head as allowed
    (7, 130, 1001, 16, 16, 64, FP),
    (1, 16, 1, 4, 2, 128, BF),
    (33, 65, 700, 8, 2, 128, BF),
    (64, 40, 2049, 20, 4, 128, FP),
    (257, 3, 129, 8, 4, 64, BF),         # more requests than one tile's rows
    (130, 0, 555, 4, 2, 24, BF),         # the prefix alone
    (9, 5, 4000, 14, 2, 80, BF),
    (300, 20, 300, 2, 2, 128, FP),
])
def test_decode(b, room, p, hq, hk, d, dt):
    g = gen(b + p + d)
    q, k, v, pk, pv = make_decode(g, b, room, p, hq, hk, d, dt)
    lens = None
    if room:
        lens = torch.randint(0, room + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
        lens[0] = room
        lens[-1] = min(room, 1) if b == 1 or p == 0 else 0
    lse = torch.full((b, hq), 7.0, device=DEV)
    out = qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, lse=lse)
    check_decode(q, k, v, lens, pk, pv, d ** -0.5, out, lse)


@pytest.mark.parametrize("b,room,p,hq,hk,d,dt", [
    (16, 30, 2500, 32, 8, 128, BF),
    (5, 0, 16500, 8, 4, 64, FP),
    (70, 9, 4700, 10, 2, 40, BF),       # more requests than one tile's rows, 5 heads of one kv head
    (3, 200, 9001, 28, 4, 128, FP),
    (160, 66, 1000, 32, 2, 80, BF),
])
def test_decode_prefix_read_once(b, room, p, hq, hk, d, dt):
    """Prefixes about the size from which they go through the tensor-core phase (the workspace then
    holds its parts)."""
    assert (qmm.qmm_workspace_bytes_attn_decode(b, room, p, hq, hk, d) > 256) == (4 * b * hk * p * d > 80e6)
    g = gen(b + p)
    q, k, v, pk, pv = make_decode(g, b, room, p, hq, hk, d, dt)
    lens = torch.randint(0, room + 1, (b,), generator=g, device=DEV, dtype=torch.int32) if room else None
    lse = torch.full((b, hq), 7.0, device=DEV)
    out = qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, lse=lse)
    check_decode(q, k, v, lens, pk, pv, d ** -0.5, out, lse)
    ws = torch.full((qmm.qmm_workspace_bytes_attn_decode(b, room, p, hq, hk, d),), 255, dtype=torch.uint8, device=DEV)
    for scale in (None, -0.2):
        a, c = (qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, workspace=w, scale=scale) for w in (ws, None))
        assert torch.equal(a, c) and qmm.qmm_read_device_status(ws) == 0
        if scale is None:
            assert torch.equal(a, out)
    check_decode(q, k, v, lens, pk, pv, -0.2, a)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("p", [0, 200])
def test_decode_lengths_and_stale_rows(bad, p):
    """Lengths 0, 1, the whole room and outside of it; the rows from a length on hold NaN or infinities."""
    b, room, hq, hk, d, dt = 7, 150, 8, 2, 64, BF
    g = gen(11)
    q, k, v, pk, pv = make_decode(g, b, room, p, hq, hk, d, dt)
    lens = torch.tensor([0, 1, 150, 151, -3, 64, 129], dtype=torch.int32, device=DEV)
    for i, n in enumerate(lens.tolist()):
        k[i, max(n, 0):], v[i, max(n, 0):] = bad, bad
    lse = torch.empty((b, hq), device=DEV)
    out = qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, lse=lse)
    check_decode(q, k, v, lens, pk, pv, d ** -0.5, out, lse)
    if p == 0:
        assert not out[0].any() and not out[4].any() and bool((lse[0] == -math.inf).all())


@pytest.mark.parametrize("where", ["prefix", "cache"])
def test_decode_sharp(where):
    """Scores far apart between the prefix and the caches, either side negligible, and a rising maximum."""
    b, room, p, hq, hk, d, dt = 4, 300, 500, 4, 2, 128, FP
    g = gen(12)
    q, k, v, pk, pv = make_decode(g, b, room, p, hq, hk, d, dt)
    (pk if where == "prefix" else k).mul_(20)
    lens = torch.tensor([300, 17, 0, 256], dtype=torch.int32, device=DEV)
    out = qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, scale=0.3)
    check_decode(q, k, v, lens, pk, pv, 0.3, out)


def test_decode_strides_streams_and_bits():
    """A heads-first cache, a prefix inside a wider buffer, another stream, a graph, the same bits twice."""
    b, room, p, hq, hk, d = 5, 90, 300, 8, 2, 64
    g = gen(13)
    ks, vs = (normal(g, b, hk, room, d).to(BF) for _ in range(2))
    pkv = normal(g, p, 2, hk, d).to(BF)
    q = normal(g, b, 3, hq, d).to(BF)[:, 1]
    k, v, pk, pv = ks.transpose(1, 2), vs.transpose(1, 2), pkv[:, 0], pkv[:, 1]
    lens = torch.tensor([90, 0, 33, 64, 1], dtype=torch.int32, device=DEV)
    first = qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv)
    check_decode(q, k, v, lens, pk, pv, d ** -0.5, first)
    ws = torch.full((qmm.qmm_workspace_bytes_attn_decode(b, room, p, hq, hk, d),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((b, 2, hq, d), 7.0, dtype=BF, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, out=out[:, 0], workspace=ws, stream=side)
    assert qmm.qmm_read_device_status(ws, stream=side) == 0
    side.synchronize()
    assert torch.equal(out[:, 0], first) and bool((out[:, 1] == 7.0).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv, out=out[:, 0], workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:, 0], first)


def test_decode_offsets_past_32_bits():
    """The second request's cache starts more than 2^32 elements after the first one's."""
    room, hk, d = 70, 2, 64
    far = 2 ** 32 + 4096
    store = torch.empty(far + room * hk * d, dtype=FP, device=DEV)
    cache = store.as_strided((2, room, hk, d), (far, hk * d, d, 1))
    g = gen(14)
    cache.copy_(normal(g, 2, room, hk, d))
    q = normal(g, 2, 4, d).to(FP)
    lens = torch.tensor([70, 41], dtype=torch.int32, device=DEV)
    out = qmm.qmm_attn_decode(q, cache, cache, lens)
    check_decode(q, cache, cache, lens, None, None, d ** -0.5, out)
    # and tokens 2^26 elements apart: the last rows of a prefix lie past 2^32 elements
    del cache
    pre = store.as_strided((65, hk, d), (2 ** 26, d, 1))
    pre.copy_(normal(g, 65, hk, d))
    out = qmm.qmm_attn_decode(q, None, None, None, prefix_k=pre, prefix_v=pre)
    check_decode(q, None, None, None, pre, pre, d ** -0.5, out)
    cu = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    cu_k = torch.tensor([0, 65], dtype=torch.int32, device=DEV)
    out = qmm.qmm_attn_prompt(q, pre, pre, cu, cu_k)
    check_prompt(q, pre, pre, [2], [65], True, d ** -0.5, out)


def test_decode_agrees_with_prompt():
    """A decode step is the last row of a prompt call over prefix and cache put together."""
    b, p, hq, hk, d = 3, 400, 8, 2, 128
    g = gen(15)
    q, k, v, pk, pv = make_decode(g, b, 60, p, hq, hk, d, BF)
    lens = torch.tensor([60, 7, 31], dtype=torch.int32, device=DEV)
    out = qmm.qmm_attn_decode(q, k, v, lens, prefix_k=pk, prefix_v=pv)
    kk = torch.cat([torch.cat((pk, k[i, :n])) for i, n in enumerate(lens.tolist())])
    vv = torch.cat([torch.cat((pv, v[i, :n])) for i, n in enumerate(lens.tolist())])
    cu_k = bounds([p + n for n in lens.tolist()])
    other = qmm.qmm_attn_prompt(q, kk, vv, bounds([1] * b), cu_k)
    for i, n in enumerate(lens.tolist()):
        a = int(cu_k[i])
        for h in range(hq):
            o, bd, _, _ = attend(q[i:i + 1, h], kk[a:a + p + n, h // 4], vv[a:a + p + n, h // 4], d ** -0.5)
            check(out[i:i + 1, h], o, bd, "decode")
            check(other[i:i + 1, h], o, bd, "prompt")


def test_decode_empty_batch():
    e = torch.empty((0, 4, 64), dtype=BF, device=DEV)
    c = torch.empty((0, 8, 4, 64), dtype=BF, device=DEV)
    lens = torch.empty(0, dtype=torch.int32, device=DEV)
    assert qmm.qmm_attn_decode(e, c, c, lens).shape == (0, 4, 64)


# ------------------------------------------------------------------------------ the binding's refusals
def test_binding_refuses():
    q = torch.zeros((4, 4, 64), dtype=BF, device=DEV)
    cu = bounds([4])
    lens = torch.zeros(4, dtype=torch.int32, device=DEV)
    cache = torch.zeros((4, 8, 2, 64), dtype=BF, device=DEV)
    f32 = q.float()
    bad = [
        (3, lambda: qmm.qmm_attn_prompt(f32, f32, f32, cu)),
        (3, lambda: qmm.qmm_attn_prompt(q, q, q.half(), cu)),
        (3, lambda: qmm.qmm_attn_prompt(q, q, q, cu.long())),
        (1, lambda: qmm.qmm_attn_prompt(q.cpu(), q, q, cu)),
        (1, lambda: qmm.qmm_attn_prompt(q, q, q.transpose(1, 2).contiguous().transpose(1, 2), cu)),
        (2, lambda: qmm.qmm_attn_prompt(q, q[:, :3], q[:, :3], cu)),               # 4 heads on 3
        (2, lambda: qmm.qmm_attn_prompt(q, q, q[:3], cu)),
        (2, lambda: qmm.qmm_attn_prompt(q[..., :60], q[..., :60], q[..., :60], cu)),  # head size 60
        (4, lambda: qmm.qmm_attn_prompt(q.view(-1)[4:4 + 3 * 256].view(3, 4, 64), q, q, cu)),
        (1, lambda: qmm.qmm_attn_prompt(q, q, q, cu, scale=float("nan"))),
        (5, lambda: qmm.qmm_attn_prompt(q, q, q, cu, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))),
        (2, lambda: qmm.qmm_attn_prompt(q, q, q, cu, lse=torch.zeros(3, device=DEV))),
        (2, lambda: qmm.qmm_attn_prompt(q, q, q, cu, torch.zeros(5, dtype=torch.int32, device=DEV))),
        (3, lambda: qmm.qmm_attn_decode(f32, cache, cache, lens)),
        (2, lambda: qmm.qmm_attn_decode(q, cache[:3], cache[:3], lens)),
        (2, lambda: qmm.qmm_attn_decode(q, None, None, None)),
        (2, lambda: qmm.qmm_attn_decode(q, cache, cache, lens[:3])),
        (1, lambda: qmm.qmm_attn_decode(q, cache, cache, None)),
        (3, lambda: qmm.qmm_qk_norm_rope(q, q.half(), q, lens, torch.ones(32, device=DEV))),
        (3, lambda: qmm.qmm_qk_norm_rope(q, q, q, lens, torch.ones(32, device=DEV), out_dtype=torch.float32)),
        (2, lambda: qmm.qmm_qk_norm_rope(q, q, q, lens, torch.ones(36, device=DEV))),  # rotates 72 of 64
        (2, lambda: qmm.qmm_qk_norm_rope(q, q, q, lens, torch.ones(2, device=DEV))),   # rotates 4
        (1, lambda: qmm.qmm_qk_norm_rope(q, q, q, None, torch.ones(32, device=DEV))),
        (2, lambda: qmm.qmm_qk_norm_rope(q, q, q, lens, torch.ones(32, device=DEV), w_q=torch.ones(63, device=DEV))),
    ]
    for i, (code, call) in enumerate(bad):
        with pytest.raises(qmm.QMMError) as e:
            call()
        assert e.value.code == code, (i, str(e.value))
