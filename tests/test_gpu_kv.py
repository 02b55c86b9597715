"""The paged key/value cache on the GPU: appending, reading back and decoding against the references of
kv_ref.py, and the calls one after another as a layer uses them."""
import math

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
import kv_ref
from attn_ref import U, check, check_prompt, norm_rope

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
QMM_ERR_IDS, QMM_ERR_DEVICE = 7, 8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qmm.build()
    qmm.lib()


@pytest.fixture(autouse=True)
def _errors():
    qmm.qmm_take_attn_error()
    yield
    qmm.qmm_set_test_fault(0)
    qmm.qmm_take_attn_error()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cache_of(n, qtype, page, hk, d, fill=255):
    """A cache whose unwritten places are NaN scales and the largest codes."""
    pages = torch.full((n, kv_ref.page_bytes(qtype, page, hk, d)), fill, dtype=torch.uint8, device=DEV)
    return qmm.KVPages(pages, qtype, page, hk, d)


# ------------------------------------------------------------------------------ appending
@pytest.mark.parametrize("m,hq,hk,d,rot,interleaved,src,dst,norm,qtype,page", [
    (1, 32, 8, 128, 128, False, F32, BF, True, "q4_0", 16),
    (1, 1, 1, 32, 32, False, F32, FP, True, "q8_0", 16),
    (1, 4, 2, 64, 64, True, BF, BF, True, "q4_0", 256),
    (77, 28, 4, 128, 64, True, FP, FP, True, "q8_0", 32),
    (33, 6, 6, 96, 48, False, F32, BF, True, "q4_0", 16),       # partners inside a block of 32 and across
    (50, 12, 2, 96, 96, False, BF, FP, True, "q8_0", 64),
    (1300, 3, 1, 64, 32, False, F32, BF, True, "q4_0", 128),    # whole tokens a block
    (700, 16, 16, 32, 24, False, F32, FP, False, "q4_0", 32),
    (40, 5, 5, 128, 0, False, FP, FP, True, "q4_0", 64),
    (129, 8, 1, 64, 64, True, F32, FP, True, "q4_0", 16),
])
def test_append(m, hq, hk, d, rot, interleaved, src, dst, norm, qtype, page):
    g = gen(m + d)
    qkv = (normal(g, m, (hq + 2 * hk) * d) * 3).to(src)
    q, k, v = (x.view(m, -1, d) for x in qkv.split((hq * d, hk * d, hk * d), 1))
    pos = torch.randint(0, 100000, (m,), generator=g, device=DEV, dtype=torch.int32)
    inv = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV) / max(rot, 1))).float() if rot else None
    wq, wk = (1 + 0.2 * normal(g, d), 1 + 0.2 * normal(g, d)) if norm else (None, None)
    n = m // page + 3
    cache = cache_of(n, qtype, page, hk, d, 0xA5)
    slots = torch.randperm(n * page, generator=g, device=DEV)[:m].to(torch.int32)
    qo, ko, vo = qmm.qmm_kv_append(q, k, v, pos, inv, cache, slots, w_q=wq, w_k=wk, eps=1e-5, interleaved=interleaved,
                                   out_dtype=dst, values=True)
    want, bound = norm_rope(q, wq, 1e-5, pos, inv, interleaved)
    check(qo, want, bound + U[dst] * (want.abs() + bound) + 2.0 ** -25, "q")
    codes, scales = kv_ref.load(cache.pages, qtype, page, hk, d, slots)
    # values are quantized from what was given: the same bits as the reference
    vc, vs = kv_ref.quantize(qtype, v.float())
    assert torch.equal(codes[1], vc) and torch.equal(scales[1], vs)
    # keys: the scale of the turned head, and the nearest code to it, within the turn's bound
    x, bx = norm_rope(k, wk, 1e-5, pos, inv, interleaved)
    x, bx = x.unflatten(-1, (-1, 32)), bx.unflatten(-1, (-1, 32))
    most, off = x.abs().amax(-1), bx.amax(-1)
    steps = 8 if qtype == "q4_0" else 127
    got = scales[0].double()
    check(got.abs(), most / steps, off / steps + 2.0 ** -11 * 1.001 * (most + off) / steps + 2.0 ** -25, "scale of k")
    c = codes[0].double().unflatten(-1, (-1, 32))
    lo, hi = (-8, 7) if qtype == "q4_0" else (-127, 127)
    best = x / got[..., None]
    slack = bx / got.abs()[..., None]
    near = (c - best).abs() <= 0.5 + slack + 2.0 ** -20
    clamped = ((c == hi) & (best + slack >= hi)) | ((c == lo) & (best - slack <= lo))
    assert bool((near | clamped).all())
    # what the call says the cache stands for, and what reading it says
    for out, cc, ss in ((ko, codes[0], scales[0]), (vo, codes[1], scales[1])):
        assert torch.equal(out, kv_ref.values(cc, ss).float().to(dst))
    # no other byte
    before = torch.full_like(cache.pages, 0xA5)
    kv_ref.store(before, qtype, page, hk, d, slots, codes, scales)
    assert torch.equal(before, cache.pages)
    # without q, without the values: the same bytes
    again = cache_of(n, qtype, page, hk, d, 0xA5)
    none = qmm.qmm_kv_append(None, k, v, pos, inv, again, slots, w_k=wk, eps=1e-5, interleaved=interleaved, out_dtype=dst)
    assert none == (None, None, None) and torch.equal(again.pages, cache.pages)


def test_append_matches_norm_rope_in_bits():
    """Queries are those of qmm_qk_norm_rope, and so are keys that are quantized after it changed nothing."""
    g = gen(3)
    q, k, v = normal(g, 21, 8, 128), normal(g, 21, 2, 128), normal(g, 21, 2, 128)
    pos, inv = torch.arange(21, device=DEV, dtype=torch.int32), torch.linspace(1, 1e-3, 64, device=DEV)
    w = 1 + 0.1 * normal(g, 128)
    cache = cache_of(4, "q4_0", 16, 2, 128)
    qo, _, _ = qmm.qmm_kv_append(q, k, v, pos, inv, cache, torch.arange(21, device=DEV, dtype=torch.int32), w_q=w, w_k=w)
    assert torch.equal(qo, qmm.qmm_qk_norm_rope(q, k, v, pos, inv, w_q=w, w_k=w)[0])


def test_append_slots_outside_and_padding():
    """A slot that is no place of the cache (padding) writes nothing; its query and values come all the same."""
    g = gen(4)
    m, hk, d = 9, 2, 64
    q, k, v = normal(g, m, 4, d), normal(g, m, hk, d), normal(g, m, hk, d)
    cache = cache_of(2, "q4_0", 16, hk, d, 7)
    slots = ints([3, -1, 31, 32, 2 ** 31 - 1, -(2 ** 31), 0, -1, 17])
    qo, ko, vo = qmm.qmm_kv_append(q, k, v, None, None, cache, slots, values=True)
    kc, ks = kv_ref.quantize("q4_0", k)
    vc, vs = kv_ref.quantize("q4_0", v)
    assert torch.equal(ko, kv_ref.values(kc, ks).float().to(BF)) and torch.equal(vo, kv_ref.values(vc, vs).float().to(BF))
    assert torch.equal(qo, q.to(BF))
    want = torch.full_like(cache.pages, 7)
    ok = ((slots >= 0) & (slots < 32)).nonzero().flatten()
    kv_ref.store(want, "q4_0", 16, hk, d, slots[ok], [kc[ok], vc[ok]], [ks[ok], vs[ok]])
    assert torch.equal(cache.pages, want)
    assert qmm.qmm_take_attn_error() == 0


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
@pytest.mark.parametrize("src", [F32, BF, FP])
def test_append_extremes(qtype, src):
    """Zeros, ties of the two signs, values half way between codes, tiny and huge blocks, NaN and infinities."""
    big = 60000.0 if src == FP else 3e38
    rows = torch.zeros(12, 1, 32, device=DEV)
    rows[1, 0, 5], rows[1, 0, 9] = 4.0, -4.0               # the positive one of two
    rows[2, 0] = torch.arange(32, device=DEV) / 4 - 4.0     # half way between codes
    rows[3, 0] = -rows[2, 0]
    rows[4, 0, :4] = torch.tensor([1e-7, -3e-8, 6e-8, 0], device=DEV)
    rows[5, 0, :4] = torch.tensor([3e-5, -1e-5, 2e-5, 0], device=DEV)
    rows[6, 0, :4] = torch.tensor([big, -big / 2, 1.0, -0.0], device=DEV)
    rows[7, 0, :4] = torch.tensor([-big, big / 2, 1.0, -0.0], device=DEV)
    rows[8, 0, :3] = torch.tensor([math.nan, 2.0, -1.0], device=DEV)
    rows[9, 0, :3] = torch.tensor([math.inf, 2.0, -1.0], device=DEV)
    rows[10, 0, :3] = torch.tensor([-math.inf, math.inf, math.nan], device=DEV)
    rows[11, 0] = math.nan
    x = rows.to(src)
    cache = cache_of(1, qtype, 16, 1, 32)
    slots = torch.arange(12, device=DEV, dtype=torch.int32)
    _, ko, vo = qmm.qmm_kv_append(None, x, x, None, None, cache, slots, out_dtype=BF, values=True)
    codes, scales = kv_ref.load(cache.pages, qtype, 16, 1, 32, slots)
    c, s = kv_ref.quantize(qtype, x.float())
    for i in range(2):
        assert torch.equal(codes[i], c) and torch.equal(scales[i], s)
    assert torch.equal(ko, kv_ref.values(c, s).float().to(BF)) and torch.equal(vo, ko)
    assert bool(ko.isfinite().all())
    for dst in (BF, FP):  # read back: values below fp16's normal range, and above its largest
        rk, rv = qmm.qmm_kv_read(cache, ints([[0]]), ints([0, 12]), 12, out_dtype=dst)
        assert torch.equal(rk, kv_ref.values(c, s).float().to(dst)) and torch.equal(rv, rk)


def test_append_strides_layers_and_streams():
    """Views of a fused product, the pages of one layer among several, outputs in place, another stream, no tokens."""
    g = gen(6)
    m, hq, hk, d = 19, 4, 2, 64
    q, k, v = (normal(g, m, h, d).to(BF) for h in (hq, hk, hk))
    slots = (5 + torch.arange(m, device=DEV)).to(torch.int32)
    pos, inv = slots.clone(), torch.linspace(1, 1e-2, 32, device=DEV)
    alone = cache_of(2, "q8_0", 32, hk, d)
    want = qmm.qmm_kv_append(q, k, v, pos, inv, alone, slots, values=True)
    n = alone.pages.shape[1]
    layers = torch.full((2, 3, n), 255, dtype=torch.uint8, device=DEV)
    one = qmm.KVPages(layers[:, 1], "q8_0", 32, hk, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    wide = torch.zeros(hq, m + 1, d, dtype=BF, device=DEV)
    got = qmm.qmm_kv_append(q, k, v, pos, inv, one, slots, values=True, q_out=wide.transpose(0, 1)[:m], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not wide[:, m].any()
    assert torch.equal(layers[:, 1], alone.pages) and bool((layers[:, 0::2] == 255).all())
    qmm.qmm_kv_append(q, k, v, pos, inv, one, slots, q_out=q, k_out=k, v_out=v)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, want[2])
    e = torch.empty((0, hk, d), device=DEV)
    out = qmm.qmm_kv_append(e, e, e, ints([]), inv, one, ints([]), values=True)
    assert [tuple(x.shape) for x in out] == [(0, hk, d)] * 3


# ------------------------------------------------------------------------------ reading back
def filled(g, lens, qtype, page, hk, d, spread=1.0, spare=3):
    """A cache with sequences of `lens` tokens in mixed pages, everything else NaN: (cache, table, codes, scales),
    the last two as [2][sequence]."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    cache = cache_of(n_pages, qtype, page, hk, d)
    order = torch.randperm(n_pages, generator=g, device=DEV)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device=DEV)
    codes, scales, at = ([], []), ([], []), 0
    for i, n in enumerate(lens):
        mine = order[at:at + need[i]]
        at += need[i]
        table[i, :need[i]] = mine.to(torch.int32)
        j = torch.arange(n, device=DEV)
        slots = mine[j // page] * page + j % page if n else j
        got = [kv_ref.quantize(qtype, normal(g, n, hk, d) * spread) for _ in range(2)]
        kv_ref.store(cache.pages, qtype, page, hk, d, slots, [x[0] for x in got], [x[1] for x in got])
        for side in range(2):
            codes[side].append(got[side][0])
            scales[side].append(got[side][1])
    return cache, table, codes, scales


@pytest.mark.parametrize("lens,hk,d,page,qtype,dst", [
    ([1], 1, 32, 16, "q4_0", BF),
    ([297], 8, 128, 16, "q4_0", BF),
    ([15, 16, 17, 0, 31, 33], 3, 64, 16, "q8_0", FP),
    ([255, 257, 1], 2, 96, 256, "q4_0", FP),
    ([500, 0, 0, 3], 4, 96, 32, "q8_0", BF),
    ([2000, 70], 8, 128, 64, "q8_0", FP),
    ([5000], 16, 32, 128, "q4_0", FP),
    ([3] * 300, 2, 64, 16, "q4_0", BF),
])
def test_read(lens, hk, d, page, qtype, dst):
    g = gen(sum(lens) + d)
    cache, table, codes, scales = filled(g, lens, qtype, page, hk, d)
    cu = ints([0] + lens).cumsum(0).to(torch.int32)
    k, v = qmm.qmm_kv_read(cache, table, cu, sum(lens), out_dtype=dst)
    for out, c, s in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
        assert torch.equal(out, kv_ref.values(torch.cat(c), torch.cat(s)).float().to(dst))
    assert qmm.qmm_take_attn_error() == 0


def test_read_rows_outside_and_bad_pages():
    """Rows before and after the sequences stay; rows of pages that do not exist are zero and reported."""
    g = gen(8)
    lens, hk, d, page = [40, 20], 2, 64, 16
    cache, table, codes, scales = filled(g, lens, "q4_0", page, hk, d)
    k, v = (torch.full((80, hk, d), 7.0, dtype=BF, device=DEV) for _ in range(2))
    cu = ints([5, 45, 65])
    qmm.qmm_kv_read(cache, table, cu, 80, k_out=k, v_out=v)
    assert bool((k[:5] == 7).all()) and bool((k[65:] == 7).all()) and bool((v[:5] == 7).all()) and bool((v[65:] == 7).all())
    want = kv_ref.values(torch.cat(codes[1]), torch.cat(scales[1])).float().to(BF)
    assert torch.equal(v[5:65], want)
    assert qmm.qmm_take_attn_error() == 0
    bad = table.clone()
    bad[0, 1] = cache.pages.shape[0]
    bad[1, 0] = -5
    k2, v2 = qmm.qmm_kv_read(cache, bad, cu, 80, k_out=k.clone(), v_out=v.clone())
    assert qmm.qmm_take_attn_error() == QMM_ERR_IDS and qmm.qmm_take_attn_error() == 0
    zero = torch.zeros(80, dtype=torch.bool, device=DEV)
    zero[5 + 16:5 + 32] = True
    zero[45:45 + 16] = True
    assert not k2[zero].any() and not v2[zero].any()
    assert torch.equal(k2[~zero], k[~zero]) and torch.equal(v2[~zero], v[~zero])
    # a table narrower than the sequence
    k3, _ = qmm.qmm_kv_read(cache, table[:, :2], cu, 80, k_out=k.clone(), v_out=v.clone())
    assert qmm.qmm_take_attn_error() == QMM_ERR_IDS
    assert not k3[5 + 32:45].any() and torch.equal(k3[5:37], k[5:37])
    # heads first, another stream
    out = torch.zeros(hk, 80, d, dtype=BF, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmm.qmm_kv_read(cache, table, cu, 80, k_out=out.transpose(0, 1), v_out=v, stream=side)
    side.synchronize()
    assert torch.equal(out.transpose(0, 1)[5:65], k[5:65])


# ------------------------------------------------------------------------------ decoding
def query(g, b, hq, d, dt, spread=1.0):
    return (normal(g, b, hq, d) * spread).to(dt)


@pytest.mark.parametrize("lens,hq,hk,d,page,qtype,dt", [
    ([1], 1, 1, 32, 16, "q4_0", BF),
    ([1], 4, 1, 128, 16, "q8_0", FP),
    ([640], 32, 8, 128, 16, "q4_0", BF),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65], 8, 2, 64, 16, "q4_0", FP),
    ([0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129], 4, 4, 128, 32, "q8_0", BF),
    ([300, 0, 5000, 77], 14, 2, 96, 64, "q4_0", BF),            # 7 heads of one kv head
    ([513, 1025], 16, 2, 96, 16, "q8_0", FP),                    # 8
    ([200, 31], 18, 2, 128, 128, "q4_0", FP),                    # 9: a block of 8 and one of 1
    ([333], 32, 2, 64, 256, "q4_0", BF),                         # 16
    ([90, 700], 128, 1, 32, 16, "q8_0", BF),                     # as many heads of one kv head as allowed
    ([1001, 999, 3], 16, 16, 64, 32, "q8_0", FP),
    ([20000], 8, 1, 128, 16, "q4_0", BF),                        # a long cache for few heads
    ([70000, 3], 4, 1, 64, 256, "q8_0", FP),
    ([65537], 5, 1, 32, 64, "q4_0", FP),
    ([100] * 200, 4, 2, 64, 16, "q4_0", BF),
    ([7] * 700, 8, 1, 128, 16, "q4_0", FP),
])
def test_decode(lens, hq, hk, d, page, qtype, dt):
    g = gen(sum(lens) + d + hq)
    cache, table, codes, scales = filled(g, lens, qtype, page, hk, d)
    q = query(g, len(lens), hq, d, dt)
    lse = torch.full((len(lens), hq), 7.0, device=DEV)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=max(lens), lse=lse)
    kv_ref.check_decode_kv(q, codes, scales, lens, d ** -0.5, qtype, out, lse)
    assert qmm.qmm_take_attn_error() == 0
    # the same bits again; with a wider bound the work is shared out in other parts
    assert torch.equal(qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=max(lens)), out)
    wide = torch.full((len(lens), table.shape[1] + 4000 // page), -7, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    more = qmm.qmm_attn_decode_kv(q, cache, wide, ints(lens), lse=lse)
    kv_ref.check_decode_kv(q, codes, scales, lens, d ** -0.5, qtype, more, lse)
    assert qmm.qmm_take_attn_error() == 0


@pytest.mark.parametrize("lens,hq,hk,d,page,qtype,dt", [
    ([7000, 1, 3000, 0, 31, 6999, 32, 64, 5000, 33], 8, 8, 32, 16, "q4_0", BF),
    ([12500, 100, 0, 6400], 36, 4, 64, 32, "q4_0", FP),          # 9 heads of a kv head
    ([25000, 0, 2000], 18, 2, 128, 256, "q8_0", BF),
    ([0, 0, 0, 26000, 0], 4, 2, 96, 64, "q8_0", FP),
    ([30000], 5, 1, 128, 16, "q4_0", FP),
    ([(37 * i) % 30 for i in range(180)] + [2500, 0, 1700, 2400] + [5] * 20, 4, 4, 32, 16, "q4_0", BF),
    ([2000 - 9 * i for i in range(200)], 4, 4, 32, 64, "q8_0", FP),
])
def test_decode_cut_into_parts(lens, hq, hk, d, page, qtype, dt):
    """The tiles of all requests in one row that resident CTAs cut: few requests, many, many short ones among long
    ones, more requests and heads than CTAs; the parts are joined in the workspace, which may hold anything."""
    g = gen(sum(lens) + d + hq)
    need = qmm.qmm_workspace_bytes_attn_decode_kv(len(lens), max(lens), hq, hk, d)
    assert need > 0
    cache, table, codes, scales = filled(g, lens, qtype, page, hk, d)
    q = query(g, len(lens), hq, d, dt)
    lse = torch.full((len(lens), hq), 7.0, device=DEV)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=max(lens), lse=lse)
    kv_ref.check_decode_kv(q, codes, scales, lens, d ** -0.5, qtype, out, lse)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=max(lens), workspace=ws), out)
    assert qmm.qmm_take_attn_error() == 0


@pytest.mark.parametrize("lens,hq,hk,d,page,qtype,dt", [
    ([(37 * i) % 201 for i in range(333)], 18, 2, 64, 16, "q4_0", BF),     # 9 heads of a kv head, a CTA that is not full
    ([(91 * i) % 500 for i in range(304)] + [500], 8, 4, 128, 32, "q8_0", FP),
    ([1 + i % 250 for i in range(700)], 3, 1, 96, 64, "q4_0", FP),
    ([32, 0, 31, 1, 5], 6, 3, 32, 16, "q8_0", BF),                          # a single tile each
])
def test_decode_many_short(lens, hq, hk, d, page, qtype, dt):
    """Many short requests, a warp for each request and kv head; one of them loses its pages."""
    g = gen(sum(lens) + d)
    assert qmm.qmm_workspace_bytes_attn_decode_kv(len(lens), max(lens), hq, hk, d) == 0
    cache, table, codes, scales = filled(g, lens, qtype, page, hk, d)
    q = query(g, len(lens), hq, d, dt)
    lse = torch.full((len(lens), hq), 7.0, device=DEV)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=max(lens), lse=lse)
    kv_ref.check_decode_kv(q, codes, scales, lens, d ** -0.5, qtype, out, lse)
    assert torch.equal(qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=max(lens)), out)
    assert qmm.qmm_take_attn_error() == 0
    bad = table.clone()
    bad[2] = cache.pages.shape[0]
    again = qmm.qmm_attn_decode_kv(q, cache, bad, ints(lens), max_len=max(lens))
    rest = torch.arange(len(lens), device=DEV) != 2
    assert not again[2].any() and torch.equal(again[rest], out[rest]) and qmm.qmm_take_attn_error() == QMM_ERR_IDS


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("spread,kspread,scale", [(8.0, 4.0, None), (1.0, 1.0, -0.3), (1.0, 1.0, 0.0), (1e-3, 0.01, 40.0),
                                                  (200.0, 0.05, None), (1.0, 1000.0, 1e-4)])
def test_decode_sharp_and_other_scales(spread, kspread, scale, qtype, dt):
    """Scores far apart, negative and zero scales, small and large queries and keys."""
    lens, hq, hk, d = [515, 130], 8, 2, 64
    g = gen(11)
    cache, table, codes, scales = filled(g, lens, qtype, 32, hk, d, kspread)
    q = query(g, 2, hq, d, dt, spread)
    q[1, 3] = 0
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=515, scale=scale)
    kv_ref.check_decode_kv(q, codes, scales, lens, d ** -0.5 if scale is None else scale, qtype, out)


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
def test_decode_rising_maximum(qtype):
    """Scores that rise key by key, so that the running maximum moves at every tile."""
    n, d, page = 900, 128, 16
    g = gen(12)
    cache, table, codes, scales = filled(g, [n], qtype, page, 1, d)
    slots = (table[0].long()[torch.arange(n, device=DEV) // page] * page + torch.arange(n, device=DEV) % page)
    k = torch.zeros(n, 1, d, device=DEV)
    k[:, 0, 0] = torch.arange(n, device=DEV) / 10
    codes[0][0], scales[0][0] = kv_ref.quantize(qtype, k)
    kv_ref.store(cache.pages, qtype, page, 1, d, slots, [c[0] for c in codes], [s[0] for s in scales])
    q = torch.zeros(1, 8, d, dtype=FP, device=DEV)
    q[..., 0] = torch.arange(8, device=DEV) - 2
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints([n]), max_len=n, scale=1.0)
    kv_ref.check_decode_kv(q, codes, scales, [n], 1.0, qtype, out)


def test_decode_lens_are_clipped_and_pages_shared():
    """lens below zero and beyond max_len; the same page in two requests' tables, and twice in one."""
    g = gen(13)
    cache, table, codes, scales = filled(g, [64, 40], "q4_0", 16, 2, 64)
    q = query(g, 4, 4, 64, BF)
    shared = torch.stack([table[0], table[0], table[1], table[0]])
    shared[3, 2] = table[0, 0]  # tokens 32..47 are tokens 0..15 again
    out = qmm.qmm_attn_decode_kv(q, cache, shared, ints([1000, -3, 40, 48]), max_len=64)
    twice = [[codes[i][0], codes[i][0], codes[i][1], torch.cat((codes[i][0][:32], codes[i][0][:16]))] for i in range(2)]
    stwice = [[scales[i][0], scales[i][0], scales[i][1], torch.cat((scales[i][0][:32], scales[i][0][:16]))] for i in range(2)]
    kv_ref.check_decode_kv(q, twice, stwice, [64, 0, 40, 48], 0.125, "q4_0", out)
    assert qmm.qmm_take_attn_error() == 0
    # no key at all
    lse = torch.zeros(4, 4, device=DEV)
    out = qmm.qmm_attn_decode_kv(q, cache, shared, ints([3, 3, 3, 3]), max_len=0, lse=lse)
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("n,page", [(200, 16), (6000, 64), (20000, 32)])
def test_decode_bad_pages(n, page):
    """Tokens of pages outside the cache count as not there, and the call says so."""
    g = gen(14)
    cache, table, codes, scales = filled(g, [n, 33], "q4_0", page, 2, 64)
    q = query(g, 2, 8, 64, FP)
    bad = table.clone()
    gone = [1, 2, (n - 1) // page]
    bad[0, gone[0]], bad[0, gone[1]], bad[0, gone[2]] = -1, cache.pages.shape[0], 2 ** 31 - 1
    out = qmm.qmm_attn_decode_kv(q, cache, bad, ints([n, 33]), max_len=n)
    assert qmm.qmm_take_attn_error() == QMM_ERR_IDS
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    for p in gone:
        keep[p * page:(p + 1) * page] = False
    for side in range(2):
        codes[side][0], scales[side][0] = codes[side][0][keep], scales[side][0][keep]
    kv_ref.check_decode_kv(q, codes, scales, [int(keep.sum()), 33], 0.125, "q4_0", out)
    # every page of a request is gone
    bad[1] = -1
    out2 = qmm.qmm_attn_decode_kv(q, cache, bad, ints([n, 33]), max_len=n)
    assert torch.equal(out2[0], out[0]) and not out2[1].any()
    assert qmm.qmm_take_attn_error() == QMM_ERR_IDS


def test_decode_strides_streams_graphs_and_bits():
    """Strided queries, outputs, tables and pages; another stream; two at once; a graph replayed on new lengths."""
    g = gen(15)
    lens, hq, hk, d, page = [900, 77, 30000], 8, 2, 128, 64
    cache, table, codes, scales = filled(g, lens, "q4_0", page, hk, d)
    q = query(g, 3, hq, d, BF)
    want = qmm.qmm_attn_decode_kv(q, cache, table, ints(lens), max_len=30000)
    kv_ref.check_decode_kv(q, codes, scales, lens, d ** -0.5, "q4_0", want)
    layers = torch.full((cache.pages.shape[0], 2, cache.pages.shape[1]), 255, dtype=torch.uint8, device=DEV)
    layers[:, 1] = cache.pages
    one = qmm.KVPages(layers[:, 1], "q4_0", page, hk, d)
    qs = torch.empty(hq, 3, d, dtype=BF, device=DEV)
    qs.copy_(q.transpose(0, 1))
    wide = torch.full((3, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    out = torch.empty_like(qs)
    need = qmm.qmm_workspace_bytes_attn_decode_kv(3, 30000, hq, hk, d)
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device=DEV)
    ll = ints(lens)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    a = qmm.qmm_attn_decode_kv(qs.transpose(0, 1), one, wide[:, :table.shape[1]], ll, max_len=30000,
                               out=out.transpose(0, 1), workspace=ws, stream=side)
    b = qmm.qmm_attn_decode_kv(q, cache, table, ll, max_len=30000, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    now = ints(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = qmm.qmm_attn_decode_kv(q, cache, table, now, max_len=30000)
    for new in (lens, [1, 0, 29999]):
        now.copy_(ints(new))
        graph.replay()
        torch.cuda.synchronize()
        kv_ref.check_decode_kv(q, codes, scales, new, d ** -0.5, "q4_0", c)
    assert torch.equal(qmm.qmm_attn_decode_kv(q, cache, table, now, max_len=30000), c)
    e = torch.empty(0, hq, d, dtype=BF, device=DEV)
    assert qmm.qmm_attn_decode_kv(e, cache, table[:0], ll[:0], max_len=0).shape == (0, hq, d)


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("lens", [[100, 5], [9000], [40] * 90, [13000, 0, 3, 20, 8000] + [1] * 20, [60] * 400],
                         ids=["short", "split", "many", "pieces", "alone"])
def test_decode_waits_that_give_up(lens, mode):
    """Copies that never come (none is issued) and a wait that gives up with copies in flight: the call ends,
    reports, and the next one is right."""
    g = gen(16)
    cache, table, codes, scales = filled(g, lens, "q8_0", 32, 2, 128)
    q, ll = query(g, len(lens), 8, 128, BF), ints(lens)
    qmm.qmm_set_test_fault(mode)
    qmm.qmm_attn_decode_kv(q, cache, table, ll, max_len=max(lens))
    qmm.qmm_set_test_fault(0)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ll, max_len=max(lens))
    assert qmm.qmm_take_attn_error() == QMM_ERR_DEVICE and qmm.qmm_take_attn_error() == 0
    kv_ref.check_decode_kv(q, codes, scales, lens, 128 ** -0.5, "q8_0", out)


def test_decode_two_workspaces_at_once():
    """Two calls whose parts lie in workspaces of their own, on two streams, again and again."""
    g = gen(18)
    lens, hq, hk, d = [26000, 700, 8000], 8, 2, 64
    cache, table, codes, scales = filled(g, lens, "q4_0", 16, hk, d)
    need = qmm.qmm_workspace_bytes_attn_decode_kv(3, 26000, hq, hk, d)
    assert need > 0
    q = [query(g, 3, hq, d, BF) for _ in range(2)]
    ll = ints(lens)
    want = [qmm.qmm_attn_decode_kv(x, cache, table, ll, max_len=26000) for x in q]
    ws = [torch.full((need,), 255, dtype=torch.uint8, device=DEV) for _ in q]
    outs = [torch.empty_like(x) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, o, w, s in zip(q, outs, ws, streams):
            qmm.qmm_attn_decode_kv(x, cache, table, ll, max_len=26000, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    with pytest.raises(qmm.QMMError):
        qmm.qmm_attn_decode_kv(q[0], cache, table, ll, max_len=26000, workspace=ws[0][:need - 256])


def test_decode_far_pages():
    """A cache of more than 2^32 bytes: pages at its far end."""
    page, hk, d = 256, 8, 128
    n = (1 << 32) // kv_ref.page_bytes("q8_0", page, hk, d) + 40
    pages = torch.empty((n, kv_ref.page_bytes("q8_0", page, hk, d)), dtype=torch.uint8, device=DEV)
    pages[-3:] = 255
    cache = qmm.KVPages(pages, "q8_0", page, hk, d)
    g = gen(17)
    m = 600
    k, v, q = normal(g, m, hk, d), normal(g, m, hk, d), query(g, 1, 32, d, BF)
    table = ints([[n - 1, n - 3, n - 2]])
    j = torch.arange(m, device=DEV)
    slots = (table[0].long()[j // page] * page + j % page).to(torch.int32)
    _, ko, vo = qmm.qmm_kv_append(None, k, v, None, None, cache, slots, values=True)
    rk, rv = qmm.qmm_kv_read(cache, table, ints([0, m]), m)
    assert torch.equal(rk, ko) and torch.equal(rv, vo)
    out = qmm.qmm_attn_decode_kv(q, cache, table, ints([m]), max_len=m)
    kc, ks = kv_ref.quantize("q8_0", k)
    vc, vs = kv_ref.quantize("q8_0", v)
    kv_ref.check_decode_kv(q, [[kc], [vc]], [[ks], [vs]], [m], d ** -0.5, "q8_0", out)


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("qtype,dt", [("q4_0", BF), ("q8_0", FP)])
def test_chunks_then_steps(qtype, dt):
    """Two prompts come in chunks (append, read the history back, attend), then go on token by token (append,
    decode), against fp64 over the bytes that the cache holds."""
    hq, hk, d, page = 8, 2, 64, 16
    g = gen(21)
    cache = cache_of(20, qtype, page, hk, d)
    order = torch.randperm(20, generator=g, device=DEV).to(torch.int32)
    table = torch.stack([order[:9], order[9:18]])
    w, inv = 1 + 0.1 * normal(g, d), torch.linspace(1, 1e-3, d // 2, device=DEV)
    have = [0, 0]

    def slots_of(new):
        pos = [torch.arange(a, a + n, device=DEV) for a, n in zip(have, new)]
        return (torch.cat([table[i].long()[p // page] * page + p % page for i, p in enumerate(pos)]).to(torch.int32),
                torch.cat(pos).to(torch.int32))

    def held(i):
        j = torch.arange(have[i], device=DEV)
        return kv_ref.load(cache.pages, qtype, page, hk, d, table[i].long()[j // page] * page + j % page)

    for new in ([37, 1], [20, 70]):
        m = sum(new)
        qkv = normal(g, m, (hq + 2 * hk) * d)
        q, k, v = (x.view(m, -1, d) for x in qkv.split((hq * d, hk * d, hk * d), 1))
        slots, pos = slots_of(new)
        qo, ko, vo = qmm.qmm_kv_append(q, k, v, pos, inv, cache, slots, w_q=w, w_k=w, out_dtype=dt, values=True)
        first = have == [0, 0]
        have = [a + n for a, n in zip(have, new)]
        cu_q, cu_k = (ints([0] + x).cumsum(0).to(torch.int32) for x in (new, have))
        kk, vv = qmm.qmm_kv_read(cache, table, cu_k, sum(have), out_dtype=dt)
        if first:
            assert torch.equal(kk, ko) and torch.equal(vv, vo)
        out = qmm.qmm_attn_prompt(qo, kk, vv, cu_q, cu_k)
        check_prompt(qo, kk, vv, new, have, True, d ** -0.5, out)
        both = [held(i) for i in range(2)]
        assert torch.equal(kk, torch.cat([kv_ref.values(c[0], s[0]) for c, s in both]).float().to(dt))
    for _ in range(5):
        qkv = normal(g, 2, (hq + 2 * hk) * d)
        q, k, v = (x.view(2, -1, d) for x in qkv.split((hq * d, hk * d, hk * d), 1))
        slots, pos = slots_of([1, 1])
        qo, _, _ = qmm.qmm_kv_append(q, k, v, pos, inv, cache, slots, w_q=w, w_k=w, out_dtype=dt)
        have = [a + 1 for a in have]
        out = qmm.qmm_attn_decode_kv(qo, cache, table, ints(have), max_len=9 * page)
        both = [held(i) for i in range(2)]
        kv_ref.check_decode_kv(qo, [[c[x] for c, _ in both] for x in range(2)], [[s[x] for _, s in both] for x in range(2)],
                               have, d ** -0.5, qtype, out)
    assert qmm.qmm_take_attn_error() == 0


def test_a_captured_step():
    """Append and decode in one graph, replayed token after token with new inputs in the same places, against the
    same calls made one by one on a cache of their own."""
    hq, hk, d, page, b = 16, 4, 128, 32, 3
    g = gen(22)
    lens0 = [40, 1, 95]
    cache, table, codes, scales = filled(g, lens0, "q4_0", page, hk, d, spare=6)
    table = torch.cat((table, torch.arange(cache.pages.shape[0] - 3, cache.pages.shape[0], device=DEV, dtype=torch.int32)[:, None]), 1)
    free = sorted(set(range(cache.pages.shape[0])) - set(table[table >= 0].tolist()))
    for i, n in enumerate(lens0):  # the page after each sequence's last
        table[i, -(-n // page)] = free[i]
    other = qmm.KVPages(cache.pages.clone(), "q4_0", page, hk, d)
    w, inv = 1 + 0.1 * normal(g, d), torch.linspace(1, 1e-3, d // 2, device=DEV)
    qkv, slots, lens = torch.zeros(b, hq + 2 * hk, d, device=DEV), ints([0] * b), ints(lens0)

    def step(where):
        q, _, _ = qmm.qmm_kv_append(qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], lens, inv, where, slots, w_q=w, w_k=w)
        return qmm.qmm_attn_decode_kv(q, where, table, lens + 1, max_len=128)

    def place():
        at = lens.long()
        slots.copy_(table[torch.arange(b, device=DEV), at // page] * page + at % page)

    place()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache)
    for _ in range(20):
        qkv.copy_(normal(g, b, hq + 2 * hk, d))
        place()
        graph.replay()
        assert torch.equal(out, step(other)) and torch.equal(cache.pages, other.pages)
        lens += 1
    assert qmm.qmm_take_attn_error() == 0


def test_binding_refuses():
    cache = cache_of(4, "q4_0", 16, 2, 64)
    q, k = torch.zeros(3, 4, 64, dtype=BF, device=DEV), torch.zeros(3, 2, 64, dtype=BF, device=DEV)
    slots, table, lens = ints([0, 1, 2]), ints([[0], [1], [2]]), ints([1, 1, 1])
    for call, code in (
            (lambda: qmm.KVPages(cache.pages[:, :-16], "q4_0", 16, 2, 64), 2),
            (lambda: qmm.KVPages(cache.pages.int(), "q4_0", 16, 2, 64), 3),
            (lambda: qmm.KVPages(cache.pages, "q8_0", 16, 2, 64), 2),
            (lambda: qmm.qmm_kv_append(q, k, k, None, None, cache, slots[:2]), 2),
            (lambda: qmm.qmm_kv_append(q, k, k, None, None, cache, slots.long()), 3),
            (lambda: qmm.qmm_kv_append(q, k, k[:2], None, None, cache, slots), 2),
            (lambda: qmm.qmm_kv_append(q, k.float(), k, None, None, cache, slots), 3),
            (lambda: qmm.qmm_kv_append(q, q, q, None, None, cache, slots), 2),
            (lambda: qmm.qmm_kv_append(q, k, k, None, None, cache, slots, out_dtype=torch.float32), 3),
            (lambda: qmm.qmm_kv_append(None, k, k, None, None, cache, slots, q_out=q), 1),
            (lambda: qmm.qmm_kv_append(q, k, k, slots.cpu(), torch.ones(32, device=DEV), cache, slots), 1),
            (lambda: qmm.qmm_kv_read(cache, table, ints([0, 1, 2]), 2), 2),
            (lambda: qmm.qmm_kv_read(cache, table.long(), ints([0, 1, 2, 3]), 3), 1),
            (lambda: qmm.qmm_kv_read(cache, table, ints([0, 1, 2, 3]), 3, out_dtype=torch.float32), 3),
            (lambda: qmm.qmm_attn_decode_kv(q, cache, table, lens, max_len=17), 2),
            (lambda: qmm.qmm_attn_decode_kv(q, cache, table[:2], lens), 2),
            (lambda: qmm.qmm_attn_decode_kv(q.float(), cache, table, lens), 3),
            (lambda: qmm.qmm_attn_decode_kv(q[..., :32], cache, table, lens), 2),
            (lambda: qmm.qmm_attn_decode_kv(q, cache, table, lens, scale=math.inf), 1)):
        with pytest.raises(qmm.QMMError) as e:
            call()
        assert e.value.code == code
