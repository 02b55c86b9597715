"""The cache calls of the C ABI refuse bad arguments before anything touches a GPU; the cache's sizes; the
reference's bytes."""
import ctypes

import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
import kv_ref

P = ctypes.c_void_p
F16, BF16, F32 = 1, 30, 0
Q4_0, Q8_0, Q4_K = 2, 8, 12


@pytest.fixture(scope="module")
def L():
    qmm.build()
    return qmm.lib()


def H(data=4096, token=512, head=64):
    return qmm.Heads(data, token, head)


def C(data=4096, n=10, stride=4608, page=32, t=Q4_0):
    return qmm.Cache(data, n, stride, page, t)


def append(L, q=H(), k=H(), v=H(), t=F32, m=4, hq=8, hk=2, d=64, wq=4096, wk=4096, eps=1e-6, pos=4096, inv=4096, r=64,
           c=C(), slots=4096, qo=H(), ko=H(), vo=H(), to=BF16):
    return L.qmm_kv_append(q, k, v, t, m, hq, hk, d, P(wq), P(wk), eps, P(pos), P(inv), r, 0, c, P(slots), qo, ko, vo, to,
                           None)


def read(L, c=C(), table=4096, width=5, stride=5, cu=4096, n=2, tokens=100, hk=2, d=64, ko=H(), vo=H(), to=F16):
    return L.qmm_kv_read(c, P(table), width, stride, P(cu), n, tokens, hk, d, ko, vo, to, None)


def decode(L, q=H(), c=C(), table=4096, width=5, stride=5, lens=4096, b=4, most=160, t=F16, hq=8, hk=2, d=64, scale=1.0,
           out=H(), lse=0, ws=0, wsb=0):
    return L.qmm_attn_decode_kv(q, c, P(table), width, stride, P(lens), b, most, t, hq, hk, d, scale, out, P(lse), P(ws),
                                wsb, None)


@pytest.mark.parametrize("t,name", [(Q4_0, "q4_0"), (Q8_0, "q8_0")])
def test_page_bytes(L, t, name):
    f = L.qmm_kv_page_bytes
    for page in (16, 32, 64, 128, 256):
        for hk, d in ((1, 32), (2, 64), (8, 96), (32, 128)):
            # 16 or 32 bytes of codes and 2 of scale a block of 32, keys and values
            assert f(t, page, hk, d) == page * hk * 2 * (d // 32) * (18 if t == Q4_0 else 34)
            assert f(t, page, hk, d) == kv_ref.page_bytes(name, page, hk, d)
    assert f(t, 8, 1, 64) == 0 and f(t, 48, 1, 64) == 0 and f(t, 512, 1, 64) == 0 and f(t, -16, 1, 64) == 0
    assert f(t, 16, 0, 64) == 0 and f(t, 16, 1, 40) == 0 and f(t, 16, 1, 160) == 0 and f(t, 16, 1, 0) == 0
    assert f(t, 16, 4097, 64) == 0
    assert f(Q4_K, 16, 1, 64) == 0 and f(0, 16, 1, 64) == 0


def bad_caches(call):
    assert call(c=None) == 1 and call(c=C(data=0)) == 1 and call(c=C(n=-1)) == 1
    assert call(c=C(t=Q4_K)) == 3 and call(c=C(t=0)) == 3
    assert call(c=C(page=48)) == 2 and call(c=C(page=512)) == 2 and call(c=C(page=0)) == 2
    assert call(c=C(stride=4592)) == 2                    # pages that overlap
    assert call(c=C(n=1 << 26)) == 2                      # slots past 31 bits
    assert call(c=C(data=4104)) == 4 and call(c=C(stride=4616)) == 4
    assert call(c=C(n=1, data=4104)) == 4                 # (the stride of a single page is never taken)


def test_append_refuses(L):
    bad_caches(lambda **kw: append(L, **kw))
    assert append(L, t=9) == 3 and append(L, to=F32) == 3
    assert append(L, m=-1) == 1 and append(L, eps=-1.0) == 1 and append(L, eps=float("nan")) == 1 and append(L, r=-8) == 1
    assert append(L, hq=0) == 1 and append(L, hk=0) == 1 and append(L, d=0) == 1
    assert append(L, d=80) == 2 and append(L, d=160) == 2 and append(L, r=72) == 2 and append(L, r=12) == 2
    assert append(L, hq=5000) == 2 and append(L, m=1 << 31) == 2
    assert append(L, k=None) == 1 and append(L, v=None) == 1 and append(L, slots=0) == 1 and append(L, pos=0) == 1
    assert append(L, q=None) == 1 and append(L, qo=None) == 1 and append(L, ko=None) == 1 and append(L, vo=None) == 1
    assert append(L, q=H(token=514)) == 4 and append(L, ko=H(token=516)) == 4 and append(L, v=H(data=4104)) == 4
    assert append(L, slots=4098) == 4 and append(L, inv=4097) == 4 and append(L, wk=4098) == 4
    assert append(L, k=H(token=32)) == 2
    assert append(L, m=0) == 0
    assert append(L, m=0, q=None, qo=None, hq=0, ko=None, vo=None) == 0


def test_read_refuses(L):
    bad_caches(lambda **kw: read(L, **kw))
    assert read(L, to=F32) == 3
    assert read(L, n=-1) == 1 and read(L, tokens=-1) == 1 and read(L, width=-1) == 1 and read(L, table=0) == 1
    assert read(L, stride=4) == 2 and read(L, n=(1 << 20) + 1) == 2 and read(L, tokens=1 << 31) == 2 and read(L, d=48) == 2
    assert read(L, cu=0) == 1 and read(L, ko=None) == 1 and read(L, vo=None) == 1
    assert read(L, table=4098) == 4 and read(L, cu=4098) == 4 and read(L, ko=H(data=4104)) == 4
    assert read(L, n=0) == 0 and read(L, tokens=0) == 0


def test_decode_refuses(L):
    bad_caches(lambda **kw: decode(L, **kw))
    assert decode(L, t=F32) == 3
    assert decode(L, b=-1) == 1 and decode(L, most=-1) == 1 and decode(L, hk=0) == 1
    assert decode(L, hq=9) == 2 and decode(L, d=80) == 2 and decode(L, b=1 << 31) == 2 and decode(L, hq=129 * 2) == 2
    assert decode(L, most=161) == 2                       # more than the table holds
    assert decode(L, scale=float("nan")) == 1 and decode(L, scale=float("inf")) == 1
    assert decode(L, lens=0) == 1 and decode(L, q=None) == 1 and decode(L, out=None) == 1 and decode(L, table=0) == 1
    assert decode(L, stride=4) == 2 and decode(L, table=4098) == 4 and decode(L, lens=4098) == 4 and decode(L, lse=4098) == 4
    assert decode(L, q=H(token=516)) == 4 and decode(L, out=H(data=4104)) == 4
    assert decode(L, b=0) == 0
    w = L.qmm_workspace_bytes_attn_decode_kv
    assert w(-1, 10, 8, 2, 64) == 0 and w(1, 10, 7, 2, 64) == 0 and w(1, 10, 8, 2, 80) == 0 and w(0, 10, 8, 2, 64) == 0


@pytest.mark.parametrize("qtype", ["q4_0", "q8_0"])
@pytest.mark.parametrize("page,hk,d", [(16, 1, 32), (32, 3, 96), (128, 2, 128)])
def test_reference_bytes(qtype, page, hk, d):
    """Every byte of a page belongs to one token's code or scale, and what is stored is loaded."""
    g = torch.Generator().manual_seed(page + d)
    n = kv_ref.page_bytes(qtype, page, hk, d)
    slots = torch.randperm(3 * page, generator=g)
    x = [torch.randn(3 * page, hk, d, generator=g) for _ in range(2)]
    codes, scales = zip(*(kv_ref.quantize(qtype, y) for y in x))
    for fill in (0, 255):
        buf = torch.full((3, n), fill, dtype=torch.uint8)
        kv_ref.store(buf, qtype, page, hk, d, slots, codes, scales)
        c, s = kv_ref.load(buf, qtype, page, hk, d, slots)
        assert all(torch.equal(a, b) for a, b in zip(c, codes)) and all(torch.equal(a, b) for a, b in zip(s, scales))
        if fill:
            assert torch.equal(buf, kept)
        kept = buf
    for y, c, s in zip(x, codes, scales):  # half a step, and at the clamped end of 4 bits a whole one
        off = (kv_ref.values(c, s) - y.double()).abs().unflatten(-1, (-1, 32)) / s.double().abs()[..., None]
        assert float(off.max()) <= (1.02 if qtype == "q4_0" else 0.57)


def test_binding_refuses_without_a_gpu():
    with pytest.raises(qmm.QMMError):
        qmm.KVPages(torch.empty((2, 4608), dtype=torch.uint8), "q4_0", 32, 2, 64)  # not on a GPU
    with pytest.raises(qmm.QMMError):
        qmm.KVPages(torch.empty((2, 4608), dtype=torch.uint8), "q4_K", 32, 2, 64)
    with pytest.raises(qmm.QMMError):
        qmm.KVPages(torch.empty((2, 4608), dtype=torch.uint8), "q4_0", 40, 2, 64)
