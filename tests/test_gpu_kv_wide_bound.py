"""Decoding over pages with max_len far above the lengths: a fixed bound and fixed places for requests, most of
them short or empty, as a captured step sees them."""
import pytest
import torch

import block_quantized_matmul_q8_gb300 as qmm
import kv_ref
from test_gpu_kv import BF, DEV, FP, _errors, _lib, filled, gen, ints, query  # noqa: F401 (two are fixtures)

pytestmark = pytest.mark.gpu


def widened(table, page, most):
    """The table with room for `most` tokens; the entries past a request's pages are no pages."""
    wide = torch.full((table.shape[0], -(-most // page)), -7, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    return wide


def check(lens, most, hq, hk, d, page, qtype, dt):
    g = gen(sum(lens) + most + hq)
    need = qmm.qmm_workspace_bytes_attn_decode_kv(len(lens), most, hq, hk, d)
    assert need > 0  # requests are cut into parts that lie in the workspace
    cache, table, codes, scales = filled(g, lens, qtype, page, hk, d)
    table, ll, q = widened(table, page, most), ints(lens), query(g, len(lens), hq, d, dt)
    got = []
    for fill in (255, 0, 0x3c):  # whatever the workspace holds: NaN, zeros, numbers
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        out, lse = torch.full_like(q, 7), torch.full((len(lens), hq), 7.0, device=DEV)
        qmm.qmm_attn_decode_kv(q, cache, table, ll, max_len=most, out=out, lse=lse, workspace=ws)
        got.append((out, lse))
    kv_ref.check_decode_kv(q, codes, scales, lens, d ** -0.5, qtype, *got[0])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert qmm.qmm_take_attn_error() == 0


@pytest.mark.parametrize("n", [0, 1, 32, 33, 64, 65, 100, 640, 1500, 1980, 4000, 7700])
@pytest.mark.parametrize("most,hq,hk,d,page,qtype,dt", [
    (32768, 32, 8, 128, 16, "q4_0", BF),
    (131072, 32, 8, 128, 32, "q4_0", FP),
    (131072, 8, 2, 128, 256, "q8_0", BF),
    (131072, 8, 1, 64, 64, "q4_0", FP),
    (25000, 9, 1, 96, 16, "q4_0", BF),                       # 9 heads of a kv head
])
def test_one_request(n, most, hq, hk, d, page, qtype, dt):
    check([n], most, hq, hk, d, page, qtype, dt)


@pytest.mark.parametrize("lens,most,hq,hk,d,page,qtype,dt", [
    ([100] + [0] * 127, 8192, 32, 8, 128, 32, "q4_0", BF),
    ([0] * 77 + [100] + [0] * 49 + [64], 8192, 32, 8, 128, 32, "q4_0", BF),
    ([300, 20], 32768, 8, 1, 128, 16, "q8_0", FP),
    ([40, 0, 33], 25000, 8, 2, 64, 64, "q8_0", BF),
    ([0, 0, 65, 0, 0, 1000, 0], 32768, 16, 16, 32, 16, "q4_0", FP),
    ([33] * 3 + [0] * 300, 8192, 4, 1, 96, 256, "q4_0", BF),
    ([50 + i for i in range(48)], 16384, 36, 4, 128, 64, "q4_0", BF),
    ([0] * 5, 32768, 4, 1, 64, 16, "q4_0", BF),
])
def test_places_without_requests(lens, most, hq, hk, d, page, qtype, dt):
    check(lens, most, hq, hk, d, page, qtype, dt)


def test_default_bound_is_the_tables_width():
    g = gen(5)
    cache, table, codes, scales = filled(g, [700, 50], "q4_0", 16, 8, 128)
    q = query(g, 2, 32, 128, BF)
    torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV)  # what the workspace may be made of
    out = qmm.qmm_attn_decode_kv(q, cache, widened(table, 16, 65536), ints([700, 50]))
    kv_ref.check_decode_kv(q, codes, scales, [700, 50], 128 ** -0.5, "q4_0", out)


def test_replayed_from_the_first_token_on():
    """One captured call of a fixed bound and three places, replayed while requests grow and others stay empty."""
    full, most, hq, hk, d, page = [3000, 3000, 500], 131072, 16, 4, 128, 64
    g = gen(6)
    cache, table, codes, scales = filled(g, full, "q4_0", page, hk, d)
    table, q, lens = widened(table, page, most), query(g, 3, hq, d, BF), ints([1, 0, 0])
    ws = torch.full((qmm.qmm_workspace_bytes_attn_decode_kv(3, most, hq, hk, d),), 255, dtype=torch.uint8, device=DEV)

    def step():
        return qmm.qmm_attn_decode_kv(q, cache, table, lens, max_len=most, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for now in ([1, 0, 0], [33, 0, 0], [100, 0, 1], [640, 40, 0], [900, 0, 500], [1979, 0, 0], [3000, 3000, 500], [64, 0, 0]):
        lens.copy_(ints(now))
        ws.fill_(255)
        graph.replay()
        kv_ref.check_decode_kv(q, codes, scales, now, d ** -0.5, "q4_0", out)
        first = out.clone()
        graph.replay()
        assert torch.equal(first, out)
    assert qmm.qmm_take_attn_error() == 0
