"""One attention layer of a decoder on the library's calls: a quantized qkv projection, the norm and
rotation of its heads, attention, and a quantized output projection, for packed prompts, for a
decoding batch that shares one long prefix, and over a paged cache in 4 or 8 bits.

    python examples/attention_layer.py

prints the time of each call for a prefix of 4096 tokens, 16 requests and a few steps, then for 16 prompts of 512
tokens in pages and a few steps after them.
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_quantized_matmul_q8_gb300 as qmm  # noqa: E402
import qmm_synth  # noqa: E402


class AttentionLayer:
    def __init__(self, hidden=1024, heads=8, kv_heads=2, dim=128, fmt="q4_K", dtype=torch.bfloat16, seed=0,
                 device="cuda:0"):
        self.hidden, self.heads, self.kv_heads, self.dim, self.fmt, self.dtype = hidden, heads, kv_heads, dim, fmt, dtype
        self.width = (heads + 2 * kv_heads) * dim
        rng = np.random.default_rng(seed)
        # values small enough that random weights give scores of order one
        self.w_qkv, self.w_o = (torch.from_numpy(qmm_synth.gen_weights(fmt, rng, n, k)).to(device)
                                for n, k in ((self.width, hidden), (hidden, heads * dim)))
        g = torch.Generator(device=device).manual_seed(seed)
        self.norm_q, self.norm_k = (1 + 0.1 * torch.randn(dim, generator=g, device=device) for _ in range(2))
        self.inv_freq = (10000.0 ** (-torch.arange(0, dim, 2, device=device) / dim)).float()

    def project(self, x):
        """x fp32 [tokens, hidden] -> the heads of q, k and v as views of the product's rows."""
        y = qmm.qmm_mul_mat_f32(self.w_qkv, self.fmt, self.width, self.hidden, x, x.shape[0])
        h = y.view(x.shape[0], -1, self.dim)
        return h[:, :self.heads], h[:, self.heads:self.heads + self.kv_heads], h[:, self.heads + self.kv_heads:]

    def qkv(self, x, positions):
        """x fp32 [tokens, hidden] -> q [tokens, heads, dim], k and v [tokens, kv_heads, dim], normed and rotated."""
        q, k, v = self.project(x)
        return qmm.qmm_qk_norm_rope(q, k, v, positions, self.inv_freq, w_q=self.norm_q, w_k=self.norm_k,
                                    out_dtype=self.dtype)

    def output(self, attended):
        """The output projection of attention rows [tokens, heads, dim], fp32 [tokens, hidden]."""
        a = attended.reshape(attended.shape[0], -1).float()
        return qmm.qmm_mul_mat_f32(self.w_o, self.fmt, self.hidden, a.shape[1], a, a.shape[0])

    def prefill(self, x, cu):
        """Packed prompts x with row bounds cu (int32, on the device): the layer's output, and the
        attention rows, queries, keys and values that a caller keeps or caches."""
        seq = torch.searchsorted(cu, torch.arange(x.shape[0], device=x.device, dtype=torch.int32), right=True) - 1
        positions = (torch.arange(x.shape[0], device=x.device) - cu[seq]).to(torch.int32)
        q, k, v = self.qkv(x, positions)
        attended = qmm.qmm_attn_prompt(q, k, v, cu)
        return self.output(attended), attended, (q, k, v)

    def step(self, x, prefix, caches, lens):
        """One token of each request, x [batch, hidden], after the shared prefix (k, v) and the
        request's own lens tokens in caches (k, v) [batch, room, kv_heads, dim], which take the new one."""
        q, k, v = self.qkv(x, lens + prefix[0].shape[0])
        rows = torch.arange(x.shape[0], device=x.device)
        caches[0][rows, lens.long()] = k
        caches[1][rows, lens.long()] = v
        lens = lens + 1
        attended = qmm.qmm_attn_decode(q, caches[0], caches[1], lens, prefix_k=prefix[0], prefix_v=prefix[1])
        return self.output(attended), attended, q, lens


class PagedAttentionLayer(AttentionLayer):
    """The same layer over a paged cache (qmm.KVPages) whose table int32 [requests, pages] says where each
    request's tokens lie."""

    def slots(self, cache, table, rows, positions):
        """Places in the cache of tokens at `positions` of the requests `rows`."""
        page = table[rows, (positions // cache.page_size).long()]
        return page * cache.page_size + positions % cache.page_size

    def chunk(self, x, cache, table, cu_q, cu_k):
        """The next tokens of every request, packed (bounds cu_q), after which the requests hold the tokens of the
        bounds cu_k: into the cache, then attention over all that each holds."""
        m = x.shape[0]
        at = torch.arange(m, device=x.device)
        rows = torch.searchsorted(cu_q, at.to(torch.int32), right=True) - 1
        held = cu_k.diff()[rows]
        positions = (held - cu_q[rows + 1] + at).to(torch.int32)
        q, k, v = self.project(x)
        q, _, _ = qmm.qmm_kv_append(q, k, v, positions, self.inv_freq, cache, self.slots(cache, table, rows, positions),
                                    w_q=self.norm_q, w_k=self.norm_k, out_dtype=self.dtype)
        k, v = qmm.qmm_kv_read(cache, table, cu_k, int(cu_k[-1]), out_dtype=self.dtype)
        attended = qmm.qmm_attn_prompt(q, k, v, cu_q, cu_k)
        return self.output(attended), attended, q

    def step(self, x, cache, table, lens, max_len):
        """One token of each request after its lens tokens, which become lens + 1 (at most max_len)."""
        rows = torch.arange(x.shape[0], device=x.device)
        q, k, v = self.project(x)
        q, _, _ = qmm.qmm_kv_append(q, k, v, lens, self.inv_freq, cache, self.slots(cache, table, rows, lens),
                                    w_q=self.norm_q, w_k=self.norm_k, out_dtype=self.dtype)
        lens = lens + 1
        attended = qmm.qmm_attn_decode_kv(q, cache, table, lens, max_len=max_len)
        return self.output(attended), attended, q, lens


def main(prefix_tokens=4096, batch=16, room=64, steps=4):
    layer = AttentionLayer()
    g = torch.Generator(device="cuda:0").manual_seed(1)
    x = torch.randn(prefix_tokens, layer.hidden, generator=g, device="cuda:0")
    cu = torch.tensor([0, prefix_tokens], dtype=torch.int32, device="cuda:0")
    caches = tuple(torch.zeros(batch, room, layer.kv_heads, layer.dim, dtype=layer.dtype, device="cuda:0") for _ in range(2))
    lens = torch.arange(batch, device="cuda:0", dtype=torch.int32) % 5

    def timed(what, call):
        call()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out = call()
        b.record()
        torch.cuda.synchronize()
        print(f"{what}: {a.elapsed_time(b) * 1e3:.0f} us")
        return out

    _, _, (_, k, v) = timed(f"prefill of {prefix_tokens} tokens", lambda: layer.prefill(x, cu))
    for i in range(steps):
        token = torch.randn(batch, layer.hidden, generator=g, device="cuda:0")
        y, _, _, lens = timed(f"step {i} of {batch} requests", lambda: layer.step(token, (k, v), caches, lens))
    paged, prompt, page = PagedAttentionLayer(), 512, 64
    cache = qmm.KVPages.empty(batch * 10, "q4_0", page, paged.kv_heads, paged.dim, device="cuda:0")
    table = torch.randperm(batch * 10, generator=g, device="cuda:0").to(torch.int32).view(batch, 10)
    x = torch.randn(batch * prompt, paged.hidden, generator=g, device="cuda:0")
    cu = torch.arange(0, batch * prompt + 1, prompt, device="cuda:0", dtype=torch.int32)
    timed(f"{batch} prompts of {prompt} tokens into pages", lambda: paged.chunk(x, cache, table, cu, cu))
    lens = torch.full((batch,), prompt, device="cuda:0", dtype=torch.int32)
    for i in range(steps):
        token = torch.randn(batch, paged.hidden, generator=g, device="cuda:0")
        y, _, _, lens = timed(f"paged step {i} of {batch} requests",
                              lambda: paged.step(token, cache, table, lens, prompt + steps))
    if qmm.qmm_take_attn_error():
        raise RuntimeError("an attention call gave up, or met a page outside the cache: its output is unspecified")
    print("finite:", bool(torch.isfinite(y).all()))


if __name__ == "__main__":
    main()
