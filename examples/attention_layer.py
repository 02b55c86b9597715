"""One attention layer of a decoder on the library's calls: a quantized qkv projection, the norm and
rotation of its heads, attention, and a quantized output projection, for packed prompts and for a
decoding batch that shares one long prefix.

    python examples/attention_layer.py

prints the time of each call for a prefix of 4096 tokens, 16 requests and a few steps.
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

    def qkv(self, x, positions):
        """x fp32 [tokens, hidden] -> q [tokens, heads, dim], k and v [tokens, kv_heads, dim], normed and rotated."""
        y = qmm.qmm_mul_mat_f32(self.w_qkv, self.fmt, self.width, self.hidden, x, x.shape[0])
        h = y.view(x.shape[0], -1, self.dim)
        q, k, v = h[:, :self.heads], h[:, self.heads:self.heads + self.kv_heads], h[:, self.heads + self.kv_heads:]
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
    if qmm.qmm_take_attn_error():
        raise RuntimeError("an attention call gave up: its output is unspecified")
    print("finite:", bool(torch.isfinite(y).all()))


if __name__ == "__main__":
    main()
