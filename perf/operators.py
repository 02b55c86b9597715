"""Cases for the attention operators: the norm and rotation of queries and keys, attention over
packed prompts, and attention of a decoding batch over a shared prefix and its own caches.

With `own` false, `run` computes them in their plain form from elementary torch operations in
fp32; with `own` true it calls the library.  `exact` is the same in fp64, written apart.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of one request: the per-layer latency of decoding
        {"name": "rope_one_token", "op": "rope", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "input": "f32", "type": "bf16", "max_position": 8192},
        # a prefill chunk whose qkv product comes in fp32 from the quantized projection
        {"name": "rope_prompt_8192", "op": "rope", "tokens": 8192, "heads": 40, "kv_heads": 8, "dim": 128,
         "rotary": 128, "interleaved": False, "input": "f32", "type": "bf16", "max_position": 32768},
        # an odd token count, small heads, half of each head rotated in adjacent pairs, 16-bit input
        {"name": "rope_odd_partial", "op": "rope", "tokens": 4100, "heads": 32, "kv_heads": 32, "dim": 64, "rotary": 32,
         "interleaved": True, "input": "f16", "type": "f16", "max_position": 4096},
        # one short prompt: a chat turn with an empty cache
        {"name": "prompt_37", "op": "prompt", "seqs": 1, "max_q": 37, "history": 0, "lens": 1, "heads": 32,
         "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16"},
        # a batch of prompts of ragged lengths, packed
        {"name": "prompt_ragged_24", "op": "prompt", "seqs": 24, "max_q": 2048, "history": 0, "lens": 2, "heads": 32,
         "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16"},
        # one long document
        {"name": "prompt_8192", "op": "prompt", "seqs": 1, "max_q": 8192, "history": 0, "lens": 3, "heads": 32,
         "kv_heads": 8, "dim": 128, "causal": True, "type": "bf16"},
        # chunks of prompts whose first part is already in the cache, small heads, one kv head per query head
        {"name": "prompt_chunks_history", "op": "prompt", "seqs": 5, "max_q": 509, "history": 3500, "lens": 4,
         "heads": 32, "kv_heads": 32, "dim": 64, "causal": True, "type": "f16"},
        # one request decoding on its own
        {"name": "decode_one", "op": "decode", "batch": 1, "prefix": 0, "room": 640, "lens": 5, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16"},
        # a batch without a common prefix, ragged caches
        {"name": "decode_ragged_48", "op": "decode", "batch": 48, "prefix": 0, "room": 8192, "lens": 6, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16"},
        # a few requests with a short system prompt, one kv head per query head, odd sizes
        {"name": "decode_prefix_small", "op": "decode", "batch": 7, "prefix": 1001, "room": 130, "lens": 7, "heads": 16,
         "kv_heads": 16, "dim": 64, "type": "f16"},
        # a batch that shares a long system prompt
        {"name": "decode_prefix_64", "op": "decode", "batch": 64, "prefix": 8192, "room": 512, "lens": 8, "heads": 32,
         "kv_heads": 8, "dim": 128, "type": "bf16"},
        # many samples of one long document
        {"name": "decode_prefix_256", "op": "decode", "batch": 256, "prefix": 32768, "room": 1000, "lens": 9,
         "heads": 40, "kv_heads": 8, "dim": 128, "type": "f16"},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads, kv_heads = rng.choice([(32, 8), (40, 8), (16, 16), (32, 32), (28, 4), (16, 4), (8, 1), (12, 2), (32, 2)])
    dim = rng.choice([64, 64, 80, 128, 128, 128])
    kind = rng.choice(["bf16", "bf16", "f16"])
    op = rng.choice(["rope", "prompt", "prompt", "decode", "decode"])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "type": kind}
    if op == "rope":
        if (heads + 2 * kv_heads) * dim == 3072:  # a width that no configuration here has
            case["dim"] = dim = 80
        rotary = rng.choice([dim, dim, dim // 2])
        case |= {"tokens": _log_int(rng, 1, 8192), "rotary": rotary, "interleaved": rng.random() < 0.4,
                 "input": rng.choice(["f32", "f32", kind]), "max_position": _log_int(rng, 1000, 32768)}
    elif op == "prompt":
        seqs = _log_int(rng, 1, 32)
        # the plain form holds seqs x heads x queries x keys scores: no more than the largest listed case
        most = int((32 * 8192 * 8192 / (seqs * heads)) ** 0.5)
        max_q = _log_int(rng, 1, min(8192, most))
        room = min(8192, most * most // max_q - max_q)
        history = 0 if rng.random() < 0.6 or room < 1 else _log_int(rng, 1, room)
        case |= {"seqs": seqs, "max_q": max_q, "history": history, "lens": rng.randrange(1000),
                 "causal": rng.random() < 0.8}
    else:
        batch = _log_int(rng, 1, 256)
        prefix = 0 if rng.random() < 0.3 else _log_int(rng, 1, 32768)
        room = _log_int(rng, 1, min(8192, 48 * 8192 * 8 // (batch * kv_heads)))
        case |= {"batch": batch, "prefix": prefix, "room": room, "lens": rng.randrange(1000)}
    return case


def _lengths(case):
    """Ragged lengths, the same for every seed: (queries, keys) of each prompt, or each cache's length."""
    r = random.Random(case["lens"])
    if case["op"] == "prompt":
        n = case["seqs"]
        q = [max(1, int(case["max_q"] * r.random() ** 1.5)) for _ in range(n)]
        q[r.randrange(n)] = case["max_q"]
        return q, [a + (r.randint(0, case["history"]) if case["history"] else 0) for a in q]
    n = case["batch"]
    lens = [r.randint(0 if case["prefix"] else 1, case["room"]) for _ in range(n)]
    lens[r.randrange(n)] = case["room"]
    return lens


# ------------------------------------------------------------------------------ inputs
def _unit(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[case["type"]]
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def heads_of(*shape):  # queries and keys as they leave the norm
        return _unit(normal(*shape)).to(dt)

    if case["op"] == "rope":
        m = case["tokens"]
        qkv = normal(m, (H + 2 * Hk) * D).mul_(0.5).to(TYPES[case["input"]])  # one fused projection's product
        start = torch.randint(0, case["max_position"], (1,), generator=g, device=DEV)
        r = case["rotary"]
        return {"case": case, "q": qkv[:, :H * D].view(m, H, D), "k": qkv[:, H * D:(H + Hk) * D].view(m, Hk, D),
                "v": qkv[:, (H + Hk) * D:].view(m, Hk, D),
                "positions": ((start + torch.arange(m, device=DEV)) % case["max_position"]).to(torch.int32),
                "inv_freq": (THETA ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)).float(),
                "w_q": 1 + 0.1 * normal(D), "w_k": 1 + 0.1 * normal(D)}
    if case["op"] == "prompt":
        lq, lk = _lengths(case)

        def bounds(lens):
            return torch.cat([torch.zeros(1, dtype=torch.int64), torch.tensor(lens).cumsum(0)]).to(torch.int32).to(DEV)

        return {"case": case, "q": heads_of(sum(lq), H, D), "k": heads_of(sum(lk), Hk, D),
                "v": normal(sum(lk), Hk, D).to(dt), "cu_q": bounds(lq), "cu_k": bounds(lk), "max_q": max(lq),
                "max_k": max(lk)}
    B, P, S = case["batch"], case["prefix"], case["room"]
    return {"case": case, "q": heads_of(B, H, D), "k": heads_of(B, S, Hk, D), "v": normal(B, S, Hk, D).to(dt),
            "lens": torch.tensor(_lengths(case), dtype=torch.int32, device=DEV),
            "prefix_k": heads_of(P, Hk, D) if P else None, "prefix_v": normal(P, Hk, D).to(dt) if P else None}


# ------------------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if not own:
        return {"rope": _plain_rope, "prompt": _plain_prompt, "decode": _plain_decode}[case["op"]](state)
    import block_quantized_matmul_q8_gb300 as qmm
    if case["op"] == "rope":
        return qmm.qmm_qk_norm_rope(state["q"], state["k"], state["v"], state["positions"], state["inv_freq"],
                                    w_q=state["w_q"], w_k=state["w_k"], eps=EPS, interleaved=case["interleaved"],
                                    out_dtype=TYPES[case["type"]])
    if case["op"] == "prompt":
        return qmm.qmm_attn_prompt(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"],
                                   causal=case["causal"])
    return qmm.qmm_attn_decode(state["q"], state["k"], state["v"], state["lens"], prefix_k=state["prefix_k"],
                               prefix_v=state["prefix_v"])


def _plain_rope(s):
    case, dt = s["case"], TYPES[s["case"]["type"]]
    r = case["rotary"]
    angle = s["positions"].float()[:, None] * s["inv_freq"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def rotated(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1 if case["interleaved"] else -2).flatten(-2)
        return torch.cat((y, x[..., r:]), -1).to(dt)

    return rotated(s["q"], s["w_q"]), rotated(s["k"], s["w_k"]), s["v"].to(dt)


def _softmax_rows(scores):
    """exp of each row less its maximum, in place, and the rows' sums; a row of -inf alone gives zeros."""
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = scores.sum(-1, keepdim=True)
    return scores, torch.where(total == 0, torch.ones_like(total), total)


def _plain_prompt(s):
    q, k, v, cu_q, cu_k = s["q"], s["k"], s["v"], s["cu_q"].long(), s["cu_k"].long()
    T, H, D = q.shape
    Hk = k.shape[1]
    n, Lq, Lk = cu_q.numel() - 1, s["max_q"], s["max_k"]
    iq, ik = torch.arange(Lq, device=q.device), torch.arange(Lk, device=q.device)
    nq, nk = cu_q.diff()[:, None], cu_k.diff()[:, None]
    inside = ik < nk
    qp = q[(cu_q[:-1, None] + iq).clamp_(max=T - 1)].float()
    at = (cu_k[:-1, None] + ik).clamp_(max=k.shape[0] - 1)
    kp, vp = k[at].float(), v[at].float().mul_(inside[..., None, None])
    qp = qp.view(n, Lq, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(n, Hk, -1, D)
    scores = (qp @ kp.permute(0, 2, 3, 1)).mul_(D ** -0.5).view(n, H, Lq, Lk)
    seen = inside[:, None, :]
    if s["case"]["causal"]:
        seen = seen & (ik <= iq[:, None] + (nk - nq)[..., None])
    scores.masked_fill_(~seen[:, None], -math.inf)
    p, total = _softmax_rows(scores)
    out = (p.view(n, Hk, -1, Lk) @ vp.permute(0, 2, 1, 3)).view(n, H, Lq, D) / total
    token = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu_q, token, right=True) - 1
    return out[seq, :, token - cu_q[seq]].to(q.dtype)


def _plain_decode(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, H, D = q.shape
    S, Hk = k.shape[1], k.shape[2]
    G = H // Hk
    inside = torch.arange(S, device=q.device) < s["lens"][:, None]
    qf = q.float().view(B, Hk, G, D).mul(D ** -0.5)
    scores = (qf @ k.float().permute(0, 2, 3, 1)).masked_fill_(~inside[:, None, None], -math.inf)
    if s["prefix_k"] is None:
        p, total = _softmax_rows(scores)
        out = p @ v.float().mul_(inside[..., None, None]).transpose(1, 2)
    else:
        P = s["prefix_k"].shape[0]
        shared = qf.transpose(0, 1).reshape(Hk, B * G, D) @ s["prefix_k"].float().permute(1, 2, 0)
        p, total = _softmax_rows(torch.cat((shared.view(Hk, B, G, P).transpose(0, 1), scores), -1))
        out = p[..., P:] @ v.float().mul_(inside[..., None, None]).transpose(1, 2)
        shared = p[..., :P].transpose(0, 1).reshape(Hk, B * G, P) @ s["prefix_v"].float().transpose(0, 1)
        out = out + shared.view(Hk, B, G, D).transpose(0, 1)
    return (out / total).view(B, H, D).to(q.dtype)


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        size = 4 if case["input"] == "f32" else 2
        m = case["tokens"]
        return {"bytes": m * ((H + 2 * Hk) * D * (size + 2) + 4) + 8 * D + 2 * case["rotary"],
                "flops": m * (H + Hk) * (4 * D + 3 * case["rotary"])}
    if case["op"] == "prompt":
        lq, lk = _lengths(case)
        pairs = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(lq, lk))
        return {"bytes": 2 * D * (2 * H * sum(lq) + 2 * Hk * sum(lk)) + 8 * (case["seqs"] + 1),
                "flops": 4 * D * H * pairs}
    lens = _lengths(case)
    B, P = case["batch"], case["prefix"]
    return {"bytes": 2 * D * (2 * H * B + 2 * Hk * (P + sum(lens))) + 4 * B, "flops": 4 * D * H * (B * P + sum(lens))}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // Hk

    def attend(q, k, v, hidden=None):
        """softmax(q k^T / sqrt(D)) v of one kv head's rows q [rows][D], in 64 bits."""
        z = torch.matmul(q.double(), k.double().t()) / math.sqrt(D)
        if hidden is not None:
            z[hidden] = -math.inf
        z -= z.max(dim=1, keepdim=True).values
        z.exp_()
        return torch.matmul(z, v.double()) / z.sum(dim=1, keepdim=True)

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    if case["op"] == "prompt":
        a = b = 0
        for lq, lk in zip(*_lengths(case)):
            hidden = None
            if case["causal"]:  # query i sees the keys up to i + (lk - lq)
                hidden = torch.ones(lq, lk, dtype=torch.bool, device=DEV).triu(lk - lq + 1)
            for h in range(H):
                out[a:a + lq, h] = attend(s["q"][a:a + lq, h], s["k"][b:b + lk, h // G], s["v"][b:b + lk, h // G],
                                          hidden)
            a, b = a + lq, b + lk
        return out
    for i, n in enumerate(_lengths(case)):
        for h in range(Hk):
            k, v = s["k"][i, :n, h], s["v"][i, :n, h]
            if case["prefix"]:
                k, v = torch.cat((s["prefix_k"][:, h], k)), torch.cat((s["prefix_v"][:, h], v))
            out[i, h * G:(h + 1) * G] = attend(s["q"][i, h * G:(h + 1) * G], k, v)
    return out


def _exact_rope(case, s):
    r = case["rotary"]
    first = torch.arange(0, r, 2, device=DEV) if case["interleaved"] else torch.arange(r // 2, device=DEV)
    second = first + (1 if case["interleaved"] else r // 2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * s["inv_freq"].double())

    def rotated(x, w):
        y = x.double()
        y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS).sqrt() * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    return rotated(s["q"], s["w_q"]), rotated(s["k"], s["w_k"]), s["v"].double()
