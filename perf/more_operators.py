"""Cases for the paged key/value cache held in 4 or 8 bits: appending tokens with the norm and rotation
of their heads, attention of a decoding batch over its pages, and reading sequences back in 16 bits.

With `own` false, `run` computes them in their plain form from elementary torch operations; with
`own` true it calls the library.  `exact` is the same in fp64, written apart.

A page holds, for each kv head and each group of 16 tokens, one record: the key codes as
[16-byte unit][token][16 bytes], the key scales as fp16 [block of 32][token pair], then the same of the values.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
THETA = 10000.0
# place of token 0..15 of a group among the scales of a block: tokens 2t, 2t + 1, 2t + 8, 2t + 9 together
PLACE = [(t % 8) // 2 * 4 + t % 2 + 2 * (t // 8) for t in range(16)]


# ------------------------------------------------------------------------------ cases
def listed():
    gqa = {"heads": 32, "kv_heads": 8, "dim": 128}
    return [
        # one new token of one request: the per-layer latency of decoding
        {"name": "append_one", "op": "append", **gqa, "type": "bf16", "cache": "q4_0", "page": 16, "tokens": 1, "lens": 1,
         "rotary": 128, "interleaved": False, "input": "f32", "max_position": 8192},
        # one token of each request of an odd batch, half of each head rotated in adjacent pairs, 16-bit input
        {"name": "append_batch_77", "op": "append", "heads": 28, "kv_heads": 4, "dim": 128, "type": "f16", "cache": "q8_0",
         "page": 32, "tokens": 77, "lens": 2, "rotary": 64, "interleaved": True, "input": "f16", "max_position": 30000},
        # a prefill chunk whose qkv product comes in fp32 from the quantized projection
        {"name": "append_chunk_2048", "op": "append", **gqa, "type": "bf16", "cache": "q4_0", "page": 64, "tokens": 2048,
         "lens": 3, "rotary": 128, "interleaved": False, "input": "f32", "max_position": 32768},
        # one request decoding on its own
        {"name": "decode_one_640", "op": "decode", **gqa, "type": "bf16", "cache": "q4_0", "page": 16, "batch": 1,
         "room": 640, "lens": 4},
        # a batch of ragged lengths
        {"name": "decode_ragged_48", "op": "decode", **gqa, "type": "bf16", "cache": "q4_0", "page": 64, "batch": 48,
         "room": 8192, "lens": 5},
        # small heads with a kv head each, 8 bits, odd lengths
        {"name": "decode_small_heads_35", "op": "decode", "heads": 16, "kv_heads": 16, "dim": 64, "type": "f16",
         "cache": "q8_0", "page": 32, "batch": 35, "room": 1001, "lens": 6},
        # one long document in 4 bits
        {"name": "decode_long_131071", "op": "decode", "heads": 40, "kv_heads": 8, "dim": 128, "type": "f16",
         "cache": "q4_0", "page": 256, "batch": 1, "room": 131071, "lens": 7},
        # a full serving batch
        {"name": "decode_batch_128", "op": "decode", **gqa, "type": "bf16", "cache": "q4_0", "page": 16, "batch": 128,
         "room": 8192, "lens": 8},
        # a decoding step: the new tokens go into the cache, and attention reads them with the others
        {"name": "step_64", "op": "step", **gqa, "type": "bf16", "cache": "q4_0", "page": 64, "batch": 64, "room": 2048,
         "lens": 9, "rotary": 128, "interleaved": False, "input": "f32"},
        # a short history for the next chunk of one prompt
        {"name": "read_one_297", "op": "read", **gqa, "type": "bf16", "cache": "q4_0", "page": 16, "seqs": 1, "room": 297,
         "lens": 10},
        # histories of several prompts, ragged, 8 bits
        {"name": "read_ragged_11", "op": "read", "heads": 12, "kv_heads": 2, "dim": 96, "type": "f16", "cache": "q8_0",
         "page": 32, "seqs": 11, "room": 5003, "lens": 11},
        # the history of one long document
        {"name": "read_32768", "op": "read", **gqa, "type": "bf16", "cache": "q4_0", "page": 128, "seqs": 1, "room": 32768,
         "lens": 12},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads, kv_heads = rng.choice([(32, 8), (40, 8), (16, 16), (32, 32), (28, 4), (16, 4), (8, 1), (12, 2), (32, 2)])
    dim = rng.choice([32, 64, 64, 96, 128, 128, 128])
    op = rng.choice(["append", "append", "decode", "decode", "decode", "step", "read", "read"])
    kind = rng.choice(["bf16", "bf16", "f16"])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "type": kind,
            "cache": rng.choice(["q4_0", "q4_0", "q8_0"]), "page": rng.choice([16, 16, 32, 64, 128, 256]),
            "lens": rng.randrange(1000)}
    if op in ("append", "step"):
        case |= {"rotary": rng.choice([dim, dim, dim // 2]), "interleaved": rng.random() < 0.4,
                 "input": rng.choice(["f32", "f32", kind])}
    # the plain form holds a request's keys at the batch's longest length: no more than the largest listed case
    most = 128 * 8192 * 8 // kv_heads
    if op == "append":
        case |= {"tokens": _log_int(rng, 1, 2048), "max_position": _log_int(rng, 1000, 32768)}
    elif op == "read":
        seqs = _log_int(rng, 1, 32)
        case |= {"seqs": seqs, "room": _log_int(rng, 1, min(32768, 32768 * 8 // (seqs * kv_heads)))}
    else:
        batch = _log_int(rng, 1, 256)
        case |= {"batch": batch, "room": _log_int(rng, 1, min(131072, most // batch))}
    return case


def _lengths(case):
    """Ragged lengths, the same for every seed: of each request's or sequence's tokens, the longest fills the room."""
    r = random.Random(case["lens"])
    n = case["batch"] if "batch" in case else case["seqs"]
    lens = [r.randint(1, case["room"]) for _ in range(n)]
    lens[r.randrange(n)] = case["room"]
    return lens


# ------------------------------------------------------------------------------ the cache
def _units(case):
    """(16-byte units of codes, blocks of 32, bytes of a record) of one token's head."""
    units, blocks = case["dim"] // (32 if case["cache"] == "q4_0" else 16), case["dim"] // 32
    return units, blocks, 2 * (units * 256 + blocks * 32)


def _parts(case, pages):
    """Views of pages [n, page_bytes]: codes and scales of keys, of values, as [n, kv head, group, ...]."""
    units, blocks, record = _units(case)
    rec = pages.view(pages.shape[0], case["kv_heads"], case["page"] // 16, record)
    at, out = 0, []
    for _ in range(2):
        out.append(rec[..., at:at + units * 256].unflatten(-1, (units, 16, 16)))
        out.append(rec[..., at + units * 256:at + units * 256 + blocks * 32].view(torch.float16).unflatten(-1, (blocks, 16)))
        at += units * 256 + blocks * 32
    return out


def _quantize(case, x):
    """x [..., dim] -> (bytes [..., units, 16], scales fp16 [..., blocks], values fp32 [..., dim])."""
    x = x.unflatten(-1, (-1, 32))
    if case["cache"] == "q4_0":
        top, low = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
        d, lo, hi = torch.where(top >= -low, top, low) / -8, -8, 7
    else:
        d, lo, hi = x.abs().amax(-1, keepdim=True) / 127, -127, 127
    d = d.clamp(-65504, 65504).half()
    code = torch.where(d == 0, 0, x / d.to(x.dtype)).round().clamp_(lo, hi)
    value = (code.float() * d.float()).flatten(-2)
    if case["cache"] == "q4_0":
        code = (code + 8).to(torch.uint8)
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    else:
        code = (code + 128).to(torch.uint8).unflatten(-1, (2, 16)).flatten(-3, -2)
    return code, d.squeeze(-1), value


def _write(case, pages, slots, k, v):
    """The quantized heads k, v of some tokens into their slots."""
    kc, ks, vc, vs = _parts(case, pages)
    place = torch.tensor(PLACE, device=pages.device)
    page, group, token = slots // case["page"], slots % case["page"] // 16, slots % 16
    for codes, scales, (c, d, _) in ((kc, ks, k), (vc, vs, v)):
        codes[page, :, group, :, token] = c
        scales[page, :, group, :, place[token]] = d


def _pages_for(case, lens, g):
    """A cache with the sequences' pages in mixed order and some pages of others: (pages, table)."""
    size, D, Hk = case["page"], case["dim"], case["kv_heads"]
    need = [-(-n // size) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    width = max(need)
    at = torch.tensor([0] + need, device=DEV).cumsum(0)[:-1, None] + torch.arange(width, device=DEV)
    used = torch.arange(width, device=DEV) < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(used, order[at.clamp_(max=n_pages - 1)], -1).to(torch.int32)
    pages = torch.empty((n_pages, Hk * (size // 16) * _units(case)[2]), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (size * Hk * D))
    places = torch.tensor(PLACE, device=DEV)
    for a in range(0, n_pages, step):  # every slot holds a token, of these sequences or of earlier ones
        part = pages[a:a + step]
        kc, ks, vc, vs = _parts(case, part)
        for codes, scales, unit in ((kc, ks, True), (vc, vs, False)):
            x = torch.randn(part.shape[0], Hk, size // 16, 16, D, generator=g, device=DEV)
            c, d, _ = _quantize(case, _unit(x) if unit else x)
            codes.copy_(c.transpose(-3, -2))
            scales[..., places] = d.transpose(-2, -1)
    return pages, table


# ------------------------------------------------------------------------------ inputs
def _unit(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    H, Hk, D, op = case["heads"], case["kv_heads"], case["dim"], case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = {"case": case}
    if op == "append":
        m, size = case["tokens"], case["page"]
        first = int(random.Random(case["lens"]).random() * size)  # the sequence ends inside a page before
        n_pages = (first + m + size - 1) // size + 2
        order = torch.randperm(n_pages, generator=g, device=DEV)
        at = first + torch.arange(m, device=DEV)
        s |= {"pages": torch.zeros((n_pages, Hk * (size // 16) * _units(case)[2]), dtype=torch.uint8, device=DEV),
              "slots": (order[at // size] * size + at % size).to(torch.int32)}
        start = torch.randint(0, case["max_position"], (1,), generator=g, device=DEV)
        s["positions"] = ((start + torch.arange(m, device=DEV)) % case["max_position"]).to(torch.int32)
    else:
        lens = _lengths(case)
        s["pages"], s["table"] = _pages_for(case, lens, g)
        if op == "read":
            s["tokens"] = sum(lens)
            s["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        else:
            m = case["batch"]
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        if op == "step":  # each request's last token is the new one
            s["positions"] = s["lens"] - 1
            last = s["positions"].long()
            s["slots"] = (s["table"][torch.arange(m, device=DEV), last // case["page"]] * case["page"]
                          + last % case["page"]).to(torch.int32)
    if op == "decode":
        s["q"] = _unit(normal(m, H, D)).to(TYPES[case["type"]])
    if op in ("append", "step"):
        qkv = normal(m, (H + 2 * Hk) * D).mul_(0.5).to(TYPES[case["input"]])  # one fused projection's product
        r = case["rotary"]
        s |= {"q": qkv[:, :H * D].view(m, H, D), "k": qkv[:, H * D:(H + Hk) * D].view(m, Hk, D),
              "v": qkv[:, (H + Hk) * D:].view(m, Hk, D),
              "inv_freq": (THETA ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)).float(),
              "w_q": 1 + 0.1 * normal(D), "w_k": 1 + 0.1 * normal(D)}
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "step": _plain_step, "read": _plain_read}[case["op"]](s)
    import block_quantized_matmul_q8_gb300 as qmm
    if "handle" not in s:  # a program describes its cache once
        s["handle"] = qmm.KVPages(s["pages"], case["cache"], case["page"], case["kv_heads"], case["dim"])
    cache = s["handle"]
    kind = TYPES[case["type"]]
    if case["op"] == "read":
        return qmm.qmm_kv_read(cache, s["table"], s["cu"], s["tokens"], out_dtype=kind)
    if case["op"] == "decode":
        return qmm.qmm_attn_decode_kv(s["q"], cache, s["table"], s["lens"], max_len=case["room"])
    new = qmm.qmm_kv_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], cache, s["slots"], w_q=s["w_q"],
                            w_k=s["w_k"], eps=EPS, interleaved=case["interleaved"], out_dtype=kind,
                            values=case["op"] == "append")
    if case["op"] == "append":
        return new
    return new[0], qmm.qmm_attn_decode_kv(new[0], cache, s["table"], s["lens"], max_len=case["room"])


def _plain_append(s):
    case, dt = s["case"], TYPES[s["case"]["type"]]
    r = case["rotary"]
    # in 64 bits: the angles of far positions, and keys next to the border between two codes
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def rotated(x, w):
        x = x.double()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1 if case["interleaved"] else -2).flatten(-2)
        return torch.cat((y, x[..., r:]), -1)

    k, v = _quantize(case, rotated(s["k"], s["w_k"])), _quantize(case, s["v"].float())
    _write(case, s["pages"], s["slots"].long(), k, v)
    return rotated(s["q"], s["w_q"]).float().to(dt), k[2].to(dt), v[2].to(dt)


def _values(case, codes, scales):
    """fp32 [..., 16 tokens, dim] of gathered codes [..., units, 16, 16] and scales [..., blocks, 16]."""
    c = codes.transpose(-3, -2)
    if case["cache"] == "q4_0":
        c = torch.stack((c & 15, c >> 4), -1).flatten(-3).float().sub_(8)
    else:
        c = c.flatten(-2).float().sub_(128)
    place = torch.tensor(PLACE, device=codes.device)
    return c.unflatten(-1, (-1, 32)).mul_(scales[..., place].transpose(-2, -1).float()[..., None]).flatten(-2)


def _gather(case, pages, table):
    """fp32 keys and values [sequence, kv head, table width * page, dim]."""
    at = table.long().clamp(min=0)
    kc, ks, vc, vs = (x[at].transpose(1, 2) for x in _parts(case, pages))
    return _values(case, kc, ks).flatten(2, 4), _values(case, vc, vs).flatten(2, 4)


def _plain_decode(s, q=None):
    case, q = s["case"], s["q"] if q is None else q
    B, H, D = q.shape
    Hk, S = case["kv_heads"], case["room"]
    k, v = _gather(case, s["pages"], s["table"])
    k, v = k[:, :, :S], v[:, :, :S]
    inside = (torch.arange(S, device=q.device) < s["lens"][:, None])[:, None]
    scores = (q.float().view(B, Hk, H // Hk, D) @ k.transpose(-1, -2)).mul_(D ** -0.5)
    scores.masked_fill_(~inside[:, :, None], -math.inf)
    p = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    return ((p @ v) / total).view(B, H, D).to(q.dtype)


def _plain_step(s):
    q = _plain_append(s)[0]
    return q, _plain_decode(s, q)


def _plain_read(s):
    case, cu = s["case"], s["cu"].long()
    k, v = _gather(case, s["pages"], s["table"])
    token = torch.arange(s["tokens"], device=cu.device)
    seq = torch.searchsorted(cu, token, right=True) - 1
    return tuple(x[seq, :, token - cu[seq]].to(TYPES[case["type"]]) for x in (k, v))


# ------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    H, Hk, D, op = case["heads"], case["kv_heads"], case["dim"], case["op"]
    held = Hk * _units(case)[2] // 16  # bytes of a token in the cache
    new = keys = 0
    flops = moved = 0
    if op in ("append", "step"):
        new = case["tokens"] if op == "append" else case["batch"]
        size = 4 if case["input"] == "f32" else 2
        moved += new * ((H + 2 * Hk) * D * size + 2 * H * D + held + 8 + (4 * Hk * D if op == "append" else 0))
        moved += 8 * D + 2 * case["rotary"]
        flops += new * ((H + Hk) * (4 * D + 3 * case["rotary"]) + 8 * Hk * D)
    if op in ("decode", "step"):
        lens, B = _lengths(case), case["batch"]
        keys = sum(lens)
        moved += keys * held + 4 * B * H * D + 4 * B + 4 * sum(-(-n // case["page"]) for n in lens)
        flops += 4 * D * H * keys
    if op == "read":
        lens = _lengths(case)
        keys = sum(lens)
        moved += keys * (held + 4 * Hk * D) + 4 * (len(lens) + 1) + 4 * sum(-(-n // case["page"]) for n in lens)
        flops += 4 * Hk * D * keys
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)[0]
    lens = _lengths(case)
    pages = s["pages"]
    if case["op"] == "read":
        both = [_exact_sequence(case, pages, s["table"][i], n) for i, n in enumerate(lens)]
        return tuple(torch.cat([x[j] for x in both]) for j in range(2))
    q, new = s["q"], None
    if case["op"] == "step":
        (q, _, _), new = _exact_append(case, s)
        q_seen = q.to(TYPES[case["type"]]).double()  # attention takes the rounded queries
    else:
        q_seen = q.double()
    H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // Hk
    out = torch.empty((len(lens), H, D), dtype=torch.float64, device=DEV)
    for i, n in enumerate(lens):
        k, v = _exact_sequence(case, pages, s["table"][i], n)
        if new is not None:
            k[n - 1], v[n - 1] = new[0][i], new[1][i]
        z = torch.einsum("hgd,nhd->hgn", q_seen[i].view(Hk, G, D), k) / math.sqrt(D)
        out[i] = torch.einsum("hgn,nhd->hgd", z.softmax(-1), v).reshape(H, D)
    return (q, out) if case["op"] == "step" else out


def _exact_sequence(case, pages, row, n):
    """fp64 keys and values [n, kv head, dim] of one sequence, byte by byte from the layout."""
    size, D, Hk = case["page"], case["dim"], case["kv_heads"]
    four = case["cache"] == "q4_0"
    unit, record = (32 if four else 16), _units(case)[2]
    token = torch.arange(n, device=DEV)[:, None, None]
    head, e = torch.arange(Hk, device=DEV)[:, None], torch.arange(D, device=DEV)
    slot = token % size
    base = (row.long()[token // size] * Hk + head) * (size // 16) * record + slot // 16 * record
    t = slot % 16
    flat, halves = pages.flatten(), pages.flatten().view(torch.float16)
    code_at = e // unit * 256 + t * 16 + (e % unit // 2 if four else e % unit)
    scale_at = D // unit * 256 + e // 32 * 32 + 2 * (t % 8 // 2 * 4 + t % 2 + 2 * (t // 8))
    got = []
    for side in (0, record // 2):
        c = flat[base + side + code_at].long()
        c = torch.where(e % 2 == 0, c % 16, c // 16) - 8 if four else c - 128
        got.append(c.double() * halves[(base + side + scale_at) // 2].double())
    return got


def _exact_append(case, s):
    """((q, values of k, values of v), (values of k, values of v)) in fp64."""
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

    def held(x):
        b = x.reshape(*x.shape[:-1], -1, 32)
        big = b.abs().max(-1, keepdim=True).values
        if case["cache"] == "q4_0":
            d = torch.where((b == big).any(-1, keepdim=True), big, -big) / -8
            steps = (-8, 7)
        else:
            d, steps = big / 127, (-127, 127)
        d = d.half().double()
        c = torch.where(d == 0, torch.zeros_like(b), b / torch.where(d == 0, torch.ones_like(d), d))
        return (torch.round(c).clamp(*steps) * d).reshape(x.shape)

    k, v = held(rotated(s["k"], s["w_k"])), held(s["v"].double())
    return (rotated(s["q"], s["w_q"]), k, v), (k, v)
