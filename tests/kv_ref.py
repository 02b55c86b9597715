"""Plain references of the paged key/value cache in 4 and 8 bits: its bytes, its quantization, and attention
over it in fp64 with elementwise bounds derived from the formulas."""
import math

import torch

from attn_ref import TINY, U, check

BIAS = {"q4_0": 8, "q8_0": 128}


def sizes(qtype, d):
    """(elements of a 16-byte unit, bytes of a side's codes, bytes of a side, bytes of a record)"""
    unit = 32 if qtype == "q4_0" else 16
    codes = d // unit * 256
    side = codes + d // 32 * 32
    return unit, codes, side, 2 * side


def page_bytes(qtype, page, hk, d):
    return hk * (page // 16) * sizes(qtype, d)[3]


def _places(qtype, page, hk, d, slots, page_stride):
    """Byte offsets of a token's code of every element, and of its block scales: [2][m, hk, d], [2][m, hk, d / 32]."""
    unit, codes, side, record = sizes(qtype, d)
    s = slots.long()[:, None, None]
    h = torch.arange(hk, device=slots.device)[:, None]
    e, b = torch.arange(d, device=slots.device), torch.arange(d // 32, device=slots.device)
    t = s % 16
    base = s // page * page_stride + (h * (page // 16) + s % page // 16) * record
    at = base + e // unit * 256 + t * 16 + (e % 32 // 2 if qtype == "q4_0" else e % 16)
    place = t % 8 // 2 * 4 + t % 2 + t // 8 * 2
    scale = base + codes + b * 32 + place * 2
    return [at, at + side], [scale, scale + side]


def load(buf, qtype, page, hk, d, slots, page_stride=None):
    """What slots hold: codes int [2][m, hk, d] and scales fp16 [2][m, hk, d / 32], byte by byte."""
    flat = buf.flatten()
    at, scale = _places(qtype, page, hk, d, slots, page_stride or page_bytes(qtype, page, hk, d))
    codes, scales = [], []
    for a, s in zip(at, scale):
        c = flat[a].int()
        if qtype == "q4_0":
            c = torch.where(torch.arange(d, device=flat.device) % 2 == 0, c & 15, c >> 4)
        codes.append(c - BIAS[qtype])
        scales.append((flat[s].int() | flat[s + 1].int() << 8).to(torch.int16).view(torch.float16))
    return codes, scales


def store(buf, qtype, page, hk, d, slots, codes, scales, page_stride=None):
    """The inverse of load: writes the slots' bytes and no others."""
    flat = buf.view(-1)
    at, scale = _places(qtype, page, hk, d, slots, page_stride or page_bytes(qtype, page, hk, d))
    for a, s, c, v in zip(at, scale, codes, scales):
        c = c + BIAS[qtype]
        if qtype == "q4_0":
            flat[a[..., 0::2]] = (c[..., 0::2] | c[..., 1::2] << 4).to(torch.uint8)
        else:
            flat[a] = c.to(torch.uint8)
        bits = v.view(torch.int16).int()
        flat[s] = (bits & 255).to(torch.uint8)
        flat[s + 1] = (bits >> 8 & 255).to(torch.uint8)


def quantize(qtype, x):
    """x fp32 [..., d] -> (codes int32, scales fp16), in fp32 as the library defines it."""
    b = x.unflatten(-1, (-1, 32))
    b = torch.where(b.isnan(), torch.zeros_like(b), b)
    if qtype == "q4_0":
        top, low = b.amax(-1), b.amin(-1)
        d, lo, hi = torch.where(top >= -low, top, low) / -8, -8, 7
    else:
        d, lo, hi = b.abs().amax(-1) / 127, -127, 127
    d = d.clamp(-65504, 65504).half()
    df = d.float()[..., None]
    c = torch.where(df == 0, torch.zeros_like(b), b / df).round().clamp(lo, hi)
    return c.int().flatten(-2), d


def values(codes, scales):
    """fp64 values [..., d]."""
    return (codes.double().unflatten(-1, (-1, 32)) * scales.double()[..., None]).flatten(-2)


def check_decode_kv(q, codes, scales, lens, scale, qtype, out, lse=None):
    """q [B, H, d]; codes and scales [2][B] lists of [n, hk, ...] (each request's tokens); lens: how many of
    them count.  The bound:
      * the output is rounded once: u |out|;
      * weights: bf16 p is rounded to fp16 and so is its product with the scale, 2 2^-11; f16 the product
        alone, 2^-11; below fp16's normal range each rounding is off by 2^-25 (times scale and code, times
        code), with the largest weight of a row being 1;
      * a score: sums of d / 16 MMAs a key whose terms are at most |q| (15 + 8) scale-units in 4 bits,
        |q| (255 + 128) in 8, in fp32: ds = (d + 5) 2^-23 scale sum_b |d_b| sum |q| (15 + 8), which moves
        every weight by at most 2 ds; a query element below 2^-28 of the head's largest is off by 2^-34 of it,
        less than those terms;
      * exp, sums and the division in fp32: (64 + n^(1/2)) 2^-23 A.
    """
    B, H, d = q.shape
    u = U[q.dtype]
    w = 2.0 ** -10 if q.dtype == torch.bfloat16 else 2.0 ** -11
    wide = 23 if qtype == "q4_0" else 383
    for b in range(B):
        n = int(lens[b])
        hk = codes[0][b].shape[1]
        g = H // hk
        for h in range(hk):
            heads = slice(h * g, (h + 1) * g)
            if n <= 0:
                assert not out[b, heads].any(), f"request {b}: no keys, but not zero"
                if lse is not None:
                    assert bool((lse[b, heads] == -math.inf).all())
                continue
            kc, vc = (c[b][:n, h] for c in codes)
            ks, vs = (s[b][:n, h] for s in scales)
            k, v = values(kc, ks), values(vc, vs)
            qd = q[b, heads].double()
            s = qd @ k.t() * scale
            reach = qd.abs().unflatten(-1, (-1, 32)).sum(-1) @ ks.double().abs().t() * (wide * abs(scale))
            ds = ((d + 5) * 2.0 ** -23 * (reach + s.abs())).amax(1, keepdim=True)
            top = s.amax(1, keepdim=True)
            p = torch.exp(s - top)
            total = p.sum(1, keepdim=True)
            want = p @ v / total
            A = p @ v.abs() / total
            bound = (u * want.abs() + A * (w + 2 * ds + (64 + n ** 0.5) * 2.0 ** -23) + TINY[q.dtype]
                     + 2.0 ** -25 * (v.abs().sum(0) + vc.double().abs().sum(0)) / total)
            check(out[b, heads], want, bound, f"request {b} kv head {h}")
            if lse is not None:
                check(lse[b, heads], (top + total.log())[:, 0], ds[:, 0] + 2.0 ** -20 * (1 + top[:, 0].abs()),
                      f"lse of request {b} kv head {h}")
