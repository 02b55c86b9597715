"""fp64 references of the attention calls, with elementwise bounds on what a correct 16-bit
kernel may be off, derived from the formulas:

  * the output is rounded once to 16 bits: u |out|, u = 2^-8 (bf16) or 2^-11 (f16);
  * the weights p may be rounded to the same 16 bits before the product with v: u A,
    A = sum_j p_j |v_j| (p normalised), and below f16's normal range by 2^-25 each, with
    the largest p of a row being at least 1: n 2^-25 max|v|;
  * a score is an fp32 sum of d exact products, scaled: its error is at most
    ds = (d + 4) 2^-23 scale sum|q k| + 2^-23 |score|, which moves every weight by at most 2 ds
    relative to the others: 2 ds A;
  * exp, the sums and the division in fp32: (64 + n^(1/2)) 2^-23 A, n the number of keys.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}


def attend(q, k, v, scale, hidden=None):
    """One head's rows q [n, d] over k, v [m, d]: (out, bound, lse, lse_bound) in fp64."""
    dt, (n, d), m = q.dtype, q.shape, k.shape[0]
    q, k, v = q.double(), k.double(), v.double()
    if m == 0:
        z = torch.zeros((n, d), dtype=torch.float64, device=q.device)
        return z, z, torch.full((n,), -math.inf, dtype=torch.float64, device=q.device), z[:, 0]
    s = (q @ k.t()) * scale
    reach = (q.abs() @ k.abs().t()) * abs(scale)
    seen = torch.ones_like(s, dtype=torch.bool) if hidden is None else ~hidden
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    reach = torch.where(seen, reach, torch.zeros_like(reach))
    ds = ((d + 5) * 2.0 ** -23 * reach).amax(1, keepdim=True)
    top = s.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.where(seen, torch.exp(s - top), torch.zeros_like(s))
    total = p.sum(1, keepdim=True)
    none = total == 0
    total = torch.where(none, torch.ones_like(total), total)
    # a key no row sees must not enter through 0 * inf
    used = seen.any(0)[:, None]
    v = torch.where(used, v, torch.zeros_like(v))
    if not torch.isfinite(v).all():  # a non-finite value reaches only the rows that see it
        fin = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
        out = p @ fin / total
        for j in (~torch.isfinite(v)).any(1).nonzero().flatten().tolist():
            bad = ~torch.isfinite(v[j])
            out[:, bad] += torch.where(seen[:, j:j + 1], v[j, bad], torch.zeros_like(v[j, bad]))
        v = fin
    else:
        out = p @ v / total
    a = p @ v.abs() / total
    u = U[dt]
    bound = u * out.abs() + a * (u + 2 * ds + (64 + m ** 0.5) * 2.0 ** -23) + TINY[dt]
    if dt == torch.float16:
        bound = bound + m * 2.0 ** -25 * v.abs().amax()
    lse = torch.where(none, torch.full_like(top, -math.inf), top + total.log())[:, 0]
    lse_bound = (ds[:, 0] + 2.0 ** -20 * (1 + top[:, 0].abs()))
    return out, bound, lse, lse_bound


def check(got, want, bound, what):
    got = got.double()
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, torch.zeros_like(want), (got - want).abs())
    over = ~(off <= torch.where(same, torch.ones_like(want), bound))
    assert not over.any(), (f"{what}: {int(over.sum())} of {over.numel()} outside the bound, first at "
                            f"{over.nonzero()[0].tolist()}: got {got[over][0].item()} want {want[over][0].item()} "
                            f"bound {bound.expand_as(want)[over][0].item()}")


def check_prompt(q, k, v, lq, lk, causal, scale, out, lse=None, at_q=None, at_k=None):
    """Every sequence and head of a packed call against attend(); at_q, at_k: first rows (packed when None)."""
    g = q.shape[1] // k.shape[1]
    a = b = 0
    for i, (n, m) in enumerate(zip(lq, lk)):
        a, b = (a if at_q is None else at_q[i]), (b if at_k is None else at_k[i])
        hidden = None
        if causal:
            hidden = torch.ones(n, m, dtype=torch.bool, device=q.device).triu(m - n + 1)
        for h in range(q.shape[1]):
            if n == 0:
                continue
            o, bd, l, lb = attend(q[a:a + n, h], k[b:b + m, h // g], v[b:b + m, h // g], scale, hidden)
            check(out[a:a + n, h], o, bd, f"sequence {i} head {h}")
            if lse is not None:
                check(lse[a:a + n, h], l, lb, f"lse of sequence {i} head {h}")
        a, b = a + n, b + m


def check_decode(q, k, v, lens, pk, pv, scale, out, lse=None):
    g = q.shape[1] // (k if k is not None else pk).shape[-2]
    for b in range(q.shape[0]):
        for h in range(0, q.shape[1], g):
            ks, vs = [], []
            if pk is not None:
                ks.append(pk[:, h // g])
                vs.append(pv[:, h // g])
            if k is not None:
                n = min(max(int(lens[b]), 0), k.shape[1])
                ks.append(k[b, :n, h // g])
                vs.append(v[b, :n, h // g])
            o, bd, l, lb = attend(q[b, h:h + g], torch.cat(ks), torch.cat(vs), scale)
            check(out[b, h:h + g], o, bd, f"request {b} heads {h}..")
            if lse is not None:
                check(lse[b, h:h + g], l, lb, f"lse of request {b} heads {h}..")


def norm_rope(x, w, eps, positions, inv_freq, interleaved):
    """(out, bound) in fp64 of qmm_qk_norm_rope's heads x [m, h, d]; the bound is for fp32 arithmetic
    (a norm of d terms, a turn by an angle good to 2^-21) without the final rounding."""
    y = x.double()
    if w is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    bound = (x.shape[-1] + 16) * 2.0 ** -24 * y.abs()
    if inv_freq is None:
        return y, bound
    r = 2 * inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    i = torch.arange(0, r, 2, device=x.device) if interleaved else torch.arange(r // 2, device=x.device)
    j = i + (1 if interleaved else r // 2)
    a, b = y[..., i], y[..., j]
    out = y.clone()
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    size = (a.abs() + b.abs()) * (2.0 ** -20 + (x.shape[-1] + 16) * 2.0 ** -24)
    bound = bound.clone()
    bound[..., i] = bound[..., j] = size
    return out, bound
