"""Plain FP64 form of the attention functions and the error bounds that their
evaluation must keep, for the tests.

Bounds, with a score s_j = scale q . k_j, weights p_j = exp(s_j - M), P their
sum, A_j = scale sum_d |q_d k_d|, over m keys:
* a score: products of BF16 or FP8 values are exact; D additions of at most
  one FP32 step (2^-23) each, the scale and the change to powers of two:
  (D + 8) 2^-23 A_j.  Its exponential: the FP32 difference from the maximum
  (2^-22 (|s_j| + |M|)) and 2^-22 of its own: together the relative error e_j
  of p_j.  It reaches the numerator with p_j |v_j| and the sum with p_j.
* the sums: at most m additions of one step: m 2^-23 of sum p_j |v_j| and of
  P, and a few roundings for joining parts and for the division: 2^-20.
* the rounding of p_j before the product with the values: half a step, h =
  2^-8 (BF16), 2^-11 (FP16, FP8 caches), of each term.  As signs differ from
  key to key (independent errors of mean zero, each within h p_j |v_j|),
  Hoeffding's bound gives 7 h sqrt(sum (p_j v_j)^2) with probability
  1 - 2 exp(-24.5), 5e-11 for each element, never more than h sum p_j |v_j|.
  FP16 weights below 2^-14 are off by at most 2^-25: 2^-25 sum |v_j|.
* the BF16 result: half a step, 2^-8 of the value.
* lse: max e_j + m 2^-23 + 2^-20 + 2^-22 |lse|.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def visible(n, m, causal=True, window=0, device="cpu"):
    """[n, m]: token i sees key j."""
    p = m - n + torch.arange(n, device=device)[:, None]
    j = torch.arange(m, device=device)[None]
    see = (j <= p) if causal else torch.ones(n, m, dtype=torch.bool, device=device)
    return see & (j > p - window) if window else see


def sequence(q, k, v, scale=None, causal=True, window=0, half=2.0 ** -8):
    """(out, its bound, lse, its bound) in FP64 of q [n, Hq, D] over k, v
    [m, Hk, D] (values already times their scale); masked keys and values may
    hold anything."""
    n, Hq, D = q.shape
    m, Hk = k.shape[:2]
    dev = q.device
    scale = D ** -0.5 if scale is None else scale
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    if m == 0:
        zero = torch.zeros(n, Hq, D, dtype=F64, device=dev)
        return zero, zero, torch.full((n, Hq), -math.inf, dtype=F64, device=dev), torch.zeros(n, Hq, dtype=F64, device=dev)
    see = visible(n, m, causal, window, dev)
    out, tol, lse, ltol = [], [], [], []
    for h in range(Hq):
        g = h // (Hq // Hk)
        s = torch.where(see, scale * (q[:, h] @ k[:, g].T), -math.inf)
        A = torch.where(see, scale * (q[:, h].abs() @ k[:, g].abs().T), 0.0)
        top = s.amax(1, keepdim=True)
        base = torch.where(top == -math.inf, 0.0, top)
        p = torch.exp(s - base)
        e = torch.where(see, (D + 8) * 2.0 ** -23 * A + 2.0 ** -22 * (s.abs() + base.abs() + 1), 0.0)
        e = torch.where(p == 0, 0.0, e)
        P = p.sum(1, keepdim=True)
        # A key whose weight is nothing for a row has no say in it.
        seen = see.any(0)
        vg = torch.where(seen[:, None], v[:, g], 0.0)
        if not torch.isfinite(vg).all():
            o = torch.stack([(p[i, see[i]][:, None] * vg[see[i]]).sum(0) for i in range(n)])
        else:
            o = p @ vg
        sums = m * 2.0 ** -23 + 2.0 ** -20
        finite = torch.nan_to_num(vg, 0.0, 0.0, 0.0).abs()
        size, root = p @ finite, ((p * p) @ (finite * finite)).sqrt()
        err = (p * e) @ finite + o.abs() / P.clamp(min=1e-300) * (p * e).sum(1, keepdim=True)
        err = err + sums * 2 * size + torch.minimum(7 * half * root, half * size)
        if half < 2.0 ** -8:
            err = err + 2.0 ** -25 * (see.to(F64) @ finite)
        empty = P == 0
        P1 = torch.where(empty, 1.0, P)
        out.append(torch.where(empty, 0.0, o / P1))
        tol.append(torch.where(empty, 0.0, err / P1 + 2.0 ** -8 * (o / P1).abs()))
        l = torch.where(empty, -math.inf, base + P1.log())[:, 0]
        lse.append(l)
        ltol.append(e.amax(1) + sums + 2.0 ** -22 * torch.where(empty[:, 0], 0.0, l).abs())
    return torch.stack(out, 1), torch.stack(tol, 1), torch.stack(lse, 1), torch.stack(ltol, 1)


def prompt(q, k, v, lengths, **how):
    """sequence() of packed [T, H, D] tensors, concatenated."""
    parts, at = [], 0
    for n in lengths:
        parts.append(sequence(q[at:at + n], k[at:at + n], v[at:at + n], **how))
        at += n
    return [torch.cat(x) for x in zip(*parts)]


def cached(cache, table, m, scale=None):
    """The first m keys or values [m, Hk, D] of one sequence; page numbers out
    of range hold zeros."""
    pages, size = cache.shape[:2]
    j = torch.arange(m, device=cache.device)
    page = table.long()[j // size]
    good = (page >= 0) & (page < pages)
    x = torch.zeros(m, *cache.shape[2:], dtype=F64, device=cache.device)
    x[good] = cache[page[good], j[good] % size].to(F64)
    return x if scale is None else x * scale.to(F64)


def paged(q, k_cache, v_cache, table, lens, ns, k_scale=None, v_scale=None, **how):
    """sequence() of packed new tokens, ns[b] of sequence b, over the cache."""
    parts, at = [], 0
    half = 2.0 ** -8 if k_cache.dtype == torch.bfloat16 else 2.0 ** -11
    for b, (n, m) in enumerate(zip(ns, lens)):
        parts.append(sequence(q[at:at + n], cached(k_cache, table[b], m, k_scale), cached(v_cache, table[b], m, v_scale),
                              half=half, **how))
        at += n
    return [torch.cat(x) for x in zip(*parts)]


def check(got, exact, tol, what="out"):
    got = got.to(F64)
    bad = ~((got - exact).abs() <= tol + 2.0 ** -134)
    bad &= ~((got == exact) | (got.isnan() & exact.isnan()))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at "
                           f"{bad.nonzero()[0].tolist()}: got {got[bad][:4].tolist()}, exact {exact[bad][:4].tolist()}, "
                           f"bound {tol[bad][:4].tolist()}")
