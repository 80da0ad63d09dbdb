"""Plain FP64 forms of the query / key functions and the error bounds that
their FP32 evaluation must keep, for the tests.

Bounds, in units u = 2^-24 (half an FP32 step), to first order:
* rstd: a row's squares are added in at most 16 + 5 steps (a lane's elements,
  then a butterfly), D * (1/D) and eps add 3, all halved by the root, whose
  own rounding adds 1: 13 u.
* n = (x rstd) w: 13 + 2, and 1 for w + bias: 16 u relative.  A rotated value
  n_a c - n_b s adds one rounding of each product and one of the sum:
  18 u (|n_a c| + |n_b s|); below, 2^-19 = 32 u of that sum.
* u = the turned-back gradient: 2 u A with A = |g_a c| + |g_b s|.  The mean
  M = mean(u w xhat): terms 2 + 3, at most 16 + 5 + 2 for the sum, rstd 13 + 2:
  44 u mean(A |w xhat|).  dx = rstd (u w - xhat M) adds rstd 13, its products
  and difference 4: at most 61 u = below 2^-18 of
  rstd (A |w| + |xhat| mean(A |w xhat|)).
* dw: terms u xhat 2 + 14 + 1, 16 plain additions before each compensated
  one, a rounding per partial row and at the end: below 36 u; 2^-18 = 64 u of
  sum A |xhat|.
A BF16 result adds half a step: 2^-8 of the value (2^-134 where subnormal);
FP8: 2^-4 (E4M3, subnormal 2^-10) or 2^-3 (E5M2, 2^-17), and 2^-22 for the
product with the rounded reciprocal of the scale.
"""
from __future__ import annotations

import torch

F64 = torch.float64
HALF_STEP = {torch.bfloat16: (2.0 ** -8, 2.0 ** -134), torch.float8_e4m3fn: (2.0 ** -4, 2.0 ** -10),
             torch.float8_e5m2: (2.0 ** -3, 2.0 ** -17)}
TOP = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}


def axis_of(half, sections, mixed):
    """The axis of each column, counted off one by one."""
    left, out, a = list(sections), [], 0
    for j in range(half):
        if mixed:
            a = j % len(left)
            if j >= len(left) * sections[a]:
                a = 0
        else:
            while left[a] == 0:
                a += 1
            left[a] -= 1
        out.append(a)
    return out


def angles(positions, inv_freq, sections=None, mixed=False, scaling=1.0):
    """[T, R] in FP64 from CPU tensors; positions [axes, T] below 2^29, where
    the FP64 product with an FP32 frequency is exact."""
    half = inv_freq.shape[0]
    at = torch.tensor(axis_of(half, sections or [half], mixed))
    a = positions.reshape(len(sections or [0]), -1)[at].T.to(F64) * inv_freq.to(F64)
    return scaling * torch.cat([a.cos(), a.sin()], 1)


def split(x, R, pairs):
    return (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])


def join(a, b, rest, pairs):
    y = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1)


def turn(x, cs, pairs, back=False):
    """x [T, H, D] turned by cs [P, R] (token t: row t % P)."""
    if cs is None:
        return x
    R = cs.shape[1]
    cs = cs.to(x.dtype)[torch.arange(x.shape[0]) % cs.shape[0]][:, None]
    c, s = cs[..., :R // 2], cs[..., R // 2:]
    s = -s if back else s
    a, b = split(x, R, pairs)
    return join(a * c - b * s, b * c + a * s, x[..., R:], pairs)


def turn_abs(x, cs, pairs):
    """The sum of the magnitudes that make each turned value."""
    if cs is None:
        return x.abs()
    R = cs.shape[1]
    cs = cs.to(x.dtype)[torch.arange(x.shape[0]) % cs.shape[0]][:, None].abs()
    c, s = cs[..., :R // 2], cs[..., R // 2:]
    a, b = split(x.abs(), R, pairs)
    return join(a * c + b * s, b * c + a * s, x[..., R:].abs(), pairs)


def normed(x, w, bias, eps):
    """(xhat, rstd, effective weight)"""
    if w is None:
        return x, torch.ones(x.shape[:-1] + (1,), dtype=F64), torch.ones(x.shape[-1], dtype=F64)
    rstd = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return x * rstd, rstd, (w.double() + bias)


def forward(x, w, cs, eps=1e-6, bias=0.0, pairs=False):
    """(y, the FP32 error bound) of [T, H, D] in FP64, on the CPU."""
    x = x.double()
    xhat, _, we = normed(x, w, bias, eps)
    n = xhat * we
    return turn(n, cs, pairs), 2.0 ** -19 * turn_abs(n, cs, pairs)


def backward(g, x, w, cs, eps=1e-6, bias=0.0, pairs=False):
    """(dx, bound, dw, bound) in FP64 (dw None without a weight)."""
    g = g.double()
    u, A = turn(g, cs, pairs, back=True), turn_abs(g, cs, pairs)
    if w is None:
        return u, 2.0 ** -19 * A, None, None
    x = x.double()
    xhat, rstd, we = normed(x, w, bias, eps)
    dx = rstd * (u * we - xhat * (u * we * xhat).mean(-1, keepdim=True))
    size = rstd * (A * we.abs() + xhat.abs() * (A * (we * xhat).abs()).mean(-1, keepdim=True))
    return dx, 2.0 ** -18 * size, (u * xhat).sum((0, 1)), 2.0 ** -18 * (A * xhat.abs()).sum((0, 1))


def check(got, exact, bound, scale=None, what="value"):
    """got (a BF16, FP8 or FP32 tensor) within half a step plus the bound."""
    got = got.detach().cpu()
    if scale is not None:
        exact, bound = exact / scale, bound / scale + 2.0 ** -22 * (exact / scale).abs()
        exact = exact.clamp(-TOP[got.dtype], TOP[got.dtype])
    rel, least = HALF_STEP.get(got.dtype, (2.0 ** -24, 2.0 ** -150))
    g = got.double() if got.dtype not in TOP else got.float().double()
    assert g.shape == exact.shape, (what, g.shape, exact.shape)
    # The half step of a value that the error lifts over a power of two is
    # that of the lifted value.
    tol = rel * (exact.abs() + bound) + least + bound
    same = (g == exact) | (g.isnan() & exact.isnan())
    bad = ~((g - exact).abs() <= tol) & ~same
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; got {g[bad][:4].tolist()} "
                           f"exact {exact[bad][:4].tolist()} tol {tol[bad][:4].tolist()}")
