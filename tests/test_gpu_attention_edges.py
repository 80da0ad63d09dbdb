"""The attention functions at the ends of their ranges: factors that leave
FP32, weights that leave FP16, values that are not finite, the border of the
short form, and what the order of a row's sums depends on."""
import math

import pytest
import torch

import attn_ref
import normalization_rmsnorm_fwd_gb300 as crm
from test_gpu_attention import BF16, DEV, E4M3, E5M2, F32, INF, NAN, cache, gen, heads, normal, starts_of

pytestmark = pytest.mark.gpu


def int32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- factors --

@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("D", [64, 100, 128, 192, 256])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("k_scale,q_size", [(2.0 ** -140, 1.0), (0.0, 1.0), (-(2.0 ** -140), 1.0), (0.05, 2.0 ** -133), (0.05, 2.0 ** -132), (2.0 ** -120, 2.0 ** -100)])
def test_scores_below_fp32_leave_a_mean(dtype, D, n, k_scale, q_size):
    # Lengths that end inside a block: masked places beside a factor that rounds to nothing.
    g = gen(D, n, k_scale)
    lens = [max(n, 77), 130, 1003]
    kc, vc, table, _, vs = cache(g, lens, 16, 2, D, dtype, junk=NAN)
    ks = torch.tensor([k_scale], device=DEV)
    q = (torch.randint(-1, 2, (3 * n, 8, D), generator=g, device=DEV) * q_size).to(BF16)
    q[0, 0, 0] = q_size
    assert q.abs().max() == q_size
    lse = torch.full(q.shape[:2], NAN, device=DEV)
    out = crm.paged_attention(q, kc, vc, table, int32(*lens), k_scale=ks, v_scale=vs, lse=lse)
    o, tol, l, ltol = attn_ref.paged(q, kc, vc, table, lens, [n] * 3, ks, vs)
    attn_ref.check(out, o, tol)
    attn_ref.check(lse, l, ltol, "lse")


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("D", [64, 100, 128, 256])
@pytest.mark.parametrize("n", [1, 40])
def test_negative_scales(dtype, D, n):
    g = gen(D, n)
    lens = [max(n, 77), 130, 1003]
    kc, vc, table, ks, vs = cache(g, lens, 16, 2, D, dtype, junk=NAN)
    q = normal(g, 3 * n, 8, D).to(BF16)
    for k_scale, v_scale in ((-ks, vs), (ks, -vs)):
        lse = torch.full(q.shape[:2], NAN, device=DEV)
        out = crm.paged_attention(q, kc, vc, table, int32(*lens), k_scale=k_scale, v_scale=v_scale, lse=lse)
        o, tol, l, ltol = attn_ref.paged(q, kc, vc, table, lens, [n] * 3, k_scale, v_scale)
        attn_ref.check(out, o, tol)
        attn_ref.check(lse, l, ltol, "lse")


# ---------------------------------------------------------------- weights --

@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("D", [64, 100, 128, 192, 256])
@pytest.mark.parametrize("n,m", [(1, 600), (1, 100001), (40, 100001)])
def test_small_weights_add_up_over_fp8(dtype, D, n, m):
    # One key that takes nearly all, of value 0, before keys of weight exp(-18) = 2^-25.97 and value 1.
    page = 64
    pages = -(-m // page)
    kc = torch.zeros(pages, page, 1, D, device=DEV)
    vc = torch.ones(pages, page, 1, D, device=DEV)
    kc[0, 0], vc[0, 0] = 1.0, 0.0
    q = torch.full((n, 2, D), 16.0 / D, dtype=BF16, device=DEV)
    scale = 18.0 / float((q[0, 0].double()).sum())
    one = torch.ones(1, device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    out = crm.paged_attention(q, kc.to(dtype), vc.to(dtype), table, int32(m), scale=scale, k_scale=one, v_scale=one)
    # Weights relative to the largest: w = exp(-18), their FP16 rounding off by at most 2^-29 (half a step of FP16's
    # smallest numbers, 2^-25, where the largest weight is 2^4 or more) or by 2^-11 of w, the exponential by 2^-17 (scores
    # of 18 in FP32, exponents of 26); sums of m terms by m 2^-24 of themselves; the result by 2^-8.
    w = math.exp(-18.0)
    for i in range(n):
        seen = m - n + i                       # of value 1
        want = seen * w / (1 + seen * w)
        tol = seen * max(2.0 ** -29, 2.0 ** -11 * w) + want * (2.0 ** -16 + seen * 2.0 ** -23 + 2.0 ** -8)
        assert ((out[i].double() - want).abs() <= tol).all(), (i, out[i, 0, 0].item(), want, tol)
