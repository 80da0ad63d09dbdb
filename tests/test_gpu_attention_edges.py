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


# ------------------------------------------------------ values not finite --

def microseconds(f, n):
    f()
    best = math.inf
    for _ in range(3):
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1000 / n)
    return best


@pytest.mark.parametrize("D,Hq,Hk", [(128, 32, 8), (64, 8, 8), (256, 8, 4)])
@pytest.mark.parametrize("window", [0, 500])
def test_a_value_that_rows_see_costs_no_time(D, Hq, Hk, window):
    # Rows that see it cannot be anything but not finite: nothing is worked out again for them.
    q, k, v = heads(gen(D), 2048, Hq, Hk, D)
    bad = v.clone()
    bad[0] = NAN
    clean = microseconds(lambda: crm.prompt_attention(q, k, v, window=window), 5)
    out = crm.prompt_attention(q, k, bad, window=window)
    last = window or 2048
    assert out[:last].isnan().all() and not out[last:].isnan().any()
    # (Twice the time, not the hundredfold of rows worked out one by one; rows beside a window's edge are.)
    if not window:
        assert microseconds(lambda: crm.prompt_attention(q, k, bad), 5) < 2 * clean + 100


@pytest.mark.parametrize("dtype", [BF16, E4M3, E5M2])
@pytest.mark.parametrize("n", [1, 4])
def test_a_bad_slot_of_a_long_cache_costs_no_time(dtype, n):
    g = gen(n)
    kc, vc, table, ks, vs = cache(g, [20000], 64, 8, 128, dtype)
    q = normal(g, n, 32, 128).to(BF16)
    bad = vc.clone()
    bad[int(table[0, 3]), 5] = NAN
    f = lambda c: crm.paged_attention(q, kc, c, table, int32(20000), k_scale=ks, v_scale=vs)
    assert f(bad).isnan().all() and f(vc).isfinite().all()
    assert microseconds(lambda: f(bad), 5) < 2 * microseconds(lambda: f(vc), 5) + 100


@pytest.mark.parametrize("dtype", [BF16, E4M3, E5M2])
@pytest.mark.parametrize("D,G,causal,window", [(128, 4, True, 0), (128, 4, True, 40), (64, 1, True, 0), (64, 1, True, 300), (256, 2, True, 40),
                                               (192, 3, True, 0), (128, 4, False, 0)])
@pytest.mark.parametrize("n,m", [(4, 200), (4, 3000), (100, 700), (300, 3000), (300, 200)])
def test_columns_are_finite_where_no_seen_value_is_bad(dtype, D, G, causal, window, n, m):
    # Bad values here and there, also among the new tokens: a result is NaN exactly where a key that the row sees has one
    # in its column.
    g = gen(D, G, n, m, window)
    Hk = 2
    kc, vc, table, ks, vs = cache(g, [m], 16, Hk, D, dtype)
    for j in (0, m // 3, m - n // 2 - 1, m - 2, m - 1):
        vc[int(table[0, j // 16]), j % 16, j % Hk, (7 * j) % D] = NAN
    q = normal(g, n, G * Hk, D).to(BF16)
    how = dict(causal=causal, window=window)
    out = crm.paged_attention(q, kc, vc, table, int32(m), k_scale=ks, v_scale=vs, **how)
    values = attn_ref.cached(vc, table[0], m, vs)                             # [m, Hk, D]
    see = attn_ref.visible(n, m, causal, window, DEV).to(torch.float64)
    has = torch.einsum("nm,mhd->nhd", see, values.isnan().to(torch.float64)) > 0
    assert torch.equal(out.isnan(), has.repeat_interleave(G, 1))
    o, tol, _, _ = attn_ref.sequence(q, attn_ref.cached(kc, table[0], m, ks), torch.nan_to_num(values, 0.0),
                                     half=2.0 ** -8 if dtype == BF16 else 2.0 ** -11, **how)
    keep = ~out.isnan()
    attn_ref.check(out[keep], o[keep], tol[keep])


@pytest.mark.parametrize("n", [1, 4, 60])
@pytest.mark.parametrize("m", [300, 5000])
@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_infinite_values_of_small_weight(dtype, n, m):
    # exp(-25) = 2^-36 of the largest weight, and 2^-50: below what a 16-bit weight may hold, and still infinite.
    D, page = 128, 16
    pages = -(-m // page)
    kc, vc = torch.zeros(pages, page, 1, D, device=DEV), torch.ones(pages, page, 1, D, device=DEV)
    kc[0, 0] = 1.0
    vc[0, 1, 0, 3], vc[0, 2, 0, 4], vc[1, 0, 0, 5] = INF, -INF, NAN
    vc[2, 0, 0, 6], vc[2, 1, 0, 6] = INF, -INF
    q = torch.full((n, 2, D), 1.0, dtype=BF16, device=DEV)
    one = torch.ones(1, device=DEV) if dtype != BF16 else None
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    for s in (25.0, 35.0):
        out = crm.paged_attention(q, kc.to(dtype), vc.to(dtype), table, int32(m), scale=s / D, k_scale=one, v_scale=one)
        assert (out[..., 3] == INF).all() and (out[..., 4] == -INF).all() and out[..., 5:7].isnan().all()
        rest = [d for d in range(D) if not 3 <= d <= 6]
        assert ((out[..., rest].double() - 1).abs() <= 2.0 ** -7).all()


@pytest.mark.parametrize("D,Hq,Hk", [(128, 32, 8), (64, 8, 8), (256, 8, 4)])
@pytest.mark.parametrize("columns", [slice(None), slice(5, 6)])
def test_values_that_are_nan_throughout_cost_no_time(D, Hq, Hk, columns):
    # A row sees its own key: what is NaN in all keys is NaN in all results, whatever lies beside.
    q, k, v = heads(gen(D), 2048, Hq, Hk, D)
    bad = v.clone()
    bad[..., columns] = NAN
    out, clean = crm.prompt_attention(q, k, bad), crm.prompt_attention(q, k, v)
    has = torch.zeros(D, dtype=torch.bool, device=DEV)
    has[columns] = True
    assert torch.equal(out.isnan(), has.expand_as(out))
    assert torch.equal(out[..., ~has], clean[..., ~has])
    assert microseconds(lambda: crm.prompt_attention(q, k, bad), 5) < 2 * microseconds(lambda: crm.prompt_attention(q, k, v), 5) + 100


@pytest.mark.parametrize("dtype", [BF16, E4M3, E5M2])
@pytest.mark.parametrize("n", [1, 4, 60])
def test_a_cache_of_nan_costs_no_time(dtype, n):
    g = gen(n)
    kc, vc, table, ks, vs = cache(g, [20000], 64, 8, 128, dtype)
    q = normal(g, n, 32, 128).to(BF16)
    bad = torch.full_like(vc.float(), NAN).to(dtype)
    f = lambda c: crm.paged_attention(q, kc, c, table, int32(20000), k_scale=ks, v_scale=vs)
    assert f(bad).isnan().all() and f(vc).isfinite().all()
    assert microseconds(lambda: f(bad), 5) < 2 * microseconds(lambda: f(vc), 5) + 100
