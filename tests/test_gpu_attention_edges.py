"""The attention functions at the ends of their ranges: factors that leave
FP32, weights that leave FP16, values that are not finite, the border of the
short form, and what the order of a row's sums depends on."""
import math

import pytest
import torch

import attn_ref
import normalization_rmsnorm_fwd_gb300 as crm
from normalization_rmsnorm_fwd_gb300 import _abi, build
from test_gpu_attention import BF16, DEV, E4M3, E5M2, F32, INF, NAN, cache, gen, heads, normal, starts_of
from test_gpu_debug_guard import run_both

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


# -------------------------------------------------------- calls as allowed --

@pytest.mark.parametrize("n", [1, 20])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("page,capacity", [(16, 624), (16, 640), (16, 656), (1, 639), (1, 640), (1, 641)])
def test_paged_calls_around_the_short_form(n, dtype, page, capacity):
    # The table's width decides: up to 640 keys no workspace, whole tiles.
    g = gen(page, capacity)
    lens = [capacity, max(n, 7), capacity // 2]
    kc, vc, table, ks, vs = cache(g, lens, page, 2, 128, dtype, junk=NAN)
    table = table[:, :capacity // page].contiguous()
    assert table.shape[1] * page == capacity
    q = normal(g, 3 * n, 8, 128).to(BF16)
    o, tol, l, ltol = attn_ref.paged(q, kc, vc, table, lens, [n] * 3, ks, vs)
    for starts in (None, starts_of([n] * 3)):
        lse = torch.full(q.shape[:2], NAN, device=DEV)
        out = crm.paged_attention(q, kc, vc, table, int32(*lens), starts=starts, k_scale=ks, v_scale=vs, lse=lse)
        attn_ref.check(out, o, tol)
        attn_ref.check(lse, l, ltol, "lse")


@pytest.mark.parametrize("n", [1, 20])
def test_page_tables_of_any_row_stride(n):
    # One table for all sequences, and the first columns of a wider one.
    g = gen(n)
    kc, vc, table, _, _ = cache(g, [900], 16, 2, 128)
    q = normal(g, 5 * n, 8, 128).to(BF16)
    lens = [900, n, 333, 0, 512]
    o, tol, _, _ = attn_ref.paged(q, kc, vc, table.expand(5, -1), lens, [n] * 5)
    wide = torch.full((5, table.shape[1] + 9), -7, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    for t in (table.expand(5, -1), wide[:, :table.shape[1]]):
        attn_ref.check(crm.paged_attention(q, kc, vc, t, int32(*lens)), o, tol)


@pytest.mark.parametrize("T", [400, 1500])
def test_graph_replays_follow_the_starts(T):
    # A captured step over packed prompts whose borders change; tokens of none stay as they are.
    g = gen(T)
    q, k, v = heads(g, T, 8, 2, 128)
    starts = starts_of([T // 2, T - T // 2, 0, 0])
    out = torch.empty_like(q.contiguous())
    crm.prompt_attention(q, k, v, starts=starts, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        crm.prompt_attention(q, k, v, starts=starts, out=out)
    for ns in ([T // 2, T - T // 2, 0, 0], [1, 0, T - 41, 0], [0, 0, 0, 77], [0, 0, 0, 0]):
        starts.copy_(starts_of(ns))
        out.fill_(3.0)
        graph.replay()
        n = sum(ns)
        if n:
            o, tol, _, _ = attn_ref.prompt(q, k, v, ns)
            attn_ref.check(out[:n], o, tol)
        assert (out[n:] == 3).all()


@pytest.mark.parametrize("D", [64, 100])
def test_a_million_sequences(D):
    # Nearly all of them empty, or of a token each.
    B = 1 << 20
    ns = torch.zeros(B, dtype=torch.int64)
    ns[5], ns[B // 2], ns[B - 2] = 300, 1, 500
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), ns.cumsum(0)]).to(device=DEV, dtype=torch.int32)
    q, k, v = heads(gen(D), 801, 4, 2, D)
    o, tol, _, _ = attn_ref.prompt(q, k, v, [300, 1, 500])
    attn_ref.check(crm.prompt_attention(q, k, v, starts=starts), o, tol)
    q = normal(gen(D, 1), B, 2, D).to(BF16)
    kc, vc = normal(gen(D, 2), 2, 1, 1, 1, D).to(BF16)
    one = torch.ones(B, dtype=torch.int32, device=DEV)
    out = crm.paged_attention(q, kc, vc, torch.zeros(B, 1, dtype=torch.int32, device=DEV), one)
    assert torch.equal(out, vc[0].expand(B, 2, D))                            # one key: its value


# ------------------------------------------------------- the order of sums --

@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("ns", [[1, 1, 1], [20, 300, 1]])
def test_bits_depend_on_what_the_contract_names(dtype, ns):
    # Not on where pages lie, on their size, on the layout of a slot, on the workspace or on whether lse is asked for.
    g = gen(len(ns), ns[0])
    lens, Hk, D = [3000, 1024, 1999], 2, 128
    kc, vc, table, ks, vs = cache(g, lens, 16, Hk, D, dtype)
    table = table[:, :192].contiguous()
    q = normal(g, sum(ns), 8, D).to(BF16)
    starts = None if len(set(ns)) == 1 else starts_of(ns)
    how = dict(starts=starts, k_scale=ks, v_scale=vs)
    want = crm.paged_attention(q, kc, vc, table, int32(*lens), **how)
    lse = torch.empty(q.shape[:2], device=DEV)
    ws = torch.full((crm.attention_workspace_bytes(D),), 0x5a, dtype=torch.uint8, device=DEV)
    assert torch.equal(want, crm.paged_attention(q, kc, vc, table, int32(*lens), lse=lse, workspace=ws, **how))
    perm = torch.randperm(kc.shape[0], generator=g, device=DEV)
    back = perm.argsort().to(torch.int32)
    moved = torch.where((table >= 0) & (table < kc.shape[0]), back[table.clamp(0, kc.shape[0] - 1).long()], table)
    swap = lambda t: t.view(torch.uint8)[perm].view(t.dtype) if dtype != BF16 else t[perm]
    assert torch.equal(want, crm.paged_attention(q, swap(kc), swap(vc), moved, int32(*lens), **how))
    lay = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(want, crm.paged_attention(q, lay(kc), lay(vc), table, int32(*lens), **how))
    # The same keys in pages of 48.
    wide = torch.zeros(3 * 64, 48, Hk, D, device=DEV)
    big = [wide.to(dtype).clone() for _ in range(2)]
    for b, m in enumerate(lens):
        for t, c in zip(big, (kc, vc)):
            rows = attn_ref.cached(c, table[b], m).to(F32).to(dtype)
            t.view(3, 64 * 48, Hk, D)[b, :m] = rows
    table48 = torch.arange(3 * 64, dtype=torch.int32, device=DEV).view(3, 64)
    assert torch.equal(want, crm.paged_attention(q, big[0], big[1], table48, int32(*lens), **how))


def test_a_cache_that_records_gradients_is_refused():
    g = gen(1)
    kc, vc, table, _, _ = cache(g, [40], 16, 2, 128)
    q = normal(g, 1, 4, 128).to(BF16)
    for a, b in ((kc.clone().requires_grad_(), vc), (kc, vc.clone().requires_grad_())):
        with pytest.raises(RuntimeError):
            crm.paged_attention(q, a, b, table, int32(40))
        with torch.no_grad():
            crm.paged_attention(q, a, b, table, int32(40))
    k8, v8 = kc.to(E4M3), vc.to(E4M3)
    one = torch.ones(1, device=DEV)
    for a, b in ((one.clone().requires_grad_(), one), (one, one.clone().requires_grad_())):
        with pytest.raises(RuntimeError):
            crm.paged_attention(q, k8, v8, table, int32(40), k_scale=a, v_scale=b)


def test_empty_sequences_between_others_cost_no_time():
    # A CTA whose work goes on behind thousands of sequences without tokens.
    some = [3000] * 60 + [300], [1] * 64 + [200]
    T = sum(some[0] + some[1])
    q, k, v = heads(gen(1), T, 4, 2, 64)
    apart, together = some[0] + [0] * 20000 + some[1] + [0] * 77, some[0] + some[1]
    one, two = starts_of(apart), starts_of(together)
    outs = [crm.prompt_attention(q, k, v, starts=s) for s in (one, two)]
    o, tol, _, _ = attn_ref.prompt(q[-264:], k[-264:], v[-264:], some[1])
    for out in outs:
        attn_ref.check(out[-264:], o, tol)
    assert torch.equal(*outs)
    assert microseconds(lambda: crm.prompt_attention(q, k, v, starts=one), 5) < microseconds(lambda: crm.prompt_attention(q, k, v, starts=two), 5) + 300


@pytest.mark.parametrize("n,m", [(60, 30), (4, 2), (300, 200)])
@pytest.mark.parametrize("bad", ["k_scale", "v_scale"])
def test_rows_without_keys_and_scales_of_nan(monkeypatch, n, m, bad):
    # Rows before the first key are not finite here, and a value that they do not see is bad: none of it leads a look
    # outside the cache (the debug build reports accesses).
    dbg = _abi.load(build.build(debug=True))

    def case():
        g = gen(n)
        kc, vc, table, ks, vs = cache(g, [m, m], 16, 2, 128, E4M3)
        vc[int(table[0, (m - 1) // 16]), (m - 1) % 16] = NAN
        if bad == "k_scale":
            ks = torch.full_like(ks, NAN)
        else:
            vs = torch.full_like(vs, NAN)
        q = normal(g, 2 * n, 8, 128).to(BF16)
        return [crm.paged_attention(q, kc, vc, table, int32(m, m), k_scale=ks, v_scale=vs),
                crm.paged_attention(q, kc, vc, table, int32(m, m), k_scale=ks, v_scale=vs, starts=starts_of([n, n]))]

    run_both(dbg, monkeypatch, case)
