"""The attention functions against the FP64 form: every head size, group,
layout and cache type, ragged and empty sequences, masks that leave rows
without keys, values that must not be seen."""
import math
import random
import zlib

import pytest
import torch

import attn_ref
import normalization_rmsnorm_fwd_gb300 as crm

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
NAN, INF = math.nan, math.inf


def gen(*seed):
    return torch.Generator(device=DEV).manual_seed(zlib.crc32(repr(seed).encode()))


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def starts_of(ns):
    at = [0]
    for n in ns:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def heads(g, T, Hq, Hk, D, layout="packed"):
    x = normal(g, T, Hq + 2 * Hk, D).to(BF16)
    if layout == "packed":
        return x.split([Hq, Hk, Hk], 1)
    if layout == "heads":                 # [H, T, D] storage
        return [t.transpose(0, 1).contiguous().transpose(0, 1) for t in x.split([Hq, Hk, Hk], 1)]
    if layout == "gated":                 # heads beside a gate
        x = normal(g, T, Hq + 2 * Hk, 2, D).to(BF16)[:, :, 0]
        return x.split([Hq, Hk, Hk], 1)
    x = normal(g, T * (Hq + 2 * Hk) * D + 1).to(BF16)[1:].view(T, Hq + 2 * Hk, D)   # odd address
    return x.split([Hq, Hk, Hk], 1)


def check_prompt(q, k, v, ns, use_starts, **how):
    lse = torch.full(q.shape[:2], NAN, device=DEV)
    out = crm.prompt_attention(q, k, v, starts=starts_of(ns) if use_starts else None, lse=lse, **how)
    o, tol, l, ltol = attn_ref.prompt(q, k, v, ns, **how)
    T = sum(ns)
    attn_ref.check(out[:T], o, tol)
    attn_ref.check(lse[:T], l, ltol, "lse")
    return out


@pytest.mark.parametrize("D", [2, 32, 50, 64, 72, 80, 96, 100, 128, 160, 192, 200, 256, 320, 512])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 1), (6, 2), (7, 1)])
def test_prompt_head_sizes(D, Hq, Hk):
    q, k, v = heads(gen(D, Hq), 150, Hq, Hk, D)
    check_prompt(q, k, v, [150], False)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513, 1000])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 70)])
def test_prompt_lengths(T, causal, window):
    q, k, v = heads(gen(T, window), T, 4, 2, 128)
    check_prompt(q, k, v, [T], False, causal=causal, window=window)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 31, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompt_groups(G, D):
    q, k, v = heads(gen(G, D), 141, 2 * G, 2, D)
    check_prompt(q, k, v, [100, 0, 41], True, window=57)


@pytest.mark.parametrize("layout", ["packed", "heads", "gated", "odd"])
@pytest.mark.parametrize("D", [64, 128, 192])
def test_prompt_layouts(layout, D):
    q, k, v = heads(gen(layout, D), 200, 6, 2, D, layout)
    check_prompt(q, k, v, [200], False)
    check_prompt(q, k, v, [3, 130, 67], True, causal=False)


@pytest.mark.parametrize("ns", [[0, 0, 5, 0], [1] * 40, [1, 300, 2, 0, 129, 64, 7], [0], [700, 1]])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_packed(ns, causal):
    T = sum(ns)
    q, k, v = heads(gen(T), T + 5, 5, 1, 128)
    out = torch.full((T + 5, 5, 128), 3.0, dtype=BF16, device=DEV)
    lse = torch.full((T + 5, 5), 3.0, device=DEV)
    crm.prompt_attention(q, k, v, starts=starts_of(ns), causal=causal, out=out, lse=lse)
    if T:
        o, tol, l, ltol = attn_ref.prompt(q, k, v, ns, causal=causal)
        attn_ref.check(out[:T], o, tol)
        attn_ref.check(lse[:T], l, ltol, "lse")
    # Rows behind the last sequence stay as they were.
    assert (out[T:] == 3).all() and (lse[T:] == 3).all()


def test_prompt_starts_behind_zero():
    # Tokens before the first sequence belong to none.
    q, k, v = heads(gen(1), 60, 4, 2, 64)
    out = torch.full((60, 4, 64), 3.0, dtype=BF16, device=DEV)
    crm.prompt_attention(q, k, v, starts=torch.tensor([7, 20, 50], dtype=torch.int32, device=DEV), out=out)
    o, tol, _, _ = attn_ref.prompt(q[7:], k[7:], v[7:], [13, 30])
    attn_ref.check(out[7:50], o, tol)
    assert (out[:7] == 3).all() and (out[50:] == 3).all()


def test_prompt_batches():
    q, k, v = (normal(gen(2), 3, 90, H, 128).to(BF16) for H in (4, 2, 2))
    out = crm.prompt_attention(q, k, v)
    assert out.shape == q.shape
    o, tol, _, _ = attn_ref.prompt(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), [90] * 3)
    attn_ref.check(out.flatten(0, 1), o, tol)
    empty = crm.prompt_attention(q[:, :0], k[:, :0], v[:, :0])
    assert empty.shape == (3, 0, 4, 128)


@pytest.mark.parametrize("scale", [0.01, 1.0, 3.0])
def test_prompt_scales(scale):
    # Sharp scores: the maximum moves by hundreds along a row.
    q, k, v = heads(gen(scale), 400, 4, 2, 128)
    check_prompt(q, k, v, [400], False, scale=scale)
    k = (k.float() * torch.linspace(0.01, 8, 400, device=DEV)[:, None, None]).to(BF16)
    check_prompt(q, k, v, [400], False, scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256, 100])
@pytest.mark.parametrize("bad", [NAN, INF, -INF, torch.finfo(BF16).min])
def test_prompt_masked_values_do_not_matter(D, bad):
    # What later tokens hold is not seen by earlier ones, whatever it is.
    q, k, v = (t.clone() for t in heads(gen(D), 300, 4, 2, D))
    k[170], v[200], v[299, :, ::7] = bad, bad, bad
    out = crm.prompt_attention(q, k, v)
    clean = crm.prompt_attention(q[:170], k[:170], v[:170])
    o, tol, _, _ = attn_ref.prompt(q[:170], k[:170], v[:170], [170])
    attn_ref.check(clean, o, tol)
    attn_ref.check(out[:170], o, tol)
    if bad != bad:
        assert out[170:].isnan().all()
    win = crm.prompt_attention(q, k, v, window=20)
    o, tol, _, _ = attn_ref.prompt(q, k, v, [300], window=20)
    for rows in (slice(0, 170), slice(190, 200), slice(220, 299)):
        attn_ref.check(win[rows], o[rows], tol[rows])


def test_later_values_do_not_matter_over_many_keys():
    # Rows worked out again key by key, over a long cache, split among CTAs or not.
    g = gen(12)
    kc, vc, table, _, _ = cache(g, [30000], 64, 1, 128)
    page, row = int(table[0, 29990 // 64]), 29990 % 64
    vc[page, row] = NAN
    for n in (4, 100):
        q = normal(g, n, 4, 128).to(BF16)
        out = crm.paged_attention(q, kc, vc, table, torch.tensor([30000], dtype=torch.int32, device=DEV))
        k0, v0 = kc.clone(), vc.clone()
        v0[page, row] = 0
        seen = 29990 - (30000 - n)               # tokens that stand before it
        if seen > 0:
            o, tol, _, _ = attn_ref.paged(q, k0, v0, table, [30000], [n])
            attn_ref.check(out[:seen], o[:seen], tol[:seen])
        assert out[max(seen, 0):].isnan().all()


def test_prompt_infinite_values_that_are_seen():
    q, k, v = (t.clone() for t in heads(gen(5), 200, 2, 1, 128))
    v[50, :, 3] = INF
    v[60, :, 4] = NAN
    out = crm.prompt_attention(q, k, v)
    assert (out[50:, :, 3] == INF).all() and out[60:, :, 4].isnan().all()
    rest = [d for d in range(128) if d not in (3, 4)]
    o, tol, _, _ = attn_ref.prompt(q, k, torch.nan_to_num(v, 0, 0, 0), [200])
    attn_ref.check(out[:, :, rest], o[..., rest], tol[..., rest])


# ----------------------------------------------------------------- cache --

def cache(g, lens, page, Hk, D, dtype=BF16, order="token", spare=3, junk=None):
    """k_cache, v_cache, page table and scales; slots that hold no key hold
    `junk`, entries of the table behind the last page name no page."""
    held = [-(-m // page) for m in lens]
    pages = sum(held) + spare
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.tensor([-1, 1 << 30], dtype=torch.int32, device=DEV).repeat(len(lens), (max(held, default=0) + 3) // 2)
    used = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        for i in range(h):
            used[perm[at + i], :min(page, lens[b] - i * page)] = True
        at += h
    scale = None if dtype == BF16 else (torch.tensor([0.06], device=DEV), torch.tensor([0.13], device=DEV))
    out = []
    for i in range(2):
        x = normal(g, pages, page, Hk, D)
        x = x if scale is None else x / scale[i]
        x[~used] = 0.0 if junk is None else junk
        x = x.to(dtype)
        out.append(x if order == "token" else x.transpose(1, 2).contiguous().transpose(1, 2))
    ks, vs = scale or (None, None)
    return out[0], out[1], table, ks, vs


def check_paged(g, ns, lens, Hq, Hk, D, page=16, dtype=BF16, order="token", junk=NAN, starts=None, q=None, **how):
    kc, vc, table, ks, vs = cache(g, lens, page, Hk, D, dtype, order, junk=junk)
    T = sum(ns)
    q = normal(g, T, Hq, D).to(BF16) if q is None else q
    lse = torch.full((T, Hq), NAN, device=DEV)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if starts is None:
        starts = len(set(ns)) > 1
    out = crm.paged_attention(q, kc, vc, table, ld, starts=starts_of(ns) if starts else None, k_scale=ks, v_scale=vs,
                              lse=lse, **how)
    o, tol, l, ltol = attn_ref.paged(q, kc, vc, table, lens, ns, ks, vs, **how)
    attn_ref.check(out, o, tol)
    attn_ref.check(lse, l, ltol, "lse")
    return out


TYPES = [(BF16, "token"), (E4M3, "head"), (E5M2, "token")]


@pytest.mark.parametrize("dtype,order", TYPES)
@pytest.mark.parametrize("D", [16, 64, 72, 80, 96, 100, 128, 192, 256, 512])
def test_decode_head_sizes(dtype, order, D):
    check_paged(gen(D, order), [1] * 5, [200, 1, 77, 16, 129], 8, 2, D, dtype=dtype, order=order)


@pytest.mark.parametrize("dtype,order", TYPES)
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100, 128])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_pages(dtype, order, page, n):
    check_paged(gen(page, n), [n] * 4, [n, 100, 333, 64], 4, 2, 128, page, dtype, order)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("m", [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 511, 513, 1023, 2049, 5000])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_decode_lengths(dtype, m, window):
    check_paged(gen(m, window), [1, 1], [m, max(1, m // 2)], 8, 2, 128, dtype=dtype, window=window)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 12, 16, 17, 32, 100, 128])
@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_decode_groups(G, dtype):
    check_paged(gen(G), [1] * 3, [300, 40, 1], 2 * G, 2, 64, dtype=dtype)
    check_paged(gen(G, 1), [1] * 3, [300, 40, 1], G, 1, 128, dtype=dtype)


@pytest.mark.parametrize("n", [2, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("window", [0, 3, 50])
def test_drafts(n, G, dtype, window):
    check_paged(gen(n, G), [n] * 4, [n, 90, 257, 130], 2 * G, 2, 128, dtype=dtype, window=window)
    check_paged(gen(n, G), [n] * 4, [n, 90, 257, 130], 2 * G, 2, 128, dtype=dtype, window=window, starts=True)


@pytest.mark.parametrize("dtype,order", TYPES)
@pytest.mark.parametrize("D,G", [(64, 7), (128, 4), (192, 3), (256, 2), (96, 5)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 90), (False, 0)])
def test_chunks(dtype, order, D, G, causal, window):
    ns, lens = [70, 1, 0, 300, 33], [500, 260, 90, 300, 129]
    check_paged(gen(D, G), ns, lens, 2 * G, 2, D, dtype=dtype, order=order, causal=causal, window=window)


@pytest.mark.parametrize("n", [1, 2, 8, 40, 300])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_rows_without_keys(n, dtype):
    # No key, fewer keys than tokens: the first rows see nothing.
    lens = [0, 1, max(1, n // 2), n + 3]
    out = check_paged(gen(n), [n] * 4, lens, 4, 2, 128, dtype=dtype)
    assert (out[:n] == 0).all()
    check_paged(gen(n), [n, 0, n, n], lens, 4, 2, 128, dtype=dtype, starts=True, window=2)


@pytest.mark.parametrize("n", [4, 60])
@pytest.mark.parametrize("bad", [INF, NAN])
def test_rows_without_keys_beside_infinite_values(n, bad):
    # The first rows see nothing; what the others see does not reach them.
    g = gen(n)
    for m, lens in ((n // 2, [n // 2]), (n // 2, [n // 2, 5000])):
        kc, vc, table, _, _ = cache(g, lens, 16, 2, 128)
        vc[int(table[0, 0]), 0] = bad
        q = normal(g, len(lens) * n, 8, 128).to(BF16)
        out = crm.paged_attention(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device=DEV))
        assert (out[:n - m] == 0).all() and not out[n - m:n].isfinite().any()


def test_no_pages():
    q = normal(gen(1), 3, 4, 128).to(BF16)
    kc = torch.empty(0, 16, 2, 128, dtype=BF16, device=DEV)
    table = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    lens = torch.tensor([0, 5, -3], dtype=torch.int32, device=DEV)       # no table: no keys
    for starts in (None, starts_of([1, 1, 1])):
        out = torch.full_like(q, NAN)
        crm.paged_attention(q, kc, kc, table, lens, starts=starts, out=out)
        assert (out == 0).all()
    table = torch.zeros(3, 2, dtype=torch.int32, device=DEV)             # page numbers, but no such page: zeros
    out = crm.paged_attention(q, kc, kc, table, lens)
    assert (out == 0).all()


@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_pages_out_of_range_read_as_zeros(n, dtype):
    g = gen(n)
    kc, vc, table, ks, vs = cache(g, [300, 300], 16, 2, 128, dtype)
    table[0, 3], table[0, 7], table[1, 0] = -1, kc.shape[0], -(1 << 31)
    q = normal(g, 2 * n, 8, 128).to(BF16)
    out = crm.paged_attention(q, kc, vc, table, torch.tensor([300, 300], dtype=torch.int32, device=DEV), k_scale=ks, v_scale=vs)
    o, tol, _, _ = attn_ref.paged(q, kc, vc, table, [300, 300], [n, n], ks, vs)
    attn_ref.check(out, o, tol)


@pytest.mark.parametrize("n", [1, 30])
def test_lengths_beyond_the_table_are_cut(n):
    g = gen(n)
    kc, vc, table, _, _ = cache(g, [64, 64], 16, 2, 128)
    table = table[:, :4].contiguous()
    q = normal(g, 2 * n, 8, 128).to(BF16)
    out = crm.paged_attention(q, kc, vc, table, torch.tensor([(1 << 31) - 1, 64], dtype=torch.int32, device=DEV))
    o, tol, _, _ = attn_ref.paged(q, kc, vc, table, [64, 64], [n, n])
    attn_ref.check(out, o, tol)


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("n", [4, 60])
def test_later_drafts_do_not_matter(bad, n):
    g = gen(n)
    kc, vc, table, _, _ = cache(g, [200], 16, 2, 128)
    q = normal(g, n, 8, 128).to(BF16)
    last = 199
    page, row = int(table[0, last // 16]), last % 16
    kc[page, row], vc[page, row] = bad, bad
    out = crm.paged_attention(q, kc, vc, table, torch.tensor([200], dtype=torch.int32, device=DEV))
    k0, v0 = kc.clone(), vc.clone()
    k0[page, row], v0[page, row] = 0, 0
    o, tol, _, _ = attn_ref.paged(q, k0, v0, table, [200], [n])
    attn_ref.check(out[:-1], o[:-1], tol[:-1])


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -14, 1.0, 2.0 ** 14, 2.0 ** 60])
def test_queries_of_any_size_over_fp8(dtype, n, size):
    # Queries beyond FP16's range either way, rows of different sizes.
    g = gen(n, size)
    q = normal(g, 2 * n, 8, 128) * size * torch.exp2(torch.randint(-9, 9, (2 * n, 8, 1), generator=g, device=DEV).float())
    q[0, 0] = 0
    q[:, 1, 3] = 0
    check_paged(g, [n, n], [150, 300], 8, 2, 128, dtype=dtype, q=q.to(BF16), scale=0.1 / size)


def test_one_long_sequence_is_split():
    # Few rows over many keys: the keys are shared out and the parts joined.
    for n in (1, 4, 17, 64):
        check_paged(gen(n), [n], [20011], 8, 2, 128, page=64)
    check_paged(gen(9), [1, 2, 3], [9000, 2, 12345], 4, 1, 64, dtype=E4M3)


def test_batch_of_many_lengths():
    r = random.Random(4)
    lens = [r.choice([1, 2, 30, 500, 1500]) for _ in range(300)]
    check_paged(gen(3), [1] * 300, lens, 2, 1, 64)
    ns = [min(m, r.choice([0, 1, 1, 1, 5, 100])) for m in lens]
    check_paged(gen(4), ns, lens, 2, 1, 64, starts=True)


def test_cache_beyond_2_31_elements():
    # Pages at element offsets beyond 2^31, one sequence in the last ones.
    pages, page, Hk, D = 2200, 1024, 8, 128
    kc = torch.zeros(pages, page, Hk, D, dtype=BF16, device=DEV)
    vc = torch.zeros(pages, page, Hk, D, dtype=BF16, device=DEV)
    assert kc.numel() > 1 << 31
    g = gen(8)
    kc[-2:], vc[-2:] = normal(g, 2, page, Hk, D).to(BF16), normal(g, 2, page, Hk, D).to(BF16)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    for n in (1, 20):
        q = normal(g, n, 16, D).to(BF16)
        out = crm.paged_attention(q, kc, vc, table, torch.tensor([1500], dtype=torch.int32, device=DEV))
        o, tol, _, _ = attn_ref.paged(q, kc, vc, table, [1500], [n])
        attn_ref.check(out, o, tol)


def test_prompt_beyond_2_31_elements():
    T, Hq, Hk, D = 1 << 20, 16, 1, 128
    x = torch.zeros(T, Hq + 2 * Hk, D, dtype=BF16, device=DEV)
    assert x.numel() > 1 << 31
    g = gen(1)
    x[-700:] = normal(g, 700, Hq + 2 * Hk, D).to(BF16)
    q, k, v = x.split([Hq, Hk, Hk], 1)
    ns = [T - 700 - 10, 400, 300]
    starts = torch.tensor([T - 700, T - 300, T], dtype=torch.int32, device=DEV)
    out = torch.zeros(T, Hq, D, dtype=BF16, device=DEV)
    crm.prompt_attention(q, k, v, starts=starts, out=out)
    o, tol, _, _ = attn_ref.prompt(q[-700:], k[-700:], v[-700:], ns[1:])
    attn_ref.check(out[-700:], o, tol)
    assert not out[:-700].any()


# ------------------------------------------------------- how it is called --

def test_outputs_given_and_strided():
    g = gen(1)
    q, k, v = heads(g, 77, 4, 2, 128)
    wide = torch.zeros(77, 4, 256, dtype=BF16, device=DEV)
    ws = torch.empty(crm.attention_workspace_bytes(128), dtype=torch.uint8, device=DEV)
    out = crm.prompt_attention(q, k, v, out=wide[..., 128:], workspace=ws)
    assert out.data_ptr() == wide[..., 128:].data_ptr()
    assert torch.equal(wide[..., 128:], crm.prompt_attention(q, k, v)) and not wide[..., :128].any()


@pytest.mark.parametrize("n", [1, 50])
def test_runs_alike_and_with_any_workspace(n):
    g = gen(n)
    lens = [3000, 700, 5000]
    kc, vc, table, _, _ = cache(g, lens, 16, 2, 128)
    q = normal(g, 3 * n, 8, 128).to(BF16)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    first = crm.paged_attention(q, kc, vc, table, ld)
    for fill in (0, 255, 0x7f):
        ws = torch.full((crm.attention_workspace_bytes(128),), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(first, crm.paged_attention(q, kc, vc, table, ld, workspace=ws))


@pytest.mark.parametrize("n", [1, 50])
def test_graph_replays_follow_the_lengths(n):
    # One captured step serves growing sequences: lengths and pages are read on the device.
    g = gen(n)
    lens = [3000, 700]
    kc, vc, table, _, _ = cache(g, lens, 16, 2, 128)
    q = normal(g, 2 * n, 8, 128).to(BF16)
    ld = torch.tensor([1000, 300], dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        crm.paged_attention(q, kc, vc, table, ld, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        crm.paged_attention(q, kc, vc, table, ld, out=out)
        crm.paged_attention(q, kc, vc, table, ld, out=out)
    for now in ([1000, 300], [3000, 1], [0, 700]):
        ld.copy_(torch.tensor(now, dtype=torch.int32))
        q.copy_(normal(g, *q.shape))
        graph.replay()
        o, tol, _, _ = attn_ref.paged(q, kc, vc, table, now, [n, n])
        attn_ref.check(out, o, tol)


def test_streams():
    # Two streams at once, each call with its own workspace.
    g = gen(1)
    lens = [4000, 100]
    kc, vc, table, _, _ = cache(g, lens, 16, 2, 128)
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = [normal(g, 2 * n, 8, 128).to(BF16) for n in (1, 40, 1, 40)]
    want = [crm.paged_attention(q, kc, vc, table, ld) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append(crm.paged_attention(q, kc, vc, table, ld))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_serving_as_it_is_used(dtype):
    """A prompt in two chunks, then tokens one by one: each appended to the
    cache, then attended; against prompt_attention of the whole text and FP64."""
    g = gen(7)
    T, Hq, Hk, D, page = 230, 8, 2, 128, 16
    x = normal(g, T, Hq + 2 * Hk, D).to(BF16)
    q, k, v = x.split([Hq, Hk, Hk], 1)
    wq, wk = (1 + 0.1 * normal(g, 2, D)).to(BF16)
    cs = crm.rope_cos_sin(torch.arange(T, device=DEV), torch.rand(D // 2, generator=g, device=DEV))
    q1, k1 = crm.qk_rmsnorm_rope_fwd(q, k, wq, wk, cs)
    whole = crm.prompt_attention(q1, k1, v)
    o, tol, _, _ = attn_ref.prompt(q1, k1, v, [T])
    attn_ref.check(whole, o, tol)
    pages = torch.randperm(20, generator=g, device=DEV).to(torch.int32)[None]
    kc, vc = (torch.zeros(20, page, Hk, D, device=DEV).to(dtype) for _ in range(2))
    one = None if dtype == BF16 else torch.full((1,), 0.05, device=DEV)
    for a, b in [(0, 100), (100, 220)] + [(t, t + 1) for t in range(220, T)]:
        t = torch.arange(a, b, device=DEV)
        slots = pages[0, t // page].long() * page + t % page
        qa = crm.qk_rmsnorm_rope_append(q[a:b], k[a:b], v[a:b], wq, wk, cs[a:b], kc, vc, slots, k_scale=one, v_scale=one)
        ld = torch.tensor([b], dtype=torch.int32, device=DEV)
        out = crm.paged_attention(qa, kc, vc, pages, ld, k_scale=one, v_scale=one)
        if dtype == BF16:
            attn_ref.check(out, o[a:b], tol[a:b])
        o2, tol2, _, _ = attn_ref.paged(qa, kc, vc, pages, [b], [b - a], one, one)
        attn_ref.check(out, o2, tol2)


def test_random_shapes():
    r = random.Random(11)
    for i in range(60):
        D = r.choice([16, 40, 64, 64, 80, 96, 128, 128, 128, 136, 192, 256])
        Hk, G = r.choice([1, 2, 3]), r.choice([1, 2, 3, 4, 5, 8])
        B = r.randint(1, 9)
        window = r.choice([0, 0, r.randint(1, 300)])
        g = gen(i)
        if r.random() < 0.4:
            ns = [r.choice([0, 1, r.randint(1, 60), r.randint(1, 600)]) for _ in range(B)]
            if sum(ns):
                q, k, v = heads(g, sum(ns), Hk * G, Hk, D, r.choice(["packed", "heads", "gated"]))
                check_prompt(q, k, v, ns, True, causal=bool(window) or r.random() < 0.7, window=window)
            continue
        n = r.choice([1, 1, 2, 3, 7, 20, 130])
        lens = [r.choice([n, r.randint(1, 300), r.randint(1, 3000)]) for _ in range(B)]
        ns = [n] * B if r.random() < 0.6 else [r.choice([1, n]) for _ in range(B)]
        check_paged(g, ns, lens, Hk * G, Hk, D, r.choice([1, 5, 16, 32, 128]), r.choice([BF16, E4M3, E5M2]),
                    r.choice(["token", "head"]), window=window)


@pytest.mark.parametrize("Hk,G", [(90, 1), (160, 1), (200, 2)])
def test_more_key_heads_than_processors(Hk, G):
    # One group of CTAs, or CTAs beyond those that run at once.
    q, k, v = heads(gen(Hk), 700, Hk * G, Hk, 64)
    check_prompt(q, k, v, [130, 570], True)
    check_prompt(q[:70], k[:70], v[:70], [70], False)
    check_paged(gen(Hk, 1), [1, 1], [900, 5], Hk * G, Hk, 64)


@pytest.mark.parametrize("n", [639, 640, 641])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_around_the_short_form(n, D):
    g = gen(n, D)
    for B in (1, 3):
        q, k, v = (normal(g, B, n, H, D).to(BF16) for H in (4, 2, 2))
        out = crm.prompt_attention(q, k, v)
        o, tol, _, _ = attn_ref.prompt(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), [n] * B)
        attn_ref.check(out.flatten(0, 1), o, tol)
    check_paged(g, [1, 1, 1], [n, 7, n // 2], 8, 2, D, dtype=E4M3)
    check_paged(g, [20, 20], [n, 64], 8, 2, D, page=1)


def test_short_calls_of_many_sequences():
    r = random.Random(2)
    lens = [r.randint(0, 500) for _ in range(700)]
    check_paged(gen(1), [1] * 700, lens, 4, 2, 64)
    check_paged(gen(2), [9] * 60, [r.randint(9, 400) for _ in range(60)], 6, 3, 128)
    q, k, v = (normal(gen(3), 90, 33, H, 64).to(BF16) for H in (6, 3, 3))
    o, tol, _, _ = attn_ref.prompt(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), [33] * 90)
    attn_ref.check(crm.prompt_attention(q, k, v).flatten(0, 1), o, tol)


def test_many_pieces_of_one_half_beside_long_ones():
    # Long tiles of two halves between many short ones, whose halves a CTA works through at their own pace.
    ns = [300] + [1, 3, 20] * 60 + [500, 2, 2, 2, 700] + [5] * 90
    q, k, v = heads(gen(6), sum(ns), 5, 1, 128)
    check_prompt(q, k, v, ns, True)
    check_paged(gen(7), ns, [n + 200 for n in ns], 5, 1, 128, dtype=E4M3)


@pytest.mark.parametrize("window", [(1 << 31) - 1, 1 << 40, 5000])
def test_windows_beyond_the_sequence(window):
    q, k, v = heads(gen(window), 300, 4, 2, 128)
    a, b = crm.prompt_attention(q, k, v, window=window), crm.prompt_attention(q, k, v)
    assert torch.equal(a, b)
    check_paged(gen(1), [40, 40], [10, 300], 4, 2, 128, window=window if window < 1 << 31 else 0)


def test_refusals():
    g = gen(1)
    q, k, v = heads(g, 20, 4, 2, 128)
    starts = starts_of([20])
    kc, vc, table, _, _ = cache(g, [20], 16, 2, 128)
    lens = torch.tensor([20], dtype=torch.int32, device=DEV)
    for bad in (dict(starts=starts.long()), dict(starts=starts.cpu()), dict(out=torch.empty(20, 4, 128, device=DEV))):
        with pytest.raises(TypeError):
            crm.prompt_attention(q, k, v, **bad)
    for bad in (dict(k=k[:, :, :64], v=v), dict(k=k[:10], v=v[:10]), dict(k=k, v=v[:, :1])):
        with pytest.raises(ValueError):
            crm.prompt_attention(q, **bad)
    with pytest.raises(ValueError):
        crm.prompt_attention(q[:, :3], k, v)                              # 3 heads over 2
    with pytest.raises(ValueError):
        crm.prompt_attention(q, k, v, lse=torch.empty(20, 3, device=DEV))
    for bad in (dict(scale=-1.0), dict(window=-1), dict(causal=False, window=4), dict(out=q)):
        with pytest.raises(crm.CrmsnError):
            crm.prompt_attention(q, k, v, **bad)
    long = heads(g, 700, 4, 2, 128)
    with pytest.raises(crm.CrmsnError):
        crm.prompt_attention(*long, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(RuntimeError):
        crm.prompt_attention(q.clone().requires_grad_(), k, v)
    with torch.no_grad():
        crm.prompt_attention(q.clone().requires_grad_(), k, v)
    for bad in (dict(lens=lens.long()), dict(page_table=table.long()), dict(k_cache=kc.float(), v_cache=vc.float()),
                dict(k_cache=kc.to(E4M3), v_cache=vc.to(E5M2)), dict(k_cache=kc.to(E4M3), v_cache=vc.to(E4M3))):
        with pytest.raises(TypeError):
            crm.paged_attention(**{**dict(q=q, k_cache=kc, v_cache=vc, page_table=table, lens=lens), **bad})
    for bad in (dict(page_table=table[:0]), dict(page_table=table.repeat(2, 1)), dict(lens=lens[:0]), dict(k_cache=kc[..., :64], v_cache=vc[..., :64]),
                dict(k_scale=torch.ones(1, device=DEV))):
        with pytest.raises(ValueError):
            crm.paged_attention(**{**dict(q=q, k_cache=kc, v_cache=vc, page_table=table, lens=lens), **bad})
    with pytest.raises(ValueError):
        crm.paged_attention(q[:19], kc, vc, table.repeat(2, 1), lens.repeat(2))   # 19 tokens over 2 sequences


def test_empty_calls():
    q, k, v = heads(gen(1), 0, 4, 2, 128)
    assert crm.prompt_attention(q, k, v).shape == (0, 4, 128)
    q, k, v = heads(gen(1), 9, 4, 2, 128)
    out = torch.full_like(q.contiguous(), 3.0)
    crm.prompt_attention(q, k, v, starts=starts_of([]), out=out)              # no sequence
    assert (out == 3).all()
    kc = torch.zeros(3, 16, 2, 128, dtype=BF16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert crm.paged_attention(q[:0], kc, kc, none.view(0, 4), none).shape == (0, 4, 128)


@pytest.mark.parametrize("G", [1, 5])
def test_short_ragged_calls(G):
    r = random.Random(G)
    for i in range(8):
        ns = [r.choice([0, 0, 1, 2, 30, 90]) for _ in range(r.choice([1, 5, 40, 700]))]
        while sum(ns) > 640:
            ns[r.randrange(len(ns))] = 0
        q, k, v = heads(gen(i, G), sum(ns), 2 * G, 2, 64)
        if sum(ns):
            check_prompt(q, k, v, ns, True, window=r.choice([0, 20]))
        ns = [r.choice([0, 1, 1, 7, 60]) for _ in range(r.choice([3, 50]))]
        check_paged(gen(i, G), ns, [n + r.randint(0, 400) for n in ns], 2 * G, 2, 128, dtype=r.choice([BF16, E4M3]))
