"""The query / key functions on the GPU against their FP64 forms (qk_ref),
with the bounds derived there; layouts, masks of the cache, limits, graphs,
streams, and runs of the functions together as a model uses them."""
import threading

import pytest
import torch

import normalization_rmsnorm_fwd_gb300 as crm
import qk_ref
from normalization_rmsnorm_fwd_gb300 import autograd as ag
from normalization_rmsnorm_fwd_gb300.binding import CrmsnError

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, E4M3, E5M2 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2


def gen(seed):
    return torch.Generator().manual_seed(seed)


def heads(g, T, H, D, layout="plain", scale=1.0):
    """A BF16 [T, H, D] on the GPU in one of the layouts, with its CPU copy."""
    x = (scale * torch.randn(T, H, D, generator=g) * torch.exp(0.5 * torch.randn(T, H, 1, generator=g))).to(BF16)
    if layout == "gated":
        buf = torch.full((T, H, 2 * D), 9.0, dtype=BF16, device=DEV)
        t = buf[..., :D]
    elif layout == "packed":
        buf = torch.full((T, H + 3, D), 9.0, dtype=BF16, device=DEV)
        t = buf[:, 2:2 + H]
    elif layout == "heads":
        t = torch.empty(H, T, D, dtype=BF16, device=DEV).transpose(0, 1)
    elif layout in ("odd", "off4", "off8"):      # 2, 4 or 8 bytes off: the element-wise form, 4- and 8-byte accesses
        n = {"odd": 1, "off4": 2, "off8": 4}[layout]
        t = torch.empty(T * H * D + n, dtype=BF16, device=DEV)[n:].view(T, H, D)
    else:
        t = torch.empty(T, H, D, dtype=BF16, device=DEV)
    t.copy_(x)
    return t, x


def weights(g, D, kind):
    if kind is None:
        return None, None, 0.0
    wq, wk = 1 + 0.2 * torch.randn(D, generator=g), 1 + 0.2 * torch.randn(D, generator=g)
    if kind == "f32":
        return (wq - 1).to(DEV), (wk - 1).to(DEV), 1.0
    return wq.to(BF16).to(DEV), wk.to(BF16).to(DEV), 0.25 if kind == "bias" else 0.0


def rotation(g, P, R):
    if R == 0:
        return None
    return qk_ref.angles(torch.randint(100000, (1, P), generator=g), 1e4 ** (-torch.arange(R // 2) / max(1, R // 2))).float().to(DEV)


def cpu(t):
    return None if t is None else t.cpu()


# T, Hq, Hk, D, R, pairs, weight, layout, tokens that share the rotations
SHAPES = [
    (1, 32, 8, 128, 128, False, "bf16", "plain", 1),
    (7, 5, 1, 128, 128, True, "f32", "packed", 7),
    (33, 4, 4, 64, 64, False, "bias", "gated", 33),
    (40, 3, 2, 64, 32, True, "bf16", "heads", 20),
    (19, 15, 5, 80, 32, False, "f32", "plain", 19),
    (21, 7, 3, 96, 96, True, "bf16", "plain", 21),
    (11, 2, 1, 256, 64, False, "f32", "gated", 11),
    (9, 3, 2, 512, 512, False, "bf16", "plain", 9),
    (6, 3, 1, 264, 16, True, "bf16", "packed", 2),
    (50, 3, 1, 8, 0, False, "bf16", "plain", 50),
    (50, 9, 2, 16, 16, False, "bf16", "plain", 50),
    (25, 9, 2, 24, 16, True, None, "plain", 25),
    (300, 40, 40, 128, 128, True, "bf16", "plain", 300),
    (3000, 20, 4, 64, 64, False, "bf16", "plain", 1000),
    (37, 3, 2, 64, 64, False, "bf16", "plain", 1),         # one rotation for all tokens
    (12, 3, 2, 128, 0, False, "f32", "plain", 12),
    (12, 3, 2, 128, 128, False, None, "plain", 12),
    # 8- and 4-byte accesses: pieces that end inside a lane
    (15, 3, 2, 72, 72, False, "bf16", "plain", 15),
    (700, 16, 16, 72, 72, True, "f32", "packed", 700),
    (31, 5, 5, 88, 88, False, "bias", "gated", 31),
    (22, 4, 1, 40, 40, True, "bf16", "heads", 11),
    (22, 4, 1, 100, 100, False, "bf16", "plain", 22),
    (1300, 7, 3, 100, 20, True, "f32", "plain", 1300),
    (9, 2, 2, 44, 8, False, None, "plain", 9),
    (23, 5, 3, 128, 128, False, "bf16", "off8", 23),
    (23, 5, 3, 128, 64, True, "bf16", "off4", 23),
    (6, 2, 1, 470, 440, False, "f32", "plain", 6),
    (30, 2, 1, 12, 0, False, "bf16", "off4", 30),
    # the element-wise form
    (13, 3, 2, 2, 2, True, "bf16", "plain", 13),
    (13, 3, 2, 6, 4, False, "f32", "plain", 13),
    (17, 5, 3, 128, 128, False, "bf16", "odd", 17),
    (17, 5, 3, 100, 50, False, "bf16", "gated", 17),
    (5, 2, 1, 510, 500, True, "bias", "plain", 5),
    (2000, 9, 1, 72, 72, False, None, "plain", 2000),
    (1500, 6, 2, 120, 40, True, "f32", "heads", 500),
    (4, 3, 0, 128, 128, False, "bf16", "plain", 4),       # queries alone
    (4, 3, 0, 126, 126, False, "bf16", "odd", 4),
]


@pytest.mark.parametrize("T,Hq,Hk,D,R,pairs,weight,layout,P", SHAPES)
def test_forward(T, Hq, Hk, D, R, pairs, weight, layout, P):
    g = gen(T + D)
    q, qc = heads(g, T, Hq, D, layout)
    k, kc = heads(g, T, Hk, D, layout) if Hk else (None, None)
    wq, wk, bias = weights(g, D, weight)
    cs = rotation(g, P, R)
    yq, yk = crm.qk_rmsnorm_rope_fwd(q, k, wq, wk if Hk else None, cs, 1e-5, bias, pairs)
    qk_ref.check(yq, *qk_ref.forward(qc, cpu(wq), cpu(cs), 1e-5, bias, pairs), what="q")
    if Hk:
        qk_ref.check(yk, *qk_ref.forward(kc, cpu(wk), cpu(cs), 1e-5, bias, pairs), what="k")
    else:
        assert yk is None
    # In place, in the inputs' own layouts: the same bits, nothing beside them.
    crm.qk_rmsnorm_rope_fwd(q, k, wq, wk if Hk else None, cs, 1e-5, bias, pairs, q_out=q, k_out=k)
    assert torch.equal(q, yq) and (not Hk or torch.equal(k, yk))
    if layout == "gated":
        assert (q._base[..., D:] == 9).all()
    if layout == "packed":
        assert (q._base[:, :2] == 9).all() and (q._base[:, 2 + Hq:] == 9).all()


@pytest.mark.parametrize("T,Hq,Hk,D,R,pairs,weight,layout,P", SHAPES)
def test_backward(T, Hq, Hk, D, R, pairs, weight, layout, P):
    g = gen(2 * T + D)
    q, qc = heads(g, T, Hq, D, layout)
    gq, gqc = heads(g, T, Hq, D, layout if layout in ("odd", "off4", "off8") else "plain", 0.02)
    (k, kc), (gk, gkc) = (heads(g, T, Hk, D, layout), heads(g, T, Hk, D, "plain", 0.02)) if Hk else ((None, None), (None, None))
    wq, wk, bias = weights(g, D, weight)
    wk = wk if Hk else None
    cs = rotation(g, P, R)
    dq, dk, dwq, dwk = crm.qk_rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, cs, 1e-5, bias, pairs)
    for name, d, dw, gc, xc, w in (("q", dq, dwq, gqc, qc, wq), ("k", dk, dwk, gkc, kc, wk)):
        if name == "k" and not Hk:
            assert d is None and dw is None
            continue
        rdx, bdx, rdw, bdw = qk_ref.backward(gc, xc, cpu(w), cpu(cs), 1e-5, bias, pairs)
        qk_ref.check(d, rdx, bdx, what="d" + name)
        assert (dw is None) == (w is None)
        if w is not None:
            qk_ref.check(dw, rdw, bdw, what="dw" + name)
    # The same bits again, into the gradients' own storage.
    again = crm.qk_rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, cs, 1e-5, bias, pairs, dq=gq, dk=gk)
    for a, b in zip(again, (dq, dk, dwq, dwk)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_weight_gradients_depend_on_sizes_and_access_width_alone():
    # dw's bits: the same for any strides and bases of one access width; other
    # widths add in another order, within the bound.
    g = gen(24)
    T, Hq, Hk, D = 3000, 6, 2, 128
    (q, qc), (k, _), (gq, gc), (gk, _) = (heads(g, T, h, D) for h in (Hq, Hk, Hq, Hk))
    wq, wk, _ = weights(g, D, "bf16")
    cs = rotation(g, T, D)
    want = crm.qk_rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, cs)
    for layout in ("gated", "packed", "heads"):
        a, b, c, d = (heads(g, T, t.shape[1], D, layout)[0].copy_(t) for t in (gq, gk, q, k))
        got = crm.qk_rmsnorm_rope_bwd(a, b, c, d, wq, wk, cs)
        assert all(torch.equal(x, y) for x, y in zip(got, want)), layout
    _, _, rdw, bdw = qk_ref.backward(gc, qc, cpu(wq), cpu(cs))
    for layout in ("off8", "off4", "odd"):
        a = heads(g, T, Hq, D, layout)[0].copy_(gq)
        got = crm.qk_rmsnorm_rope_bwd(a, None, q, None, wq, None, cs)
        qk_ref.check(got[2], rdw, bdw, what=layout)
        assert torch.equal(crm.qk_rmsnorm_rope_bwd(a, None, q, None, wq, None, cs)[2], got[2])


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,R,sections,mixed", [(1, 128, None, False), (77, 2, None, False), (5, 126, None, False), (1000, 64, [32], False),
                                                (63, 128, [16, 24, 24], False), (63, 80, [0, 17, 23], False), (40, 128, [22, 21, 21], True),
                                                (9, 20, [6, 4], True), (3, 512, [64, 64, 64, 64], True), (5000, 96, [16, 16, 16], False)])
def test_angles(T, R, sections, mixed, kind):
    g = gen(T + R)
    axes = len(sections or [0])
    pos = torch.randint(-1 << 28, 1 << 28, (axes, T), generator=g)
    pos[:, :T // 2] = torch.randint(0, 5000, (axes, T // 2), generator=g)
    pos[0, 0] = 0
    f = 1e6 ** (-torch.arange(R // 2, dtype=torch.float64) / (R // 2))
    f = f.float()
    p = pos if axes > 1 else pos[0]
    out = crm.rope_cos_sin(p.to(kind).to(DEV), f.to(DEV), sections, mixed, 0.75)
    assert out.shape == (T, R)
    # The polynomials' steps (at most 2 u of values up to 1), the angle's
    # rounding (an eighth of a turn in 24 bits, times pi: below u) and the
    # scaling's: below 6 u of the scaling.
    exact = qk_ref.angles(pos, f, sections, mixed, 0.75)
    assert ((out.cpu().double() - exact).abs() <= 6 * 2.0 ** -24 * 0.75).all()
    assert out[0, 0] == 0.75 or axes > 1 and sections[0] == 0


def test_angles_far_positions_and_odd_frequencies():
    # Whole frequencies and positions whose product is known modulo 2 pi by
    # integer arithmetic alone: cos(p f) with f = m / 2^k as exact fractions.
    from fractions import Fraction
    import math
    # 2 pi to 200 bits by Machin's formula.
    def arctan_inv(n):
        s, t, k = Fraction(0), Fraction(1, n), 0
        while abs(t) > Fraction(1, 1 << 220):
            s += t / (2 * k + 1) * (-1) ** k
            t /= n * n
            k += 1
        return s
    two_pi = 8 * (4 * arctan_inv(5) - arctan_inv(239))
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 + 12345, 2 ** 32 - 1, 123456789]
    freqs = [1.0, 0.1, 1e-6, 3.0, 12345.678, -0.5, 2.0 ** 39, 0.0]
    f = torch.tensor(freqs, dtype=torch.float32)
    out = crm.rope_cos_sin(torch.tensor(pos, device=DEV), f.to(DEV)).cpu().double()
    for i, p in enumerate(pos):
        for j, x in enumerate(f.tolist()):
            a = Fraction(x) * p % two_pi
            # 6 u as above and the angle's own bound, 2^-61 |p|.
            assert abs(float(out[i, j]) - math.cos(a)) <= 6 * 2.0 ** -24 + 2.0 ** -29, (p, x)
            assert abs(float(out[i, 8 + j]) - math.sin(a)) <= 6 * 2.0 ** -24 + 2.0 ** -29, (p, x)
    bad = torch.tensor([float("nan"), float("inf"), 2.0 ** 40, 1.0], device=DEV)
    out = crm.rope_cos_sin(torch.tensor([3], device=DEV), bad)
    assert out.isnan().tolist() == [[True, True, True, False] * 2]


def test_angles_of_opposite_positions():
    # cos(-a) = cos(a) and sin(-a) = -sin(a) to the bit, far and near.
    g = gen(23)
    f = torch.cat([torch.rand(24, generator=g), 10.0 ** -torch.arange(40)]).to(DEV)
    pos = torch.cat([torch.arange(500), torch.randint(1 << 31, (500,), generator=g)]).to(DEV)
    a, b = crm.rope_cos_sin(pos, f), crm.rope_cos_sin(-pos, f)
    assert torch.equal(a[:, :64], b[:, :64]) and torch.equal(a[:, 64:], -b[:, 64:])


def test_angles_next_to_a_whole_turn():
    # Small angles of either sign keep the angle's bound, 2^-61 |p|, and the
    # sine's few roundings of itself: the rest of a turn within 2^-22 of
    # itself (two halves and their sum round), the polynomial's steps 2^-22.
    pos = torch.tensor([1, -1, 2, -2, 3, -3, 1000, -1000, 12345, -12345])
    f = torch.tensor([1e-9, 3e-10, 1e-10, 3e-11, 1e-11, 1e-12, 1e-14, 1e-16, 1e-18, 2.0 ** -62], dtype=torch.float32)
    out = crm.rope_cos_sin(pos.to(DEV), f.to(DEV)).cpu().double()
    exact = (pos.double()[:, None] * f.double()).sin()
    assert ((out[:, 10:] - exact).abs() <= 2.0 ** -61 * pos.double().abs()[:, None] + 2.0 ** -21 * exact.abs()).all()
    assert (out[:, :10] == 1).all()


def test_angles_layouts_and_empty():
    f = torch.rand(16, device=DEV)
    pos = torch.randint(9999, (3, 4, 5), device=DEV)
    whole = crm.rope_cos_sin(pos, f, [6, 5, 5])
    assert whole.shape == (4, 5, 32)
    assert torch.equal(whole.view(20, 32), crm.rope_cos_sin(pos.view(3, 20), f, [6, 5, 5]))
    wide = torch.randint(9999, (3, 40), device=DEV)
    wide[:, :20] = pos.view(3, 20)
    guard = torch.full((20, 48), 7.0, device=DEV)
    crm.rope_cos_sin(wide[:, :20], f, [6, 5, 5], out=guard[:, 4:36])
    assert torch.equal(guard[:, 4:36], whole.view(20, 32)) and (guard[:, :4] == 7).all() and (guard[:, 36:] == 7).all()
    odd = torch.full((20, 33), 7.0, device=DEV)
    crm.rope_cos_sin(wide[:, :20], f, [6, 5, 5], out=odd[:, :32])          # rows of no 16-byte alignment
    assert torch.equal(odd[:, :32], whole.view(20, 32)) and (odd[:, 32] == 7).all()
    assert crm.rope_cos_sin(torch.zeros(0, dtype=torch.int64, device=DEV), f).shape == (0, 32)


@pytest.mark.parametrize("mixed", [False, True])
def test_angles_of_text_alone_are_those_of_one_axis(mixed):
    # One position per token, expanded over the axes, in both column orders.
    f = torch.rand(32, device=DEV)
    pos = torch.randint(1 << 20, (4, 25), device=DEV)
    one = crm.rope_cos_sin(pos, f)
    assert torch.equal(crm.rope_cos_sin(pos.expand(3, 4, 25), f, [12, 10, 10], mixed), one)


def test_rows_do_not_depend_on_their_call():
    # A token's outputs are the same bits alone, in a larger batch, with other
    # heads, and in the appended form.
    g = gen(5)
    T, Hq, Hk, D = 500, 12, 4, 128
    q, _ = heads(g, T, Hq, D)
    k, _ = heads(g, T, Hk, D)
    v, _ = heads(g, T, Hk, D)
    wq, wk, _ = weights(g, D, "bf16")
    cs = rotation(g, T, D)
    yq, yk = crm.qk_rmsnorm_rope_fwd(q, k, wq, wk, cs)
    for t in (0, 17, 499):
        a, b = crm.qk_rmsnorm_rope_fwd(q[t:t + 1], k[t:t + 1], wq, wk, cs[t:t + 1])
        assert torch.equal(a, yq[t:t + 1]) and torch.equal(b, yk[t:t + 1])
        a, _ = crm.qk_rmsnorm_rope_fwd(q[t:t + 1, 3:4], None, wq, None, cs[t:t + 1])
        assert torch.equal(a, yq[t:t + 1, 3:4])
    kc, vc = (torch.zeros(T, 1, Hk, D, dtype=BF16, device=DEV) for _ in range(2))
    a = crm.qk_rmsnorm_rope_append(q, k, v, wq, wk, cs, kc, vc, torch.arange(T, device=DEV))
    assert torch.equal(a, yq) and torch.equal(kc[:, 0], yk) and torch.equal(vc[:, 0], v)


def test_empty():
    w = torch.ones(64, dtype=BF16, device=DEV)
    z = torch.zeros(0, 3, 64, dtype=BF16, device=DEV)
    cs = torch.zeros(1, 64, device=DEV)
    a, b = crm.qk_rmsnorm_rope_fwd(z, z, w, w, cs)
    assert a.shape == b.shape == z.shape
    dw = torch.full((64,), 5.0, device=DEV)
    _, _, dwq, dwk = crm.qk_rmsnorm_rope_bwd(z, z, z, z, w, w, cs, dwq=dw)
    assert (dwq == 0).all() and (dwk == 0).all() and dwq is dw
    cache = torch.full((2, 4, 3, 64), 3.0, dtype=BF16, device=DEV)
    crm.qk_rmsnorm_rope_append(z, z, z, w, w, cs, cache, cache.clone(), torch.zeros(0, dtype=torch.int64, device=DEV))
    assert (cache == 3).all()


def test_no_key_heads():
    # Keys of no heads: outputs of no heads, a zero weight gradient.
    g = gen(6)
    q, _ = heads(g, 5, 2, 64)
    k = torch.zeros(5, 0, 64, dtype=BF16, device=DEV)
    wq, wk, _ = weights(g, 64, "f32")
    cs = rotation(g, 5, 64)
    a, b = crm.qk_rmsnorm_rope_fwd(q, k, wq, wk, cs)
    assert torch.equal(a, crm.qk_rmsnorm_rope_fwd(q, None, wq, None, cs)[0]) and b.shape == k.shape
    dwk = torch.full((64,), 5.0, device=DEV)
    out = crm.qk_rmsnorm_rope_bwd(a, b, q, k, wq, wk, cs, dwk=dwk)
    one = crm.qk_rmsnorm_rope_bwd(a, None, q, None, wq, None, cs)
    assert torch.equal(out[0], one[0]) and torch.equal(out[2], one[2]) and (dwk == 0).all()


def test_batches_are_rows_of_tokens():
    # [batch, sequence, heads, D] tensors, [batch, sequence] positions and
    # slots: the bits of the same tokens in one dimension.
    g = gen(7)
    B, S, Hq, Hk, D = 3, 11, 4, 2, 64
    (q, _), (k, _), (v, _) = (heads(g, B * S, h, D) for h in (Hq, Hk, Hk))
    wq, wk, _ = weights(g, D, "bf16")
    pos, f = torch.randint(999, (B, S), generator=g).to(DEV), torch.rand(D // 2, device=DEV)
    cs, flat = crm.rope_cos_sin(pos, f), crm.rope_cos_sin(pos.view(-1), f)
    assert cs.shape == (B, S, D) and torch.equal(cs.view(-1, D), flat)
    q4, k4, v4 = (t.view(B, S, -1, D) for t in (q, k, v))
    want = crm.qk_rmsnorm_rope_fwd(q, k, wq, wk, flat)
    got = crm.qk_rmsnorm_rope_fwd(q4, k4, wq, wk, cs, q_out=torch.empty_like(q4))
    assert all(torch.equal(a.view(b.shape), b) for a, b in zip(got, want))
    want = crm.qk_rmsnorm_rope_bwd(q, k, q, k, wq, wk, flat)
    got = crm.qk_rmsnorm_rope_bwd(q4, k4, q4, k4, wq, wk, cs, dk=torch.empty_like(k4))
    assert all(torch.equal(a.view(b.shape), b) for a, b in zip(got, want))
    kc, vc = (torch.zeros(5, 8, Hk, D, dtype=BF16, device=DEV) for _ in range(2))
    slots = torch.randperm(40, generator=g)[:B * S].view(B, S).to(DEV)
    crm.qk_rmsnorm_rope_append(q4, k4, v4, wq, wk, cs, kc, vc, slots)
    assert torch.equal(vc.view(40, Hk, D)[slots], v4)
    # The rotations of one sequence for every sequence of the batch.
    got = crm.qk_rmsnorm_rope_fwd(q4, k4, wq, wk, cs[1])
    want = crm.qk_rmsnorm_rope_fwd(q, k, wq, wk, cs[1:2].expand(B, S, D).reshape(-1, D))
    assert all(torch.equal(a.view(b.shape), b) for a, b in zip(got, want))


def test_dimensions_of_size_one():
    # Single frames whose padding is cut off have no one token stride: direct
    # calls refuse them, autograd copies them.
    g = gen(21)
    B, S, H, D = 2, 5, 3, 64
    frames = torch.randn(B, 1, 8, H, D, generator=g).to(BF16).to(DEV)[:, :, :S]
    x, gr = frames.contiguous(), torch.randn(B, 1, S, H, D, generator=g).to(BF16).to(DEV)
    w, cs = weights(g, D, "bf16")[0], rotation(g, S, D)
    cache, slots = torch.zeros(B * S, 1, H, D, dtype=BF16, device=DEV), torch.arange(B * S, device=DEV)
    with pytest.raises(ValueError):
        crm.qk_rmsnorm_rope_fwd(frames, None, w, None, cs)
    with pytest.raises(ValueError):
        crm.qk_rmsnorm_rope_fwd(x, None, w, None, cs, q_out=frames)
    with pytest.raises(ValueError):
        crm.qk_rmsnorm_rope_bwd(gr, None, frames, None, w, None, cs)
    with pytest.raises(ValueError):
        crm.qk_rmsnorm_rope_append(None, frames, x, None, w, cs, cache, cache.clone(), slots)
    y, _ = crm.qk_rmsnorm_rope_fwd(x, None, w, None, cs)
    dq, _, dw, _ = crm.qk_rmsnorm_rope_bwd(gr, None, x, None, w, None, cs)
    leaf, weight = frames.detach().requires_grad_(), w.clone().requires_grad_()
    z, _ = crm.qk_rmsnorm_rope(leaf, None, weight, None, cs)
    a, b = torch.autograd.grad(z, (leaf, weight), gr)
    assert torch.equal(z, y) and torch.equal(a, dq) and torch.equal(b, dw.to(BF16))
    # One token of each sequence in [B, heads, 1, D] storage is read in place.
    one = torch.randn(7, H, 1, D, generator=g).to(BF16).to(DEV).transpose(1, 2)
    y, _ = crm.qk_rmsnorm_rope_fwd(one, None, w, None, cs[:1])
    assert torch.equal(y, crm.qk_rmsnorm_rope_fwd(one.contiguous(), None, w, None, cs[:1])[0])


def test_special_values_stay_in_their_rows():
    # Infinities, NaN, zeros and the largest values give what the formula
    # gives, in their own row only (their own pair only, without norms).
    g = gen(8)
    T, H, D = 8, 3, 64
    q, _ = heads(g, T, H, D)
    clean = q.clone()
    q[1, 1, 5], q[2, 0, 40], q[3, 2], q[4, 1, :] = float("inf"), float("nan"), 0.0, 3e38
    w, _, _ = weights(g, D, "bf16")
    cs = rotation(g, T, D // 2)
    y, _ = crm.qk_rmsnorm_rope_fwd(q, None, w, None, cs)
    ref, _ = crm.qk_rmsnorm_rope_fwd(clean, None, w, None, cs)
    touched = torch.zeros(T, H, dtype=torch.bool, device=DEV)
    touched[1, 1] = touched[2, 0] = touched[3, 2] = touched[4, 1] = True
    assert torch.equal(y[~touched], ref[~touched])
    assert (y[3, 2] == 0).all() and y[1, 1, 5].isnan() and y[2, 0].isnan().all()
    assert (y[1, 1][torch.arange(D) > D // 2] == 0).all()          # x * rstd with rstd = 0
    assert (y[4, 1] == 0).all()                                    # the squares overflow FP32: rstd = 0
    r, _ = crm.qk_rmsnorm_rope_fwd(q, None, None, None, cs)
    base, _ = crm.qk_rmsnorm_rope_fwd(clean, None, None, None, cs)
    same = torch.ones(T, H, D, dtype=torch.bool, device=DEV)
    same[1, 1, [5, 5 + D // 4]] = same[3, 2] = same[4, 1] = False
    same[2, 0, 40] = False                                         # not rotated: alone
    assert torch.equal(r[same], base[same]) and r[1, 1, 5].isinf() and r[1, 1, 5 + D // 4].isinf()
    # The unrotated part takes nothing from the cosines and sines.
    bad = torch.full_like(cs, float("nan"))
    r, _ = crm.qk_rmsnorm_rope_fwd(clean, None, None, None, bad)
    assert torch.equal(r[..., D // 2:], clean[..., D // 2:]) and r[..., :D // 2].isnan().all()


# ------------------------------------------------------------------ cache --

def caches(g, pages, page, Hk, D, dtype, order):
    """(k view, v view, storage): the views are [pages, page, Hk, D]."""
    if order == "token":
        s = torch.randn(2, pages, page, Hk, D, generator=g).to(dtype).to(DEV)
        return s[0], s[1], s
    if order == "head":
        s = torch.randn(2, pages, Hk, page, D, generator=g).to(dtype).to(DEV)
        return s[0].transpose(1, 2), s[1].transpose(1, 2), s
    if order == "both":          # keys and values of a page in one buffer
        s = torch.randn(pages, 2, page, Hk, D, generator=g).to(dtype).to(DEV)
        return s[:, 0], s[:, 1], s
    s = torch.randn(pages, page, Hk, 2, D + 2, generator=g).to(dtype).to(DEV)      # "mixed": odd strides
    return s[:, :, :, 0, :D], s[:, :, :, 1, 2:], s


@pytest.mark.parametrize("dtype", [BF16, E4M3, E5M2])
@pytest.mark.parametrize("T,Hq,Hk,D,R,pairs,weight,page,order,idx", [
    (1, 32, 8, 128, 128, False, "bf16", 16, "token", torch.int64),
    (37, 8, 2, 128, 128, False, "bf16", 16, "head", torch.int32),
    (100, 3, 1, 64, 32, True, "f32", 1, "token", torch.int64),
    (65, 6, 6, 80, 32, False, None, 24, "both", torch.int64),
    (700, 16, 4, 64, 64, False, "bf16", 7, "both", torch.int32),
    (29, 3, 2, 256, 256, True, "bf16", 64, "mixed", torch.int64),
    (31, 3, 3, 50, 20, False, "bias", 5, "token", torch.int64),
    (23, 0, 2, 128, 128, False, "bf16", 16, "token", torch.int64),
    (90, 4, 2, 72, 72, False, "f32", 16, "token", torch.int64),
    (90, 4, 2, 100, 60, True, "bf16", 16, "head", torch.int32),
    (41, 2, 1, 40, 40, True, None, 3, "both", torch.int64),
])
def test_append(T, Hq, Hk, D, R, pairs, weight, page, order, idx, dtype):
    g = gen(3 * T + D)
    layout = "packed" if order == "token" else "plain"
    q, qc = heads(g, T, Hq, D, layout) if Hq else (None, None)
    (k, kc), (v, vc) = heads(g, T, Hk, D, layout), heads(g, T, Hk, D, layout, 3.0)
    wq, wk, bias = weights(g, D, weight)
    cs = rotation(g, T, R)
    pages = -(-T // page) + 3
    ck, cv, storage = caches(g, pages, page, Hk, D, dtype, order)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[::5] = -1                                  # padding
    if T > 20:
        slots[7], slots[8], slots[9] = pages * page, pages * page + 5, -7
        if idx == torch.int64:
            slots[11] = 1 << 40
    scales = dict(k_scale=torch.tensor([0.03], device=DEV), v_scale=torch.tensor([0.07], device=DEV)) if dtype != BF16 else {}
    before = storage.clone().view(torch.uint8).cpu()
    y = crm.qk_rmsnorm_rope_append(q, k, v, wq if Hq else None, wk, cs, ck, cv, slots.to(idx).to(DEV), 1e-6, bias, pairs, **scales)
    if Hq:
        qk_ref.check(y, *qk_ref.forward(qc, cpu(wq), cpu(cs), 1e-6, bias, pairs), what="q_out")
    ok = (slots >= 0) & (slots < pages * page)
    at = slots[ok]
    sk, sv = (float(scales[n]) if scales else None for n in ("k_scale", "v_scale"))
    rk, bk = qk_ref.forward(kc, cpu(wk), cpu(cs), 1e-6, bias, pairs)
    raw = torch.int16 if dtype == BF16 else torch.uint8          # FP8 tensors take no index
    got_k, got_v = (c.view(raw).cpu()[at // page, at % page].view(dtype) for c in (ck, cv))
    qk_ref.check(got_k, rk[ok], bk[ok], scale=sk, what="k_cache")
    qk_ref.check(got_v, vc[ok].double(), torch.zeros(1, dtype=torch.float64), scale=sv, what="v_cache")
    if dtype == BF16:
        assert torch.equal(got_v, vc[ok])            # values are copied
    # Everything but the named slots is as it was.
    for c in (ck, cv):
        rest = storage.view(raw).as_strided(c.shape, c.stride(), c.storage_offset())
        old = before.view(raw).view(storage.shape).as_strided(c.shape, c.stride(), c.storage_offset())
        rest[(at // page).to(DEV), (at % page).to(DEV)] = old[at // page, at % page].to(DEV)
    assert torch.equal(storage.view(torch.uint8).cpu(), before)


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
def test_append_saturates(dtype):
    T, H, D = 4, 2, 64
    v = torch.zeros(T, H, D, dtype=BF16, device=DEV)
    v[0], v[1, 0], v[1, 1], v[2] = 3e38, float("inf"), -float("inf"), float("nan")
    k = v.clone()
    kc, vc = (torch.zeros(T, 1, H, D, device=DEV).to(dtype) for _ in range(2))
    one = torch.ones(1, device=DEV)
    crm.qk_rmsnorm_rope_append(None, k, v, None, None, None, kc, vc, torch.arange(T, device=DEV), k_scale=one * 0.01, v_scale=one)
    top = qk_ref.TOP[dtype]
    for c in (kc.float()[:, 0], vc.float()[:, 0]):
        assert (c[0] == top).all() and (c[1, 0] == top).all() and (c[1, 1] == -top).all() and c[2].isnan().all() and (c[3] == 0).all()


@pytest.mark.parametrize("dtype", [E4M3, E5M2])
@pytest.mark.parametrize("scale", [2.0 ** -149, 3 * 2.0 ** -140, 2.0 ** -129, 2.0 ** -128, 2.0 ** -126 - 2.0 ** -149, 2.0 ** -126, 1e-30, 1e30])
@pytest.mark.parametrize("D,layout", [(64, "plain"), (100, "plain"), (64, "off4"), (64, "odd")])
def test_append_scales_of_any_size(D, layout, scale, dtype):
    # Values that are zero, subnormal, next to the scale, and large.  The
    # reciprocal of a scale up to 2^-128 is taken as the largest FP32 value.
    g = gen(22)
    T, H = 6, 2
    v, vc = heads(g, T, H, D, layout)
    vc[0], vc[1] = 0.0, vc[1] * 2.0 ** -127
    vc[2] = (vc[2].double() * 16 * scale).to(BF16)
    vc[3] = (vc[3].double() * 300 * scale).to(BF16)
    vc[4, 0, 0], vc[4, 0, 1], vc[4, 0, 2], vc[4, 1] = 2.0 ** -133, -0.0, 3e38, vc[4, 1] * 2.0 ** 100
    v.copy_(vc)
    kc, vcache = (torch.zeros(T, 1, H, D, device=DEV).to(dtype) for _ in range(2))
    s = torch.tensor([scale], dtype=torch.float32)
    assert float(s) == pytest.approx(scale, rel=2.0 ** -24)
    crm.qk_rmsnorm_rope_append(None, v.clone() if layout == "plain" else heads(g, T, H, D, layout)[0].copy_(vc), v, None, None, None,
                               kc, vcache, torch.arange(T, device=DEV), k_scale=s.to(DEV), v_scale=s.to(DEV))
    zero = torch.zeros(1, dtype=torch.float64)
    for c in (kc, vcache):
        got = c.view(torch.uint8)[:, 0].contiguous().view(dtype)
        qk_ref.check(got, vc.double(), zero, scale=max(float(s), 1 / torch.finfo(torch.float32).max))
        assert (got.cpu().float()[0] == 0).all()


def test_append_far_slots():
    # A cache of more than 2^32 elements: the last pages' offsets pass 32 bits.
    g = gen(9)
    T, H, D, page = 6, 8, 128, 16
    pages = (1 << 32) // (page * H * D) + 40
    kc = torch.empty(pages, page, H, D, dtype=torch.uint8, device=DEV).view(E4M3)
    vc = torch.empty(pages, H, page, D, dtype=torch.uint8, device=DEV).view(E4M3).transpose(1, 2)
    k, kcpu = heads(g, T, H, D)
    v, vcpu = heads(g, T, H, D)
    n = pages * page
    slots = torch.tensor([0, n // 2 + 3, n - 1, n - page, 17, n])
    one = torch.full((1,), 0.05, device=DEV)
    kc.view(torch.uint8)[0].zero_(), vc.view(torch.uint8)[0].zero_()
    crm.qk_rmsnorm_rope_append(None, k, v, None, None, None, kc, vc, slots.to(DEV), k_scale=one, v_scale=one)
    zero = torch.zeros(1, dtype=torch.float64)
    for t in range(5):
        s = int(slots[t])
        for c, x in ((kc, kcpu), (vc, vcpu)):
            qk_ref.check(c.view(torch.uint8)[s // page, s % page].contiguous().view(E4M3), x[t].double(), zero, scale=0.05)
    assert (kc.view(torch.uint8)[0, 1:] == 0).all()


def test_long_tensors_pass_32_bits():
    # Token offsets beyond 2^31 elements: a sparse token stride.
    g = gen(10)
    T, H, D = 5, 2, 64
    ld = (1 << 30) + 8
    buf = torch.empty(ld * (T - 1) + H * D, dtype=BF16, device=DEV)
    q = buf.as_strided((T, H, D), (ld, D, 1))
    x, xc = heads(g, T, H, D)
    q.copy_(x)
    w, _, _ = weights(g, D, "bf16")
    cs = rotation(g, T, D)
    y, _ = crm.qk_rmsnorm_rope_fwd(q, None, w, None, cs)
    qk_ref.check(y, *qk_ref.forward(xc, cpu(w), cpu(cs)))
    dq, _, _, _ = crm.qk_rmsnorm_rope_bwd(x, None, q, None, w, None, cs)
    assert torch.equal(dq, crm.qk_rmsnorm_rope_bwd(x, None, x, None, w, None, cs)[0])


# ------------------------------------------------------- refusals, streams --

def test_refusals():
    g = gen(11)
    q, _ = heads(g, 4, 2, 64)
    w, _, _ = weights(g, 64, "bf16")
    cs = rotation(g, 4, 64)
    c = torch.zeros(4, 2, 2, 64, dtype=BF16, device=DEV)
    slots = torch.arange(4, device=DEV)
    f, b, a = crm.qk_rmsnorm_rope_fwd, crm.qk_rmsnorm_rope_bwd, crm.qk_rmsnorm_rope_append
    with pytest.raises(TypeError):
        f(q.float(), None, w, None, cs)
    with pytest.raises(TypeError):
        f(q, None, w, None, cs.to(BF16))
    with pytest.raises(TypeError):
        f(q, None, w, None, cs.cpu())
    with pytest.raises(TypeError):
        f(q, q, w, w.float(), cs)
    with pytest.raises(ValueError):
        f(q, q, w, None, cs)
    with pytest.raises(ValueError):
        f(q, None, w[:32], None, cs)
    with pytest.raises(ValueError):
        f(q, q[:3], w, w, cs)
    with pytest.raises(CrmsnError):
        f(q, None, w, None, cs[:3])                  # 4 tokens, 3 rows
    with pytest.raises(CrmsnError):
        f(q, None, w, None, torch.zeros(4, 128, device=DEV))      # more columns than D
    with pytest.raises(CrmsnError):
        f(q, q, w, w, cs, q_out=q, k_out=q)          # one output twice
    with pytest.raises(CrmsnError):
        b(q, None, q, None, w, None, cs, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        b(q, None, None, None, w, None, cs)
    with pytest.raises(ValueError):
        b(q, None, q, None, w, None, cs, dwq=torch.zeros(32, device=DEV))
    with pytest.raises(TypeError):
        a(q, q, q, w, w, cs, c, c.to(E4M3), slots)
    with pytest.raises(TypeError):
        a(q, q, q, w, w, cs, c, c.clone(), slots.float())
    with pytest.raises(ValueError):
        a(q, q, q, w, w, cs, c, c.clone(), slots[:3])
    with pytest.raises(ValueError):
        a(q, q, q, w, w, cs, c[:, :, :1], c[:, :, :1], slots)
    with pytest.raises(ValueError):
        a(q, q, q, w, w, cs, c, c.clone(), slots, k_scale=torch.ones(1, device=DEV))
    with pytest.raises(TypeError):
        a(q, q, q, w, w, cs, c.to(E4M3), c.to(E4M3), slots)
    with pytest.raises(CrmsnError):
        a(q, q, q, w, w, cs, c, c, slots)            # one cache for both
    with pytest.raises(CrmsnError):
        crm.rope_cos_sin(slots, torch.rand(8, device=DEV), [7])
    with pytest.raises(TypeError):
        crm.rope_cos_sin(slots.float(), torch.rand(8, device=DEV))
    with pytest.raises(ValueError):
        crm.rope_cos_sin(slots, torch.rand(8, device=DEV), [4, 4])
    with pytest.raises(ValueError):
        ag.qk_rmsnorm_rope(q, None, w, None, cs.clone().requires_grad_())


def test_streams_and_threads():
    # Calls on side streams from several host threads, each with its own
    # tensors and the default workspace, give the bits of a lone call.
    g = gen(12)
    T, Hq, Hk, D = 700, 8, 2, 128
    sets = []
    for _ in range(4):
        q, _ = heads(g, T, Hq, D)
        k, _ = heads(g, T, Hk, D)
        wq, wk, _ = weights(g, D, "bf16")
        cs = rotation(g, T, D)
        sets.append((q, k, q, k, wq, wk, cs))
    want = [crm.qk_rmsnorm_rope_bwd(*s) + crm.qk_rmsnorm_rope_fwd(*s[2:]) for s in sets]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = crm.qk_rmsnorm_rope_bwd(*sets[i]) + crm.qk_rmsnorm_rope_fwd(*sets[i][2:])

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_dependent_calls_back_to_back():
    # Each call reads what the call before it wrote, with nothing between.
    g = gen(13)
    T, H, D = 900, 6, 64
    x, _ = heads(g, T, H, D)
    wq, wk, _ = weights(g, D, "bf16")
    pos = torch.arange(T, device=DEV)
    f = torch.rand(32, device=DEV)

    def chain(sync):
        y, outs = x, []
        for i in range(4):
            cs = crm.rope_cos_sin(pos + i, f)
            sync()
            a, b = crm.qk_rmsnorm_rope_fwd(y, x, wq, wk, cs)
            sync()
            c, d, e, h = crm.qk_rmsnorm_rope_bwd(a, b, y, x, wq, wk, cs)
            sync()
            y = c
            outs += [cs, a, b, c, d, e, h]
        torch.cuda.synchronize()
        return outs

    for a, b in zip(chain(lambda: None), chain(torch.cuda.synchronize)):
        assert torch.equal(a, b)


def test_graph_replays():
    # A decode step and a backward captured once, replayed on new contents.
    g = gen(14)
    T, Hq, Hk, D, page = 16, 8, 2, 128, 16
    (q, _), (k, _), (v, _) = (heads(g, T, h, D) for h in (Hq, Hk, Hk))
    wq, wk, _ = weights(g, D, "bf16")
    f = torch.rand(64, device=DEV)
    pos, slots = torch.zeros(T, dtype=torch.int64, device=DEV), torch.zeros(T, dtype=torch.int64, device=DEV)
    kc, vc = (torch.zeros(8, page, Hk, D, dtype=BF16, device=DEV) for _ in range(2))
    y, dq = torch.empty_like(q), torch.empty_like(q)

    def step():
        cs = crm.rope_cos_sin(pos, f)
        crm.qk_rmsnorm_rope_append(q, k, v, wq, wk, cs, kc, vc, slots, q_out=y)
        return crm.qk_rmsnorm_rope_bwd(q, k, q, k, wq, wk, cs, dq=dq)

    def load(seed):
        h = gen(seed)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=h))
        pos.copy_(torch.randint(9999, (T,), generator=h))
        slots.copy_(torch.randperm(8 * page, generator=h)[:T])
        slots[seed % T:] = -1
        kc.zero_(), vc.zero_()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        load(0)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):                                # two graphs, each with its own workspace
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    for seed in (3, 9, 15):
        load(seed)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, kc, vc, *outs[0], *outs[1])]
        load(seed)
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, kc, vc, *want, *want)))


# --------------------------------------------------------------- autograd --

def plain_autograd(q, k, wq, wk, cs, eps, bias, pairs):
    """The same function in FP64 PyTorch, for its gradients."""
    def one(x, w):
        if w is not None:
            x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (w + bias)
        return qk_ref.turn(x.reshape(-1, *x.shape[-2:]), cs, pairs).view(x.shape)
    return one(q, wq), one(k, wk)


@pytest.mark.parametrize("weight,pairs,layout", [("bf16", False, "batch"), ("f32", True, "batch"), (None, False, "batch"), ("bf16", True, "heads")])
def test_autograd(weight, pairs, layout):
    g = gen(15)
    B, S, Hq, Hk, D, R = 2, 30, 6, 2, 64, 64
    make = lambda H: torch.randn(B, S, H, D, generator=g).to(BF16)
    if layout == "heads":        # [B, H, S, D] storage: copied once
        make = lambda H: torch.randn(B, H, S, D, generator=g).to(BF16).transpose(1, 2)
    qc, kc, gqc, gkc = make(Hq), make(Hk), make(Hq), make(Hk)
    wq, wk, bias = weights(g, D, weight)
    cs = rotation(g, S, R)
    leaves = [t.to(DEV).requires_grad_() for t in (qc, kc)] + ([w.requires_grad_() for w in (wq, wk)] if weight else [])
    yq, yk = crm.qk_rmsnorm_rope(leaves[0], leaves[1], wq, wk, cs, 1e-6, bias, pairs)
    got = torch.autograd.grad((yq, yk), leaves, (gqc.to(DEV), gkc.to(DEV)))
    ref = [t.detach().cpu().double().requires_grad_() for t in leaves]
    zq, zk = plain_autograd(ref[0], ref[1], *(ref[2:] or (None, None)), cs.cpu(), 1e-6, bias, pairs)
    want = torch.autograd.grad((zq, zk), ref, (gqc.double(), gkc.double()))
    for x, gr, w, y, dx in ((qc, gqc, wq, yq, got[0]), (kc, gkc, wk, yk, got[1])):
        flat = lambda t: t.reshape(B * S, -1, D)
        w = None if w is None else w.detach().cpu()
        qk_ref.check(flat(y), *qk_ref.forward(flat(x), w, cs.cpu(), 1e-6, bias, pairs))
        rdx, bdx, _, _ = qk_ref.backward(flat(gr), flat(x), w, cs.cpu(), 1e-6, bias, pairs)
        qk_ref.check(flat(dx), rdx, bdx)
    for a, b in zip(got, want):
        assert a.shape == b.shape
        # Loosely against autograd's own: a BF16 step of the largest value.
        assert (a.cpu().double() - b).abs().max() <= 2.0 ** -7 * b.abs().max()
    for w, a in zip(leaves[2:], got[2:]):
        assert a.dtype == w.dtype


def test_autograd_shared_and_missing_gradients():
    g = gen(16)
    T, H, D = 20, 3, 64
    x = heads(g, T, H, D)[0].requires_grad_()
    w = weights(g, D, "f32")[0].requires_grad_()
    cs = rotation(g, T, D)
    # The same tensor as queries and keys, the same weight for both.
    yq, yk = crm.qk_rmsnorm_rope(x, x, w, w, cs)
    gr = torch.randn(T, H, D, generator=g).to(BF16).to(DEV)
    yq.backward(gr)                                    # no gradient reaches yk
    one = crm.qk_rmsnorm_rope_bwd(gr, None, x.detach(), None, w.detach(), None, cs)
    assert torch.equal(x.grad, one[0]) and torch.equal(w.grad, one[2])
    x.grad = w.grad = None
    yq, yk = crm.qk_rmsnorm_rope(x, x, w, w, cs)
    torch.autograd.backward([yq, yk], [gr, gr])
    assert torch.equal(w.grad, 2 * one[2]) and torch.equal(x.grad, 2 * one[0])
    # An expanded gradient, queries alone, and no second derivative.
    x.grad = w.grad = None
    yq, none = crm.qk_rmsnorm_rope(x, None, w, None, cs)
    assert none is None
    yq.sum().backward()
    ones = crm.qk_rmsnorm_rope_bwd(torch.ones_like(gr), None, x.detach(), None, w.detach(), None, cs)
    assert torch.equal(x.grad, ones[0]) and torch.equal(w.grad, ones[2])
    yq, _ = crm.qk_rmsnorm_rope(x, None, w, None, cs)
    (d,) = torch.autograd.grad(yq, x, gr, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()


def test_autograd_capture():
    # Forward and backward in one graph; with an eager graph of the same leaf
    # alive from another stream the capture is refused before anything waits.
    g = gen(17)
    T, H, D = 64, 4, 64
    x, _ = heads(g, T, H, D)
    w = weights(g, D, "f32")[0].requires_grad_()
    cs, gr = rotation(g, T, D), heads(g, T, H, D)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            y, _ = crm.qk_rmsnorm_rope(x, None, w, None, cs)
            y.backward(gr)
            want, w.grad = w.grad, None
            del y
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = crm.qk_rmsnorm_rope(x, None, w, None, cs)
        y.backward(gr)
    w.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w.grad, want)
    eager, _ = crm.qk_rmsnorm_rope(x, None, w, None, cs)
    refused = torch.cuda.CUDAGraph()
    with torch.cuda.graph(refused):
        z = x + 1
        with pytest.raises(RuntimeError, match="recorded outside"):
            crm.qk_rmsnorm_rope(z, None, w, None, cs)
    torch.cuda.synchronize()
    assert eager.grad_fn is not None
    # Nothing is refused where no gradient is recorded.
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph), torch.no_grad():
        z, _ = crm.qk_rmsnorm_rope(x, None, w, None, cs)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, eager)


# ------------------------------------------------------------- run together --

def attention(q, k, v, mask):
    """Plain attention [T, Hq, D] over [S, Hk, D] in FP64, grouped heads."""
    n = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(n, 1), v.repeat_interleave(n, 1)
    a = torch.einsum("thd,shd->hts", q, k) / q.shape[-1] ** 0.5
    return torch.einsum("hts,shd->thd", a.masked_fill(~mask, float("-inf")).softmax(-1), v)


def test_prompt_then_single_tokens():
    # A prompt and then single tokens, appended to shuffled pages: attention
    # over what the pages hold equals attention over the whole sequence.
    g = gen(18)
    P, N, Hq, Hk, D, page = 45, 12, 8, 2, 64, 16
    S = P + N
    hidden, wn = heads(g, S, 1, 256)[0].view(S, 256), (1 + 0.1 * torch.randn(256, generator=g)).to(BF16).to(DEV)
    proj = (torch.randn(256, (Hq + 2 * Hk) * D, generator=g) / 16).to(BF16).to(DEV)
    wq, wk, _ = weights(g, D, "bf16")
    f = (1e4 ** (-torch.arange(D // 2) / (D // 2))).to(DEV)
    pages = 6
    kc, vc = (torch.full((pages, page, Hk, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    order = torch.randperm(pages, generator=g)
    pos = torch.arange(S)
    slots = (order[pos // page] * page + pos % page).to(DEV)
    outs, rows = [], []
    for lo, hi in [(0, P)] + [(t, t + 1) for t in range(P, S)]:
        y, _, _ = crm.rmsnorm_fwd(hidden[lo:hi], wn)
        qkv = (y @ proj).view(hi - lo, Hq + 2 * Hk, D)
        cs = crm.rope_cos_sin(torch.arange(lo, hi, device=DEV), f)
        q = crm.qk_rmsnorm_rope_append(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], wq, wk, cs, kc, vc, slots[lo:hi])
        k, v = (c.view(-1, Hk, D)[slots[:hi]].double().cpu() for c in (kc, vc))
        mask = torch.arange(hi)[None] <= torch.arange(lo, hi)[:, None]
        outs.append(attention(q.double().cpu(), k, v, mask))
        rows.append(qkv.cpu())
    # The same rows in one call: the same bits, so the same attention up to
    # FP64 sums (values below 10, at most 57 terms).
    qkv = torch.cat(rows)
    q, k = crm.qk_rmsnorm_rope_fwd(qkv[:, :Hq].to(DEV), qkv[:, Hq:Hq + Hk].to(DEV), wq, wk, crm.rope_cos_sin(pos.to(DEV), f))
    want = attention(q.double().cpu(), k.double().cpu(), qkv[:, Hq + Hk:].double(), pos[None] <= pos[:, None])
    assert (torch.cat(outs) - want).abs().max() <= 1e-12
    used = torch.zeros(pages * page, dtype=torch.bool)
    used[slots.cpu()] = True
    assert kc.view(-1, Hk, D)[~used.to(DEV)].isnan().all()


def test_training_block():
    # rmsnorm, projection, per-head norms with rotation, attention: the
    # gradients of the block against FP64 autograd.
    g = gen(19)
    S, C, Hq, Hk, D = 24, 128, 4, 2, 32
    x0 = torch.randn(S, C, generator=g).to(BF16)
    params = [(1 + 0.1 * torch.randn(C, generator=g)).to(BF16), (torch.randn(C, (Hq + 2 * Hk) * D, generator=g) / 11).to(BF16),
              (1 + 0.1 * torch.randn(D, generator=g)).to(BF16), (1 + 0.1 * torch.randn(D, generator=g)).to(BF16)]
    gout = torch.randn(S, Hq, D, generator=g)
    f = 1e4 ** (-torch.arange(D // 2) / (D // 2))
    mask = torch.arange(S)[None] <= torch.arange(S)[:, None]

    def block(x, wn, proj, wq, wk, ours):
        if ours:
            y = crm.rmsnorm(x, wn)
            qkv = (y @ proj).view(S, Hq + 2 * Hk, D)
            cs = crm.rope_cos_sin(torch.arange(S, device=DEV), f.to(DEV))
            q, k = crm.qk_rmsnorm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], wq, wk, cs)
        else:
            y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * wn
            qkv = (y @ proj).view(S, Hq + 2 * Hk, D)
            q, k = plain_autograd(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], wq, wk, qk_ref.angles(torch.arange(S)[None], f), 1e-6, 0.0, False)
        return attention(q.double(), k.double(), qkv[:, Hq + Hk:].double(), mask.to(x.device))

    ours = [t.to(DEV).requires_grad_() for t in [x0] + params]
    ref = [t.double().requires_grad_() for t in [x0] + params]
    a = torch.autograd.grad(block(*ours, True), ours, gout.double().to(DEV))
    b = torch.autograd.grad(block(*ref, False), ref, gout.double())
    # Five BF16 roundings on the way forth and as many back, each at most
    # 2^-8 of a value: 10 * 2^-8 of the gradient's size in the 2-norm, with a
    # factor of 2 for sums that cancel.
    for x, y in zip(a, b):
        assert (x.cpu().double() - y).norm() <= 20 * 2.0 ** -8 * y.norm()


# ------------------------------------------------------------ random shapes --

def spaced(g, rng, T, H, D, scale=1.0):
    """Heads somewhere in a larger buffer: random gaps, order and offset, the
    rest of the buffer 9.  Returns the view, its CPU copy and the buffer."""
    step = rng.choice([1, 2, 4, 8, 8, 8])                  # alignment of strides and offset, in elements
    up = lambda n: -(-n // step) * step
    if rng.random() < 0.3:                                 # head-major
        ld = up(D) + step * rng.randint(0, 2)
        hs = up((T - 1) * ld + D) + step * rng.randint(0, 2)
    else:
        hs = up(D) + step * rng.randint(0, 2)
        ld = up((H - 1) * hs + D) + step * rng.randint(0, 2)
    off = step * rng.randint(0, 3)
    size = off + (T - 1) * ld + (H - 1) * hs + D
    buf = torch.full((size + 16,), 9.0, dtype=BF16, device=DEV)
    x = (scale * torch.randn(T, H, D, generator=g)).to(BF16)
    t = buf.as_strided((T, H, D), (ld, hs, 1), off)
    t.copy_(x)
    return t, x, buf


@pytest.mark.parametrize("seed", range(48))
def test_random_shapes(seed):
    import random
    rng, g = random.Random(seed), gen(seed)
    D = rng.choice([64, 128, 256, 2 * rng.randint(1, 256), 4 * rng.randint(1, 64), 8 * rng.randint(1, 64), 16 * rng.randint(1, 32)])
    R = rng.choice([0, D, D, D // 4 * 2, min(D, 2 * rng.randint(1, 128))])
    Hk, pairs = rng.randint(1, 9), rng.random() < 0.5
    Hq = Hk * rng.randint(1, 4)
    P = rng.choice([1, 1, 2, 7, rng.randint(1, 400)])
    T = P * rng.randint(1, max(1, 1500 // P // max(1, Hq * D // 512)) or 1)
    wq, wk, bias = weights(g, D, rng.choice(["bf16", "f32", "bias", None]))
    cs = rotation(g, P if R else 1, R)
    if not R:
        P = 1
    (q, qc, _), (k, kc, _), (v, vc, _) = spaced(g, rng, T, Hq, D), spaced(g, rng, T, Hk, D), spaced(g, rng, T, Hk, D)
    qo, _, qbuf = spaced(g, rng, T, Hq, D)
    before = qbuf.clone()
    yq, yk = crm.qk_rmsnorm_rope_fwd(q, k, wq, wk, cs, 1e-6, bias, pairs, q_out=qo)
    for y, x, w in ((yq, qc, wq), (yk, kc, wk)):
        qk_ref.check(y, *qk_ref.forward(x, cpu(w), cpu(cs), 1e-6, bias, pairs))
    rest = qbuf.clone()                                    # nothing beside the output is written
    rest.as_strided(qo.shape, qo.stride(), qo.storage_offset()).copy_(before.as_strided(qo.shape, qo.stride(), qo.storage_offset()))
    assert torch.equal(rest, before)
    (gq, gqc, _), (gk, gkc, _) = spaced(g, rng, T, Hq, D, 0.1), spaced(g, rng, T, Hk, D, 0.1)
    dq, dk, dwq, dwk = crm.qk_rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, cs, 1e-6, bias, pairs)
    for d, dw, gr, x, w in ((dq, dwq, gqc, qc, wq), (dk, dwk, gkc, kc, wk)):
        rdx, bdx, rdw, bdw = qk_ref.backward(gr, x, cpu(w), cpu(cs), 1e-6, bias, pairs)
        qk_ref.check(d, rdx, bdx, what="dx")
        if w is not None:
            qk_ref.check(dw, rdw, bdw, what="dw")
    page = rng.choice([1, 5, 16, 64])
    pages = -(-T // page) + 2
    kc_, vc_, _ = caches(g, pages, page, Hk, D, BF16, rng.choice(["token", "head", "both", "mixed"]))
    slots = torch.randperm(pages * page, generator=g)[:T].to(DEV)
    z = crm.qk_rmsnorm_rope_append(q, k, v, wq, wk, cs, kc_, vc_, slots, 1e-6, bias, pairs)
    got_k, got_v = (c[slots // page, slots % page] for c in (kc_, vc_))
    qk_ref.check(z, *qk_ref.forward(qc, cpu(wq), cpu(cs), 1e-6, bias, pairs))
    qk_ref.check(got_k, *qk_ref.forward(kc, cpu(wk), cpu(cs), 1e-6, bias, pairs))
    assert torch.equal(got_v.cpu(), vc)


def test_more_than_2_31_elements():
    # 2.3e9 elements a tensor: the last tokens' rows have the bits of a call
    # on those tokens alone.
    T, H, D = 280000, 64, 128
    q = torch.randn(T, H, D, dtype=BF16, device=DEV)
    w = weights(gen(20), D, "bf16")[0]
    cs = crm.rope_cos_sin(torch.arange(T, device=DEV), torch.rand(D // 2, device=DEV))
    y, _ = crm.qk_rmsnorm_rope_fwd(q, None, w, None, cs)
    dq, _, dw, _ = crm.qk_rmsnorm_rope_bwd(y, None, q, None, w, None, cs)
    for lo in (0, T // 2 - 3, T - 7):
        part = slice(lo, lo + 7)
        z, _ = crm.qk_rmsnorm_rope_fwd(q[part], None, w, None, cs[part])
        assert torch.equal(z, y[part])
        assert torch.equal(crm.qk_rmsnorm_rope_bwd(z, None, q[part], None, w, None, cs[part])[0], dq[part])
    # dw against FP64 sums of the same terms, 64 u of the sum of magnitudes
    # (qk_ref); with g = y the turned-back gradient is n up to BF16's rounding
    # of y, so the terms are computed from y itself, a part at a time.
    sums, sizes = torch.zeros(D, dtype=torch.float64, device=DEV), torch.zeros(D, dtype=torch.float64, device=DEV)
    c, s = cs.double().chunk(2, -1)
    for lo in range(0, T, 20000):
        part = slice(lo, lo + 20000)
        a, b = y[part].double().chunk(2, -1)
        cc, ss = c[part, None], s[part, None]
        u = torch.cat([a * cc + b * ss, b * cc - a * ss], -1)
        size = torch.cat([a.abs() * cc.abs() + b.abs() * ss.abs(), b.abs() * cc.abs() + a.abs() * ss.abs()], -1)
        x = q[part].double()
        xhat = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        sums += (u * xhat).sum((0, 1))
        sizes += (size * xhat.abs()).sum((0, 1))
    assert ((dw.double() - sums).abs() <= 2.0 ** -18 * sizes).all()
