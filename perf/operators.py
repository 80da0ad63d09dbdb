"""Cases for the query / key operators: rotary angles, per-head RMSNorm with
the rotation (forward and backward), and the append to a paged cache.

`run` computes a case with elementary torch operations in FP32 (`own` false)
or with this package's kernels (`own` true); `exact` computes it in FP64 from
the definition."""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
CACHE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    angles = dict(op="angles", axes=1, sections="", mixed=False, wide=True, far=False)
    heads = dict(period=0, axes=1, pairs=False, weight="bf16", layout="packed")
    paged = dict(cache="bf16", page=16, order="token", padded=False)
    return [
        # The angles of one decode step's 64 sequences, one rotation for every layer.
        dict(angles, name="angles decode", T=64, R=128, far=True),
        # A long prompt of text and video: three axes in blocks of columns.
        dict(angles, name="angles long 3 axes", T=131072, R=128, axes=3, sections="16,24,24", wide=False),
        # A training step's attention input at hidden size 4096 with grouped keys, one packed projection.
        dict(heads, name="train forward", op="forward", T=16384, hq=32, hk=8, d=128, r=128, period=4096),
        # Images and video: as many key heads as query heads at hidden size 5120, adjacent pairs, three axes.
        dict(heads, name="video forward", op="forward", T=32768, hq=40, hk=40, d=128, r=128, axes=3, pairs=True, layout="separate"),
        # A ragged batch of a small model: head size 80, a quarter rotated, FP32 zero-centred weights.
        dict(heads, name="ragged forward", op="forward", T=1001, hq=15, hk=5, d=80, r=32, weight="fp32", layout="separate"),
        # The gradient of the training step's attention input.
        dict(heads, name="train backward", op="backward", T=16384, hq=32, hk=8, d=128, r=128, period=4096),
        # Wide heads beside an output gate (head stride 2 d), partly rotated, FP32 zero-centred weights.
        dict(heads, name="gated backward", op="backward", T=8192, hq=16, hk=2, d=256, r=64, weight="fp32", layout="gated"),
        # Fine-tuning on one short text: few rows, where latency counts.
        dict(heads, name="short backward", op="backward", T=333, hq=16, hk=16, d=64, r=64, pairs=True),
        # One token of one sequence, cache as it is.
        dict(heads, **paged, name="append one token", op="append", T=1, hq=32, hk=8, d=128, r=128),
        # A decode batch padded to a captured graph's size, FP8 cache with heads before slots.
        dict(heads, **dict(paged, cache="e4m3", order="head", padded=True), name="append decode fp8", op="append", T=256, hq=32, hk=8, d=128, r=128),
        # A prompt written into pages of 16.
        dict(heads, **paged, name="append prompt", op="append", T=8192, hq=32, hk=8, d=128, r=128),
        # A ragged chunk without norms: rotation only, E5M2 cache, pages of 64.
        dict(heads, **dict(paged, cache="e5m2", page=64), name="append chunk rotate", op="append", T=4099, hq=14, hk=2, d=64, r=64, weight="none"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["angles", "forward", "forward", "backward", "backward", "append", "append"])
    if op == "angles":
        axes = rng.choice([1, 1, 2, 3])
        half = 4 * rng.randint(4, 32)
        cut = sorted(rng.sample(range(1, half), axes - 1)) if axes > 1 else []
        parts = [b - a for a, b in zip([0] + cut, cut + [half])]
        mixed = axes > 1 and rng.random() < 0.5
        if mixed:  # equal shares for the later axes, so that every column finds its axis
            share = rng.randint(1, half // axes)
            parts = [half - (axes - 1) * share] + [share] * (axes - 1)
        return dict(op="angles", T=_spread(rng, 1, 131072), R=2 * half, axes=axes,
                    sections=",".join(map(str, parts)) if axes > 1 else "", mixed=mixed,
                    wide=rng.random() < 0.5, far=rng.random() < 0.3)
    d = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256, 512, 8 * rng.randint(2, 32)])
    hk = rng.randint(1, 16)
    hq = hk * rng.choice([1, 1, 2, 4, 5, 8])
    r = rng.choice([d, d, d // 2, 16 * max(1, d // 64)]) // 16 * 16 or 16
    c = dict(op=op, hq=hq, hk=hk, d=d, r=min(r, d), period=0, axes=rng.choice([1, 1, 3]), pairs=rng.random() < 0.4,
             weight=rng.choice(["bf16", "bf16", "fp32"]), layout=rng.choice(["packed", "separate", "gated", "heads"]))
    most = max(1, min(32768, (1 << 27) // ((hq + hk) * d)))
    c["T"] = _spread(rng, 1, most)
    if op != "append" and rng.random() < 0.3:
        c["period"] = max(1, c["T"] // rng.choice([1, 2, 4]))
        c["T"] = c["period"] * (c["T"] // c["period"])
    if op == "append":
        c["weight"] = rng.choice(["bf16", "fp32", "none"])
        c.update(cache=rng.choice(["bf16", "e4m3", "e5m2"]), page=rng.choice([1, 16, 24, 64, 128]),
                 order=rng.choice(["token", "head"]), padded=rng.random() < 0.3)
    return c


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activations(g, T, width):
    """Rows of different sizes with a few large channels, as projections give."""
    x = _normal(g, T, width) * torch.exp(0.5 * _normal(g, T, 1))
    big = torch.randint(width, (max(1, width // 64),), generator=g, device=DEV)
    x[:, big] *= 8.0
    return x.to(BF16)


def _heads(g, c):
    """q [T, hq, d], k and v [T, hk, d] in the case's layout."""
    T, hq, hk, d = c["T"], c["hq"], c["hk"], c["d"]
    if c["layout"] == "packed":
        qkv = _activations(g, T, (hq + 2 * hk) * d).view(T, hq + 2 * hk, d)
        return qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    k = _activations(g, T, hk * d).view(T, hk, d)
    v = _activations(g, T, hk * d).view(T, hk, d)
    if c["layout"] == "gated":
        return _activations(g, T, hq * 2 * d).view(T, hq, 2 * d)[..., :d], k, v
    q = _activations(g, T, hq * d).view(T, hq, d)
    if c["layout"] == "heads":
        q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    return q, k, v


def _weights(g, c):
    """(wq, wk, bias): BF16 near one, FP32 near zero with a bias of one, or none."""
    if c["weight"] == "none":
        return None, None, 0.0
    if c["weight"] == "fp32":
        return 0.1 * _normal(g, c["d"]), 0.1 * _normal(g, c["d"]), 1.0
    return (1 + 0.1 * _normal(g, c["d"])).to(BF16), (1 + 0.1 * _normal(g, c["d"])).to(BF16), 0.0


def _inv_freq(r, base=1e6):
    return (base ** (-torch.arange(0, r, 2, dtype=F64, device=DEV) / r)).to(F32)


def _positions(g, T, axes, far, wide):
    """Text: consecutive positions, or one far position for each sequence;
    video: frame, row and column of a grid."""
    kind = torch.int64 if wide else torch.int32
    if far:
        p = torch.randint(1 << 20, (axes, T), generator=g, device=DEV)
    else:
        first = torch.randint(1 << 12, (1,), generator=g, device=DEV)
        i = torch.arange(T, device=DEV)
        p = torch.stack([first + (i if a == 0 and axes == 1 else (i // 4096, i // 64 % 64, i % 64)[a % 3]) for a in range(axes)])
    return p[0].to(kind) if axes == 1 else p.to(kind)


def _axis_of(half, sections, mixed):
    """The axis of each of the `half` columns, as a list."""
    if len(sections) <= 1:
        return [0] * half
    if mixed:
        n = len(sections)
        return [j % n if j < n * sections[j % n] else 0 for j in range(half)]
    return [a for a, n in enumerate(sections) for _ in range(n)]


def _sections(text, half):
    return [int(s) for s in text.split(",")] if text else [half]


def _rotation(g, c, rows):
    """FP32 [rows, r]: cosines, then sines, of the case's positions."""
    p = _positions(g, rows, c["axes"], c["op"] == "append" and rows <= 512, True).reshape(c["axes"], rows)
    half = c["r"] // 2
    sections = [half] if c["axes"] == 1 else [half - 2 * (half // 3), half // 3, half // 3]
    at = torch.tensor(_axis_of(half, sections, False), device=DEV)
    a = p.T.to(F64)[:, at] * _inv_freq(c["r"]).to(F64)
    return torch.cat([a.cos(), a.sin()], 1).to(F32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "angles":
        half = c["R"] // 2
        return dict(case=c, positions=_positions(g, c["T"], c["axes"], c["far"], c["wide"]), inv_freq=_inv_freq(c["R"]),
                    sections=_sections(c["sections"], half))
    T, hq, hk, d = c["T"], c["hq"], c["hk"], c["d"]
    q, k, v = _heads(g, c)
    wq, wk, bias = _weights(g, c)
    s = dict(case=c, q=q, k=k, wq=wq, wk=wk, bias=bias, cos_sin=_rotation(g, c, c["period"] or T))
    if c["op"] == "backward":
        s["gq"], s["gk"] = (_normal(g, T, hq, d) * 0.02).to(BF16), (_normal(g, T, hk, d) * 0.02).to(BF16)
    if c["op"] == "append":
        pages = -(-T // c["page"]) + 8
        shape = (pages, c["page"], hk, d) if c["order"] == "token" else (pages, hk, c["page"], d)
        for name in ("k_cache", "v_cache"):
            t = _normal(g, *shape).to(CACHE[c["cache"]])
            s[name] = t if c["order"] == "token" else t.transpose(1, 2)
        s["v"] = v
        s["q_out"] = torch.empty(T, hq, d, dtype=BF16, device=DEV)
        s["k_scale"] = s["v_scale"] = None
        if c["cache"] != "bf16":
            s["k_scale"], s["v_scale"] = torch.tensor([0.05], device=DEV), torch.tensor([0.11], device=DEV)
        if T <= 512:  # decode: each token in its own sequence's last page
            slots = torch.randperm(pages * c["page"], generator=g, device=DEV)[:T]
        else:         # a prompt from inside its first page on, over pages in any order
            order = torch.randperm(pages, generator=g, device=DEV)
            i = torch.arange(T, device=DEV) + c["page"] // 2
            slots = order[i // c["page"]] * c["page"] + i % c["page"]
        if c["padded"]:
            slots[T - T // 8:] = -1
        s["slots"] = slots
    return s


# ------------------------------------------------------------- plain form --

def _plain_angles(s):
    half = s["case"]["R"] // 2
    p = s["positions"].reshape(len(s["sections"]), -1)
    at = torch.tensor(_axis_of(half, s["sections"], s["case"]["mixed"]), device=DEV)
    a = p[at].T.to(F64) * s["inv_freq"].to(F64)
    return torch.cat([a.cos(), a.sin()], 1).to(F32)


def _cos_sin(s, T):
    """Cosines and sines [T, 1, r / 2] of each token."""
    cs = s["cos_sin"]
    cs = cs.repeat(T // cs.shape[0], 1) if cs.shape[0] != T else cs
    return cs[:, None].chunk(2, -1)


def _halves(x, r, pairs):
    return (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])


def _joined(a, b, rest, pairs):
    y = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([y, rest], -1)


def _rotate(x, cos, sin, r, pairs):
    a, b = _halves(x, r, pairs)
    return _joined(a * cos - b * sin, b * cos + a * sin, x[..., r:], pairs)


def _plain_forward(x, w, s):
    c = s["case"]
    cos, sin = _cos_sin(s, c["T"])
    x = x.to(F32)
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (w.to(F32) + s["bias"])
    return _rotate(x, cos, sin, c["r"], c["pairs"])


def _plain_backward(g, x, w, s):
    c = s["case"]
    cos, sin = _cos_sin(s, c["T"])
    g, x, w = _rotate(g.to(F32), cos, -sin, c["r"], c["pairs"]), x.to(F32), w.to(F32) + s["bias"]
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xhat, gw = x * rstd, g * w
    dx = rstd * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
    return dx.to(BF16), (g * xhat).sum((0, 1))


def _plain_append(s):
    c = s["case"]
    kind, top = CACHE[c["cache"]], {"bf16": None, "e4m3": 448.0, "e5m2": 57344.0}[c["cache"]]
    used = (s["slots"] >= 0).nonzero()[:, 0] if c["padded"] else slice(None)
    slots = s["slots"][used]
    for name, x, scale in (("k_cache", _plain_forward(s["k"], s["wk"], s), s["k_scale"]), ("v_cache", s["v"].to(F32), s["v_scale"])):
        if top is not None:
            x = (x / scale).clamp(-top, top)
        s[name][slots // c["page"], slots % c["page"]] = x[used].to(kind)
    return [_plain_forward(s["q"], s["wq"], s).to(BF16), s["k_cache"], s["v_cache"]]


def run(state):
    s, c = state, state["case"]
    if own:
        import normalization_rmsnorm_fwd_gb300 as crm

        if c["op"] == "angles":
            return crm.rope_cos_sin(s["positions"], s["inv_freq"], sections=s["sections"], interleaved_axes=c["mixed"])
        how = dict(eps=EPS, weight_bias=s["bias"], interleaved=c["pairs"])
        if c["op"] == "forward":
            return crm.qk_rmsnorm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], **how)
        if c["op"] == "backward":
            return crm.qk_rmsnorm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], **how)
        crm.qk_rmsnorm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos_sin"], s["k_cache"], s["v_cache"],
                                   s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"], **how)
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    if c["op"] == "angles":
        return _plain_angles(s)
    if c["op"] == "forward":
        return [_plain_forward(s["q"], s["wq"], s).to(BF16), _plain_forward(s["k"], s["wk"], s).to(BF16)]
    if c["op"] == "backward":
        (dq, dwq), (dk, dwk) = _plain_backward(s["gq"], s["q"], s["wq"], s), _plain_backward(s["gk"], s["k"], s["wk"], s)
        return [dq, dk, dwq, dwk]
    return _plain_append(s)


def work(case):
    c = case
    if c["op"] == "angles":
        return {"bytes": c["T"] * (c["axes"] * (8 if c["wide"] else 4) + 4 * c["R"]) + 2 * c["R"], "flops": c["T"] * c["R"]}
    T, d, hq, hk = c["T"], c["d"], c["hq"], c["hk"]
    wbytes = {"bf16": 4, "fp32": 8, "none": 0}[c["weight"]] * d
    turn = 4 * c["r"] * (c["period"] or T)
    if c["op"] == "forward":
        return {"bytes": 4 * T * (hq + hk) * d + turn + wbytes, "flops": 8 * T * (hq + hk) * d}
    if c["op"] == "backward":
        return {"bytes": 6 * T * (hq + hk) * d + turn + wbytes + 8 * d, "flops": 16 * T * (hq + hk) * d}
    kept = T - T // 8 if c["padded"] else T
    cell = 2 if c["cache"] == "bf16" else 1
    return {"bytes": 4 * T * hq * d + kept * 2 * hk * d * (2 + cell) + turn + wbytes + 8 * T, "flops": 8 * T * (hq + hk) * d}


# ------------------------------------------------------------------ exact --
# The definition in FP64, with the rotation as a complex product.

def _exact_turn(x, turn, r, pairs):
    """x [T, h, d] in FP64, each pair times the complex `turn` [T, r / 2]."""
    y = x.clone()
    first = torch.arange(r // 2, device=DEV) * (2 if pairs else 1)
    second = first + (1 if pairs else r // 2)
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_norm(x, w, bias):
    """(x / rms, rms, effective weight) in FP64; w None: (x, 1, 1)."""
    x = x.to(F64)
    if w is None:
        return x, 1.0, 1.0
    rms = (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    return x / rms, rms, w.to(F64) + bias


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "angles":
        p = s["positions"].to(F64).reshape(len(s["sections"]), -1)
        out = torch.empty(c["T"], c["R"], dtype=F64, device=DEV)
        half, n = c["R"] // 2, len(s["sections"])
        left, at = list(s["sections"]), 0
        for j in range(half):
            if c["mixed"]:
                at = j % n if (j % n and left[j % n] > 0) else 0
            while not c["mixed"] and left[at] == 0:
                at += 1
            left[at] -= 1
            z = torch.polar(torch.ones_like(p[at]), p[at] * s["inv_freq"][j].to(F64))
            out[:, j], out[:, half + j] = z.real, z.imag
        return out
    half = c["r"] // 2
    cs = s["cos_sin"].to(F64)
    turn = torch.complex(cs[:, :half], cs[:, half:])[torch.arange(c["T"], device=DEV) % cs.shape[0]]

    def forward(x, w):
        xhat, _, we = _exact_norm(x, w, s["bias"])
        return _exact_turn(xhat * we, turn, c["r"], c["pairs"])

    def backward(g, x, w):
        xhat, rms, we = _exact_norm(x, w, s["bias"])
        u = _exact_turn(g.to(F64), turn.conj(), c["r"], c["pairs"])
        along = (u * we * xhat).mean(-1, keepdim=True)
        return (u * we - xhat * along) / rms, (u * xhat).sum((0, 1))

    if c["op"] == "forward":
        return [forward(s["q"], s["wq"]), forward(s["k"], s["wk"])]
    if c["op"] == "backward":
        (dq, dwq), (dk, dwk) = backward(s["gq"], s["q"], s["wq"]), backward(s["gk"], s["k"], s["wk"])
        return [dq, dk, dwq, dwk]
    top = {"bf16": math.inf, "e4m3": 448.0, "e5m2": 57344.0}[c["cache"]]
    out = [forward(s["q"], s["wq"])]
    t = (s["slots"] >= 0).nonzero()[:, 0]
    page, row = s["slots"][t].div(c["page"], rounding_mode="floor"), s["slots"][t].remainder(c["page"])
    for name, x, scale in (("k_cache", forward(s["k"], s["wk"]), s["k_scale"]), ("v_cache", s["v"].to(F64), s["v_scale"])):
        cache = s[name].to(F64)
        cache[page, row] = (x if scale is None else x / scale.to(F64)).clamp(-top, top)[t]
        # E5M2's own rounding (1/8 of a value) hides any error: its codes are compared with the plain form's alone.
        out.append(None if c["cache"] == "e5m2" else cache)
    return out
