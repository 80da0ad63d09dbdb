"""Cases for the attention operators: a whole prompt (packed sequences of
different lengths, grouped heads), and new tokens over a paged key / value
cache (one token of each sequence, drafts to verify, chunks of a prompt).

`run` computes a case with elementary torch operations in FP32 (`own` false)
or with this package's kernels (`own` true); `exact` computes it in FP64 from
the definition."""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
CACHE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------ cases --

def listed():
    prompt = dict(op="prompt", batch=1, ragged=False, hq=32, hk=8, d=128, causal=True, window=0)
    paged = dict(op="paged", batch=1, n=1, lens="same", hq=32, hk=8, d=128, window=0, cache="bf16", page=16, order="token")
    return [
        # One short question: a single small launch, where latency counts.
        dict(prompt, name="prompt short", n=77),
        # One long document.
        dict(prompt, name="prompt long", n=16384),
        # A server's batch of prompts of very different lengths, packed, five query heads to a key head.
        dict(prompt, name="prompt packed", batch=24, n=4099, ragged=True, hq=40, hk=8),
        # Texts to embed: many short ones that see themselves whole, small heads, as many key heads as query heads.
        dict(prompt, name="prompt texts", batch=64, n=500, ragged=True, hq=16, hk=16, d=64, causal=False),
        # A layer of wide heads that looks back over a window only.
        dict(prompt, name="prompt window", n=8192, hq=16, hk=8, d=256, window=1024),
        # One token of one short conversation.
        dict(paged, name="decode one", lens="same", ctx=517),
        # A decode step of a full server, conversations of all lengths.
        dict(paged, name="decode batch", batch=128, lens="ragged", ctx=8192),
        # Two long documents being asked about, FP8 cache with heads before slots.
        dict(paged, name="decode long fp8", batch=2, ctx=131071, cache="e4m3", page=64, order="head"),
        # Four drafted tokens of each conversation to verify.
        dict(paged, name="decode drafts", batch=16, n=4, lens="ragged", ctx=16384, cache="e4m3"),
        # A chunk of a long prompt over what is in the cache already.
        dict(paged, name="chunk long", n=2048, ctx=32768, page=64),
        # A step that carries one prompt's chunk beside the single tokens of others, FP8 cache.
        dict(paged, name="chunk mixed fp8", batch=41, n=1003, lens="mixed", ctx=8192, cache="e4m3"),
        # A small model's chunk: seven query heads to a key head, E5M2.
        dict(paged, name="chunk small", n=777, ctx=5000, hq=14, hk=2, d=64, cache="e5m2", page=64),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    hk = rng.choice([1, 2, 3, 4, 8, 8])
    hq = hk * rng.choice([1, 2, 4, 4, 5, 7, 8])
    window = rng.choice([0, 0, 0, _spread(rng, 64, 4096)])
    c = dict(op=rng.choice(["prompt", "paged"]), hq=hq, hk=hk, d=d, window=window)
    flops = 1 << 39                       # of the scores and their products with the values
    if c["op"] == "prompt":
        batch = rng.choice([1, 1, _spread(rng, 2, 64)])
        c.update(batch=batch, ragged=batch > 1 and rng.random() < 0.8, causal=window > 0 or rng.random() < 0.8,
                 n=_spread(rng, 1, max(2, min(16384, int(math.sqrt(flops / (4 * hq * d * batch)))))))
        return c
    kind = rng.choice(["decode", "decode", "drafts", "chunk", "mixed"])
    batch = 1 if kind == "chunk" else _spread(rng, 1 if kind != "mixed" else 2, 256)
    cache = rng.choice(["bf16", "bf16", "e4m3", "e5m2"])
    room = (1 << 30) // (hk * d * batch)  # keys of a sequence that the cache holds
    n = {"decode": 1, "drafts": rng.randint(2, 8)}.get(kind) or _spread(rng, 9, 4096)
    ctx = _spread(rng, 16, max(32, min(131072, room)))
    n = max(1, min(n, ctx, flops // (4 * hq * d * ctx)))
    c.update(batch=batch, n=n, ctx=ctx, lens="mixed" if kind == "mixed" else "same" if batch == 1 else rng.choice(["same", "ragged"]),
             cache=cache, page=rng.choice([1, 16, 16, 24, 64, 128]), order=rng.choice(["token", "head"]))
    return c


def _lengths(c):
    """[(new tokens, keys)] of the case's sequences."""
    r = random.Random("%d %d %d" % (c["batch"], c["n"], c.get("ctx", 0)))
    if c["op"] == "prompt":
        ns = [c["n"] if i == 0 or not c["ragged"] else _spread(r, 1, c["n"]) for i in range(c["batch"])]
        r.shuffle(ns)
        return [(n, n) for n in ns]
    ns = [c["n"] if i == 0 or c["lens"] != "mixed" else 1 for i in range(c["batch"])]
    r.shuffle(ns)
    return [(n, c["ctx"] if c["lens"] == "same" else r.randint(max(n, c["ctx"] // 8), c["ctx"])) for n in ns]


# ----------------------------------------------------------------- inputs --

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _heads(g, *shape):
    """Queries or keys as their norms leave them: unit rows with weights of their own for each column."""
    return _normal(g, *shape) * (1 + 0.25 * _normal(g, shape[-1]))


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    hq, hk, d, lengths = c["hq"], c["hk"], c["d"], _lengths(case)
    T = sum(n for n, _ in lengths)
    s = dict(case=c, lengths=lengths, starts=None)
    if len({n for n, _ in lengths}) > 1:
        ends = torch.tensor([n for n, _ in lengths]).cumsum(0)
        s["starts"] = torch.cat([torch.zeros(1, dtype=torch.int64), ends]).to(device=DEV, dtype=torch.int32)
    if c["op"] == "prompt":
        # The projection that holds queries, keys and values side by side.
        qkv = torch.cat([_heads(g, T, hq, d), _heads(g, T, hk, d), _normal(g, T, hk, d)], 1).to(BF16)
        if s["starts"] is None and c["batch"] > 1:
            qkv = qkv.view(c["batch"], c["n"], hq + 2 * hk, d)
        s["q"], s["k"], s["v"] = qkv.split([hq, hk, hk], -2)
        return s
    page = c["page"]
    held = [-(-m // page) for _, m in lengths]
    pages = sum(held) + 8
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["batch"], max(held) + 3), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = order[at:at + h]
        at += h
    shape = (pages, page, hk, d) if c["order"] == "token" else (pages, hk, page, d)
    s["k_scale"] = s["v_scale"] = None
    if c["cache"] != "bf16":
        s["k_scale"], s["v_scale"] = torch.tensor([0.05], device=DEV), torch.tensor([0.11], device=DEV)
    for name, scale in (("k_cache", s["k_scale"]), ("v_cache", s["v_scale"])):
        x = _heads(g, *shape) if name == "k_cache" else _normal(g, *shape)
        t = (x if scale is None else x / scale).to(CACHE[c["cache"]])
        s[name] = t if c["order"] == "token" else t.transpose(1, 2)
    s["q"] = _heads(g, T, hq, d).to(BF16)
    s["table"] = table
    s["lens"] = torch.tensor([m for _, m in lengths], dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------- plain form --

def _plain_attention(q, k, v, lens, c):
    """FP32 [B, n, hq, d] of q [B, n, hq, d] over k, v [B, m, hk, d], the last
    query of sequence b standing on key lens[b] - 1."""
    B, n, hq, d = q.shape
    m, hk = k.shape[1:3]
    q = q.to(F32).view(B, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(B, hk, -1, d)
    x = (q @ k.permute(0, 2, 3, 1)).view(B, hq, n, m)
    x *= d ** -0.5
    key, last = torch.arange(m, device=DEV), lens[:, None, None]
    pos = torch.arange(n, device=DEV)[:, None] + last - n
    hidden = (key >= last) if not c.get("causal", True) else (key > pos)
    if c["window"]:
        hidden = hidden | (key <= pos - c["window"])
    x.masked_fill_(hidden[:, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    total = x.sum(-1, keepdim=True).transpose(1, 2)
    o = x.view(B, hk, -1, m) @ v.transpose(1, 2)
    return o.view(B, hq, n, d).transpose(1, 2) / total


def _paged(cache, table, m, page, scale):
    """The first m keys or values of each sequence in FP32 [B, m, hk, d]."""
    at = torch.arange(m, device=DEV)
    x = cache[table[:, at // page].clamp(min=0).long(), at % page].to(F32)
    return x if scale is None else x * scale


def _plain(s):
    c, lengths, q = s["case"], s["lengths"], s["q"]

    def attend(q, b, m):
        """q [B, n, hq, d] of the sequences b, with at most m keys."""
        if c["op"] == "prompt":
            return _plain_attention(q, s["k"][b].to(F32).view(*q.shape[:2], c["hk"], c["d"]), s["v"][b].to(F32).view(*q.shape[:2], c["hk"], c["d"]),
                                    torch.full(q.shape[:1], m, device=DEV), c)
        k, v = (_paged(s[name], s["table"][b], m, c["page"], s[scale]) for name, scale in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
        return _plain_attention(q, k, v, s["lens"][b], c)

    most = max(m for _, m in lengths)
    if s["starts"] is None:
        return attend(q.reshape(len(lengths), -1, c["hq"], c["d"]), slice(None), most).to(BF16).reshape(q.shape)
    ends = [sum(n for n, _ in lengths[:i]) for i in range(len(lengths) + 1)]
    whole = c["op"] == "prompt"
    return torch.cat([attend(q[ends[i]:ends[i + 1]][None], slice(ends[i], ends[i + 1]) if whole else slice(i, i + 1), m)[0].to(BF16)
                      for i, (_, m) in enumerate(lengths)])


def run(state):
    s, c = state, state["case"]
    if own:
        import normalization_rmsnorm_fwd_gb300 as crm

        if c["op"] == "prompt":
            return crm.prompt_attention(s["q"], s["k"], s["v"], starts=s["starts"], causal=c["causal"], window=c["window"])
        return crm.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], starts=s["starts"], window=c["window"],
                                   k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _plain(s)


def _seen(n, m, c):
    """(pairs of a query and a key that it sees, keys that some query sees) of one sequence."""
    if not c.get("causal", True):
        return n * m, m
    w = c["window"] or m
    first = m - n + 1                     # keys that the first query sees, the window aside
    full = max(0, min(n, w - first + 1))  # queries whose window does not cut
    return full * first + full * (full - 1) // 2 + (n - full) * w, min(m, n - 1 + w)


def work(case):
    c = case
    seen = [_seen(n, m, c) for n, m in _lengths(c)]
    T = sum(n for n, _ in _lengths(c))
    cell = 2 if c["op"] == "prompt" or c["cache"] == "bf16" else 1
    keys = sum(k for _, k in seen)
    index = 0 if c["op"] == "prompt" else 4 * sum(-(-k // c["page"]) for _, k in seen) + 4 * c["batch"]
    return {"bytes": 4 * T * c["hq"] * c["d"] + 2 * keys * c["hk"] * c["d"] * cell + index,
            "flops": 4 * c["hq"] * c["d"] * sum(p for p, _ in seen)}


# ------------------------------------------------------------------ exact --
# The definition in FP64: one sequence, one key head and a block of queries at
# a time, over the keys that the block may see.

def exact(case, seed):
    c = case
    if work(c)["flops"] > 3e12:
        return None
    s = prepare(c, seed)
    hq, hk, d = c["hq"], c["hk"], c["d"]
    q = s["q"].reshape(-1, hq, d)
    out = torch.empty(q.shape, dtype=F64, device=DEV)
    first = 0
    for i, (n, m) in enumerate(s["lengths"]):
        if c["op"] == "prompt":
            k, v = (s[name].reshape(-1, hk, d)[first:first + n] for name in ("k", "v"))
        else:
            slots = torch.arange(m, device=DEV)
            pages = s["table"][i].long()[slots.div(c["page"], rounding_mode="floor")]
            k, v = (s[name][pages, slots.remainder(c["page"])] for name in ("k_cache", "v_cache"))
        for h in range(hk):
            kh, vh = k[:, h].to(F64), v[:, h].to(F64)
            if s.get("k_scale") is not None:
                kh, vh = kh * s["k_scale"].to(F64), vh * s["v_scale"].to(F64)
            for a in range(0, n, 2048):
                b = min(n, a + 2048)
                hi = m - n + b if c.get("causal", True) else m
                lo = max(0, m - n + a + 1 - c["window"]) if c["window"] else 0
                x = torch.einsum("ngd,kd->gnk", q[first + a:first + b, h * (hq // hk):(h + 1) * (hq // hk)].to(F64), kh[lo:hi]) / math.sqrt(d)
                behind = torch.arange(m - n + a, m - n + b, device=DEV)[:, None] - torch.arange(lo, hi, device=DEV)
                if c.get("causal", True):
                    x = torch.where(behind >= 0, x, -math.inf)
                if c["window"]:
                    x = torch.where(behind < c["window"], x, -math.inf)
                p = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
                out[first + a:first + b, h * (hq // hk):(h + 1) * (hq // hk)] = torch.einsum("gnk,kd->ngd", p, vh[lo:hi])
        first += n
    return out.view(s["q"].shape)
