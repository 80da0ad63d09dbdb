"""The query / key functions in the debug build: every global access inside
the call's tensors, and the bits of the normal build (small and ragged shapes,
both forms, several tasks per warp, every cache layout)."""
import pytest
import torch

import normalization_rmsnorm_fwd_gb300 as crm
from normalization_rmsnorm_fwd_gb300 import _abi, build
from test_gpu_debug_guard import run_both

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dbg():
    return _abi.load(build.build(debug=True))


def inputs(T, Hq, Hk, D, R, kind, off):
    g = torch.Generator().manual_seed(T + D)

    def t(H):
        x = torch.randn(T * H * D + off, generator=g).to(BF16).to(DEV)
        return x[off:].view(T, H, D)

    w = [None, None] if kind is None else [(1 + 0.1 * torch.randn(D, generator=g)).to(DEV).to(kind) for _ in range(2)]
    cs = None
    if R:
        cs = crm.rope_cos_sin(torch.arange(T, device=DEV), torch.rand(R // 2, generator=g).to(DEV))
    return g, t(Hq), t(Hk), t(Hk), *w, cs


SHAPES = [(1, 32, 8, 128, 128, BF16, 0), (5, 3, 1, 64, 32, torch.float32, 0), (900, 20, 8, 128, 128, BF16, 0),
          (33, 5, 2, 80, 80, BF16, 0), (7, 2, 1, 512, 64, BF16, 0), (40, 3, 3, 24, 16, None, 0), (40, 2, 1, 8, 0, BF16, 0),
          (17, 3, 2, 50, 18, BF16, 0), (1200, 3, 2, 128, 128, torch.float32, 1), (9, 2, 2, 2, 2, None, 0),
          (60, 4, 2, 72, 72, BF16, 0), (60, 4, 2, 100, 36, torch.float32, 0), (60, 4, 2, 128, 128, BF16, 2), (30, 2, 1, 88, 88, None, 4)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("pairs", [False, True])
def test_forward_and_backward(dbg, monkeypatch, shape, pairs):
    def case():
        _, q, k, v, wq, wk, cs = inputs(*shape)
        out = crm.qk_rmsnorm_rope_fwd(q, k, wq, wk, cs, interleaved=pairs)
        grads = crm.qk_rmsnorm_rope_bwd(q, v, q, k, wq, wk, cs, interleaved=pairs)
        alone = crm.qk_rmsnorm_rope_bwd(q, None, q, None, wq, None, cs, interleaved=pairs)
        return [t for t in (*out, *grads, *alone, cs) if t is not None]

    run_both(dbg, monkeypatch, case)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, torch.float8_e4m3fn, torch.float8_e5m2])
@pytest.mark.parametrize("order", ["token", "head"])
def test_append(dbg, monkeypatch, shape, dtype, order):
    def case():
        g, q, k, v, wq, wk, cs = inputs(*shape)
        T, Hk, D, page = shape[0], shape[2], shape[3], 8
        pages = -(-T // page) + 1
        size = (2, pages, page, Hk, D) if order == "token" else (2, pages, Hk, page, D)
        cache = torch.randn(size, generator=g).to(dtype).to(DEV)
        kc, vc = (c if order == "token" else c.transpose(1, 2) for c in cache)
        slots = torch.randperm(pages * page, generator=g)[:T]
        slots[::3] = torch.tensor([-1, pages * page, -5])[torch.arange(len(slots[::3])) % 3]
        one = None if dtype == BF16 else torch.full((1,), 0.05, device=DEV)
        y = crm.qk_rmsnorm_rope_append(q, k, v, wq, wk, cs, kc, vc, slots.to(DEV), k_scale=one, v_scale=one)
        return [y, cache]

    run_both(dbg, monkeypatch, case)


@pytest.mark.parametrize("T,R,sections", [(1, 128, None), (777, 2, None), (50, 126, [20, 23, 20]), (4000, 512, [100, 156])])
def test_angles(dbg, monkeypatch, T, R, sections):
    def case():
        g = torch.Generator().manual_seed(T)
        pos = torch.randint(9999, (len(sections or [0]), T), generator=g).to(DEV)
        return [crm.rope_cos_sin(pos if sections else pos[0], torch.rand(R // 2, generator=g).to(DEV), sections)]

    run_both(dbg, monkeypatch, case)
