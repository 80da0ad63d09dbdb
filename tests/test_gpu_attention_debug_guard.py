"""The attention functions in the debug build: every global access inside the
call's tensors, and the bits of the normal build."""
import pytest
import torch

import normalization_rmsnorm_fwd_gb300 as crm
from normalization_rmsnorm_fwd_gb300 import _abi, build
from test_gpu_attention import BF16, DEV, E4M3, E5M2, cache, gen, heads, normal, starts_of
from test_gpu_debug_guard import run_both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbg():
    return _abi.load(build.build(debug=True))


@pytest.mark.parametrize("D", [64, 72, 100, 128, 192, 256, 512])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("layout", ["packed", "heads", "odd"])
def test_prompt(dbg, monkeypatch, D, G, layout):
    def case():
        q, k, v = heads(gen(D, G), 333, 2 * G, 2, D, layout)
        lse = torch.zeros(333, 2 * G, device=DEV)
        out = torch.zeros(333, 2 * G, D, dtype=BF16, device=DEV)
        crm.prompt_attention(q, k, v, starts=starts_of([3, 0, 200, 129]), lse=lse, out=out)
        return [out, lse, crm.prompt_attention(q, k, v, window=50), crm.prompt_attention(q[:3], k[:3], v[:3]),
                crm.prompt_attention(q, k, v, causal=False)]

    run_both(dbg, monkeypatch, case)


@pytest.mark.parametrize("D", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("dtype", [BF16, E4M3, E5M2])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("page", [1, 16, 100])
def test_paged(dbg, monkeypatch, D, dtype, n, page):
    def case():
        g = gen(D, n)
        lens = [n, 1000, 0, 77, 4001]
        kc, vc, table, ks, vs = cache(g, lens, page, 2, D, dtype, "head" if page == 16 else "token")
        table[1, 3 if page > 1 else 30] = -5
        q = normal(g, 5 * n, 8, D).to(BF16)
        ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
        lse = torch.zeros(5 * n, 8, device=DEV)
        out = crm.paged_attention(q, kc, vc, table, ld, k_scale=ks, v_scale=vs, lse=lse)
        ragged = starts_of([n, 1, 0, 2 * n, 2 * n - 1])
        return [out, lse, crm.paged_attention(q, kc, vc, table, ld, k_scale=ks, v_scale=vs, window=33),
                crm.paged_attention(q, kc, vc, table, ld, k_scale=ks, v_scale=vs, starts=ragged)]

    run_both(dbg, monkeypatch, case)
