"""The waits inside the tiled attention, in the debug build, which can be told
(CRMSN_DEBUG_WAIT_TRIES) to give them up early."""
import pytest
import torch

import attn_ref
import normalization_rmsnorm_fwd_gb300 as crm
from normalization_rmsnorm_fwd_gb300 import _abi, build
from test_gpu_attention import BF16, DEV, E4M3, E5M2, NAN, cache, gen, heads, normal, starts_of
from test_gpu_attention_edges import int32

pytestmark = pytest.mark.gpu


@pytest.fixture
def dbg(monkeypatch):
    monkeypatch.setattr(_abi, "_lib", _abi.load(build.build(debug=True)))


@pytest.mark.parametrize("dtype", [BF16, E5M2])
def test_rows_worked_out_again_keep_no_wait(dbg, monkeypatch, dtype):
    # More tiles than groups of CTAs, so that CTAs have whole tiles and go on behind them.  2^15 tries are some 6 ms; a warp
    # works 32 rows of 4096 keys out again for 45.
    monkeypatch.setenv("CRMSN_DEBUG_WAIT_TRIES", str(1 << 15))
    g = gen(dtype)
    B, n, m = 200, 128, 4096
    kc, vc, table, ks, vs = cache(g, [m], 64, 1, 64, dtype)
    page, row = int(table[0, (m - 10) // 64]), (m - 10) % 64
    zeroed = vc.clone()
    zeroed[page, row] = 0
    vc[page, row] = NAN
    q = normal(g, n, 2, 64).to(BF16)
    out = crm.paged_attention(q.repeat(B, 1, 1), kc, vc, table.repeat(B, 1), torch.full((B,), m, dtype=torch.int32, device=DEV),
                              k_scale=ks, v_scale=vs).view(B, n, 2, 64)
    seen = n - 10                                # tokens that stand before it
    o, tol, _, _ = attn_ref.paged(q, kc, zeroed, table, [m], [n], ks, vs)
    for b in range(B):
        attn_ref.check(out[b, :seen], o[:seen], tol[:seen])
    assert out[:, seen:].isnan().all()
