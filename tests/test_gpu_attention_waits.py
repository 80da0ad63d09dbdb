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


def prompt_case(ns, Hq, Hk, D):
    q, k, v = heads(gen(D, len(ns)), sum(ns), Hq, Hk, D)
    return lambda **how: crm.prompt_attention(q, k, v, starts=starts_of(ns), **how), q.shape


def paged_case(ns, lens, Hq, Hk, D, dtype):
    g = gen(D, dtype)
    kc, vc, table, ks, vs = cache(g, lens, 16, Hk, D, dtype)
    q = normal(g, sum(ns), Hq, D).to(BF16)
    return lambda **how: crm.paged_attention(q, kc, vc, table, int32(*lens), starts=starts_of(ns), k_scale=ks, v_scale=vs, **how), q.shape


CASES = {
    "short": lambda: prompt_case([300, 1, 0, 200, 64], 8, 2, 128),
    "prompt": lambda: prompt_case([1500, 3, 900], 8, 2, 128),
    "many": lambda: prompt_case([60] * 150 + [700] * 12, 4, 4, 64),
    "wide": lambda: prompt_case([1100, 30], 4, 2, 256),
    "chunk": lambda: paged_case([200, 1, 1, 1], [3000, 900, 7, 2000], 8, 2, 128, E4M3),
    "small": lambda: paged_case([500, 40], [1500, 640], 6, 2, 64, E5M2),
}


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("tries", [1, 2, 5, 20, 100, 300, 1000, 4000])
def test_a_wait_that_runs_out_leaves_nan_and_a_status(dbg, monkeypatch, case, tries):
    # Whatever the waits make of it: a row is what it would have been, or NaN with its lse, and NaN is reported, once.
    f, shape = CASES[case]()
    want_lse = torch.full(shape[:2], 3.0, device=DEV)
    want = f(lse=want_lse)
    crm.attention_status()                       # nothing so far
    monkeypatch.setenv("CRMSN_DEBUG_WAIT_TRIES", str(tries))
    ws = torch.full((crm.attention_workspace_bytes(shape[2]) // 4,), 1.0, device=DEV)      # parts that would pass for some
    out, lse = torch.full(shape, 3.0, dtype=BF16, device=DEV), torch.full(shape[:2], 3.0, device=DEV)
    f(out=out, lse=lse, workspace=ws)
    gone = lse.isnan()
    assert torch.equal(out.isnan(), gone[..., None].expand_as(out))
    assert torch.equal(out[~gone], want[~gone]) and torch.equal(lse[~gone], want_lse[~gone])
    if gone.any():
        with pytest.raises(crm.CrmsnError) as e:
            crm.attention_status()
        assert e.value.status == 9
    crm.attention_status()
    if tries == 1:
        assert gone.any()
    monkeypatch.delenv("CRMSN_DEBUG_WAIT_TRIES")
    assert torch.equal(f(), want)
    crm.attention_status()
