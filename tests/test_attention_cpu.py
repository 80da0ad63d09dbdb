"""The attention functions without a GPU: the C ABI's refusals (fake device
addresses are never dereferenced), the binding's packed structs and refusals,
and the FP64 form that the GPU tests compare with, against sums written out."""
import ctypes
import math
import subprocess

import pytest
import torch

import attn_ref
import normalization_rmsnorm_fwd_gb300 as crm
from normalization_rmsnorm_fwd_gb300 import _abi
from normalization_rmsnorm_fwd_gb300 import build as nbuild
from test_qk_rope_cpu import A, ALIAS, ALIGN, ARG, CUDA, DTYPE, G, NULL, OK, SHAPE, UNSUP, WS, call, fields


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("fake device addresses: only where no GPU could follow them")
    nbuild.build()
    return _abi.load()


SHARED = "l:T l:D l:Hq l:Hk l:B h:q h:o p:lse p:starts f:scale i:causal l:window p:ws l:wsn "


class Prompt(ctypes.Structure):
    _fields_ = fields(SHARED + "h:k h:v")


class Paged(ctypes.Structure):
    _fields_ = fields(SHARED + "p:kc l:kps l:kss l:khs p:vc l:vps l:vss l:vhs l:pages l:page p:table l:ldt l:tp p:lens "
                      "p:ks p:vs i:kind i:zero")


def test_packed_calls_have_the_structs_layout():
    for packed, struct in ((_abi.PROMPT_ATTENTION_CALL, Prompt), (_abi.PAGED_ATTENTION_CALL, Paged)):
        values = [1.5 + i if t is ctypes.c_float else 1 if n == "causal" else 1000 + i for i, (n, t) in enumerate(struct._fields_)]
        assert packed.pack(*values) == bytes(struct(*values))


def test_structs_are_the_headers(tmp_path):
    source = tmp_path / "layout.c"
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "crmsnorm.h"', "int main(void) {"]
    for n, last in (("crmsn_prompt_attention_call", "v.hs"), ("crmsn_paged_attention_call", "reserved")):
        lines.append(f'printf("%zu %zu %zu %zu\\n", sizeof({n}), offsetof({n}, attention.scale), '
                     f"offsetof({n}, attention.workspace_bytes), offsetof({n}, {last}));")
    source.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", nbuild.INCLUDE, "-I", "/usr/local/cuda/include", str(source), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    for line, struct, end in zip(out, (Prompt, Paged), ("hsv", "zero")):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(struct), struct.scale.offset, struct.wsn.offset,
                                                  getattr(struct, end).offset]


BASE = dict(T=6404, D=128, Hq=8, Hk=2, B=4, q=A, ldq=1024, hsq=128, o=A + G, ldo=1024, hso=128, lse=A + 2 * G, starts=A + 3 * G,
            scale=0.1, causal=1, window=0, ws=A + 4 * G, wsn=1 << 29)
PROMPT = dict(BASE, k=A + 5 * G, ldk=256, hsk=128, v=A + 6 * G, ldv=256, hsv=128)
PAGED = dict(BASE, kc=A + 5 * G, kps=4096, kss=256, khs=128, vc=A + 6 * G, vps=4096, vss=256, vhs=128, pages=100, page=16,
             table=A + 7 * G, ldt=100, tp=100, lens=A + 8 * G, ks=None, vs=None, kind=0, zero=0)


def prompt(L, **kw):
    return call(L, "prompt_attention", Prompt, PROMPT, kw)


def paged(L, **kw):
    return call(L, "paged_attention", Paged, PAGED, kw)


@pytest.mark.parametrize("f", [prompt, paged])
def test_shared_refusals(L, f):
    assert f(L) == CUDA                         # valid: without a GPU the launch fails
    assert f(L, T=-1) == SHAPE and f(L, T=1 << 31) == SHAPE and f(L, B=-1) == SHAPE and f(L, B=(1 << 20) + 1) == SHAPE
    assert f(L, Hq=0) == SHAPE and f(L, Hk=0) == SHAPE and f(L, Hq=7) == SHAPE and f(L, Hq=4098, ldq=1 << 20, ldo=1 << 20) == SHAPE
    assert f(L, Hq=129, Hk=1, ldq=1 << 20, ldo=1 << 20) == SHAPE                     # more heads than a tile's rows
    assert f(L, D=0) == SHAPE and f(L, D=127) == UNSUP and f(L, D=514) == UNSUP
    assert f(L, starts=None) == CUDA and f(L, starts=None, B=5) == SHAPE             # shared out evenly, or not
    assert f(L, starts=None, B=0) == SHAPE and f(L, starts=None, B=0, T=0) == OK
    for bad in (0.0, -1.0, math.inf, math.nan):
        assert f(L, scale=bad) == ARG
    assert f(L, window=-1) == ARG and f(L, window=5, causal=0) == ARG and f(L, window=5) == CUDA
    assert f(L, window=1 << 40) == CUDA
    assert f(L, q=None) == NULL and f(L, o=None) == NULL and f(L, ws=None) == NULL and f(L, lse=None) == CUDA
    assert f(L, q=A + 1) == ALIGN and f(L, o=A + G + 1) == ALIGN and f(L, lse=A + 2 * G + 2) == ALIGN and f(L, starts=A + 3 * G + 2) == ALIGN
    assert f(L, ldq=64) == SHAPE and f(L, hsq=64) == SHAPE and f(L, ldo=512) == SHAPE
    assert f(L, wsn=0) == WS
    assert f(L, T=0, q=None, o=None, ws=None) == OK and f(L, B=0) == OK
    assert f(L, o=A, ldo=1024) == ALIAS                                              # not in place
    assert f(L, lse=A + G) == ALIAS and f(L, ws=A + G) == ALIAS and f(L, starts=A + G) == ALIAS and f(L, ws=A) == ALIAS
    assert f(L, D=126) == CUDA and f(L, q=A + 2) == CUDA                             # any layout


def test_short_calls_need_no_workspace(L):
    assert prompt(L, T=640, ws=None, wsn=0) == CUDA and prompt(L, T=641, ws=None) == NULL
    assert prompt(L, T=2560, starts=None, ws=None) == CUDA and prompt(L, T=2564, starts=None, ws=None) == NULL
    assert paged(L, tp=40, ws=None, wsn=0) == CUDA and paged(L, tp=41, ws=None) == NULL
    assert paged(L, tp=40, starts=None, ws=None) == CUDA
    assert prompt(L, T=640, o=A + G, ws=A + G) == CUDA            # not used: not looked at


def test_prompt_refusals(L):
    assert prompt(L, k=None) == NULL and prompt(L, v=None) == NULL and prompt(L, k=A + 5 * G + 1) == ALIGN
    assert prompt(L, ldk=128) == SHAPE and prompt(L, hsv=64) == SHAPE
    assert prompt(L, o=A + 5 * G) == ALIAS and prompt(L, ws=A + 6 * G) == ALIAS
    assert L.prompt_attention(None, None) == NULL and L.paged_attention(None, None) == NULL


def test_paged_refusals(L):
    assert paged(L, kind=3) == DTYPE and paged(L, kind=-1) == DTYPE
    assert paged(L, pages=-1) == SHAPE and paged(L, page=0) == SHAPE and paged(L, pages=1 << 28) == SHAPE and paged(L, tp=1 << 28) == SHAPE
    assert paged(L, tp=-1) == SHAPE and paged(L, ldt=-1) == SHAPE and paged(L, ldt=0) == CUDA       # one table for all
    assert paged(L, lens=None) == NULL and paged(L, table=None) == NULL and paged(L, kc=None) == NULL and paged(L, vc=None) == NULL
    assert paged(L, tp=0, table=None) == CUDA and paged(L, pages=0, kc=None, vc=None) == CUDA
    assert paged(L, lens=A + 8 * G + 2) == ALIGN and paged(L, table=A + 7 * G + 1) == ALIGN and paged(L, kc=A + 5 * G + 1) == ALIGN
    assert paged(L, kss=64) == SHAPE and paged(L, vhs=0) == SHAPE
    assert paged(L, kss=128, khs=16 * 128) == CUDA                                   # heads before slots
    assert paged(L, kind=1) == NULL and paged(L, kind=1, ks=A + 9 * G, vs=A + 9 * G + 4) == CUDA
    assert paged(L, kind=2, ks=A + 9 * G + 2, vs=A + 9 * G + 4) == ALIGN
    assert paged(L, o=A + 5 * G) == ALIAS and paged(L, ws=A + 7 * G) == ALIAS and paged(L, lse=A + 8 * G) == ALIAS


def test_supported_sizes(L):
    assert L.rmsnorm_supports(128, 0, _abi.OP_ATTENTION) == OK and L.rmsnorm_supports(512, 0, _abi.OP_ATTENTION) == OK
    assert L.rmsnorm_supports(127, 0, _abi.OP_ATTENTION) == UNSUP and L.rmsnorm_supports(514, 0, _abi.OP_ATTENTION) == UNSUP
    assert L.rmsnorm_supports(128, 1, _abi.OP_ATTENTION) == DTYPE
    assert L.attention_workspace_bytes(127, 0) == 0 and L.attention_workspace_bytes(128, -1) == 0


def test_no_cpu_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        crm.prompt_attention(x, x, x)
    with pytest.raises(TypeError):
        crm.paged_attention(x, x[None], x[None], torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("n,m", [(1, 1), (3, 3), (2, 7), (5, 3), (3, 0)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 2)])
def test_reference_is_the_sum_written_out(n, m, causal, window):
    g = torch.Generator().manual_seed(n * 10 + m)
    q, k, v = (torch.randn(t, h, 4, generator=g, dtype=torch.float64) for t, h in ((n, 4), (m, 2), (m, 2)))
    out, tol, lse, ltol = attn_ref.sequence(q, k, v, 0.7, causal, window)
    for i in range(n):
        for h in range(4):
            total, o = 0.0, [0.0] * 4
            for j in range(m):
                behind = m - n + i - j
                if causal and (behind < 0 or (window and behind >= window)):
                    continue
                w = math.exp(0.7 * sum(float(q[i, h, d] * k[j, h // 2, d]) for d in range(4)))
                total += w
                o = [a + w * float(v[j, h // 2, d]) for d, a in enumerate(o)]
            want = [a / total for a in o] if total else o
            assert torch.allclose(out[i, h], torch.tensor(want, dtype=torch.float64), atol=1e-12)
            assert math.isclose(float(lse[i, h]), math.log(total), abs_tol=1e-12) if total else lse[i, h] == -math.inf


def test_reference_notices_mistakes():
    # A key more, a key less and a shifted mask pass the bounds' size many times.
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(t, h, 64, generator=g).to(torch.bfloat16) for t, h in ((40, 4), (400, 2), (400, 2)))
    out, tol, lse, ltol = attn_ref.sequence(q, k, v)
    for wrong in (attn_ref.sequence(q, k[1:], v[1:]), attn_ref.sequence(q, k, v, window=398), attn_ref.sequence(q, k, v, causal=False),
                  attn_ref.sequence(q, k, v, scale=0.13)):
        assert ((wrong[0] - out).abs() > tol).any() and ((wrong[2] - lse).abs() > ltol).any()
    with pytest.raises(AssertionError):
        attn_ref.check(out + 2 * tol, out, tol)
