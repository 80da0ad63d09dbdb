"""The query / key functions without a GPU: the C ABI's refusals (fake device
addresses are never dereferenced), the binding's layouts and refusals, and the
FP64 forms that the GPU tests compare with, against differences."""
import ctypes
import subprocess

import pytest
import torch

import normalization_rmsnorm_fwd_gb300 as crm
import qk_ref
from normalization_rmsnorm_fwd_gb300 import _abi
from normalization_rmsnorm_fwd_gb300 import autograd as ag
from normalization_rmsnorm_fwd_gb300 import binding as B
from normalization_rmsnorm_fwd_gb300 import build as nbuild

OK, NULL, SHAPE, UNSUP, ALIGN, DTYPE, WS, ALIAS, CUDA, TIMEOUT, ARG, SCRATCH = range(12)
A = 1 << 40
G = 1 << 30            # distance between the fake tensors


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("fake device addresses: only where no GPU could follow them")
    nbuild.build()
    return _abi.load()


def fields(text):
    """ctypes fields of a struct of the header, each with its short name here:
    "p" pointer, "l" int64, "i" int32, "f" float, "h" crmsn_heads."""
    kinds = {"p": [("", ctypes.c_void_p)], "l": [("", ctypes.c_int64)], "i": [("", ctypes.c_int32)], "f": [("", ctypes.c_float)]}
    out = []
    for word in text.split():
        kind, name = word.split(":")
        if kind == "h":
            out += [(name, ctypes.c_void_p), ("ld" + name, ctypes.c_int64), ("hs" + name, ctypes.c_int64)]
        else:
            out += [(name, t) for _, t in kinds[kind]]
    return out


LAYER = "l:T l:D l:Hq l:Hk p:wq p:wk i:wd i:inter f:bias f:eps p:cs l:ldcs l:rows l:R "


class Fwd(ctypes.Structure):
    _fields_ = fields(LAYER + "h:q h:k h:qo h:ko")


class Bwd(ctypes.Structure):
    _fields_ = fields(LAYER + "h:gq h:gk h:q h:k h:dq h:dk p:dwq p:dwk p:ws l:wsn")


class Append(ctypes.Structure):
    _fields_ = fields(LAYER + "h:q h:k h:v h:qo p:kc l:kps l:kss l:khs p:vc l:vps l:vss l:vhs i:kind i:sd l:pages l:page "
                      "p:slots p:ks p:vs")


def call(L, name, struct, defaults, kw):
    for k in kw:
        assert k in defaults, k
    names = {n for n, _ in struct._fields_}
    a = struct(**{k: v for k, v in {**defaults, **kw}.items() if k in names})
    return getattr(L, name)(bytes(a), None)


def test_packed_calls_have_the_structs_layout():
    for packed, struct in ((_abi.ROPE_CALL, Rope), (_abi.QK_FWD_CALL, Fwd), (_abi.QK_BWD_CALL, Bwd), (_abi.QK_APPEND_CALL, Append)):
        values = [1.5 + i if t is ctypes.c_float else 1000 + i for i, (_, t) in enumerate(struct._fields_)]
        assert packed.pack(*values) == bytes(struct(*values))


def test_structs_are_the_headers(tmp_path):
    # Sizes and offsets as a C compiler sees them.
    last = {"layer": "layer.R", "Fwd": "k_out.hs", "Bwd": "workspace_bytes", "Append": "v_scale"}
    rope = 'printf("%zu %zu %zu\\n", sizeof(crmsn_rope_call), offsetof(crmsn_rope_call, inv_freq), offsetof(crmsn_rope_call, ldcs));'
    source = tmp_path / "layout.c"
    names = {"Fwd": "crmsn_qk_fwd_call", "Bwd": "crmsn_qk_bwd_call", "Append": "crmsn_qk_append_call"}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "crmsnorm.h"', "int main(void) {"]
    for k, n in names.items():
        lines.append(f'printf("%zu %zu %zu %zu\\n", sizeof({n}), offsetof({n}, layer.interleaved), '
                     f"offsetof({n}, {last['layer']}), offsetof({n}, {last[k]}));")
    source.write_text("\n".join(lines + [rope, "return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", nbuild.INCLUDE, "-I", "/usr/local/cuda/include", str(source), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    for line, struct, end in zip(out, (Fwd, Bwd, Append), ("hsko", "wsn", "vs")):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(struct), struct.inter.offset, struct.R.offset,
                                                  getattr(struct, end).offset]
    assert [int(x) for x in out[3].split()] == [ctypes.sizeof(Rope), Rope.freq.offset, Rope.ldo.offset]


def test_no_struct(L):
    assert L.qk_rmsnorm_rope_fwd(None, None) == NULL
    assert L.qk_rmsnorm_rope_bwd(None, None) == NULL
    assert L.qk_rmsnorm_rope_append(None, None) == NULL


HEADS = dict(q=A, ldq=1024, hsq=128, Hq=8, k=A + G, ldk=256, hsk=128, Hk=2, wq=A + 2 * G, wk=A + 3 * G, wd=0, bias=0.0,
             eps=1e-6, cs=A + 4 * G, ldcs=128, rows=16, R=128, inter=0, T=16, D=128, qo=A + 5 * G, ldqo=1024, hsqo=128,
             ko=A + 6 * G, ldko=256, hsko=128)


def fwd(L, **kw):
    return call(L, "qk_rmsnorm_rope_fwd", Fwd, HEADS, kw)


def test_fwd_refusals(L):
    assert fwd(L) == CUDA                       # valid: without a GPU the launch fails
    assert fwd(L, T=-1) == SHAPE
    assert fwd(L, T=1 << 31) == SHAPE
    assert fwd(L, Hq=0) == SHAPE
    assert fwd(L, Hk=-1) == SHAPE
    assert fwd(L, Hq=4097, ldq=1 << 20, ldqo=1 << 20) == SHAPE
    assert fwd(L, D=127) == UNSUP and fwd(L, D=514) == UNSUP and fwd(L, D=0) == SHAPE
    assert fwd(L, R=130) == SHAPE and fwd(L, R=63) == SHAPE and fwd(L, R=-2) == SHAPE
    assert fwd(L, wd=2) == DTYPE
    assert fwd(L, eps=-1.0) == ARG and fwd(L, eps=float("nan")) == ARG and fwd(L, bias=float("inf")) == ARG
    assert fwd(L, wq=None, wk=None, eps=-1.0) == CUDA         # no norm: eps is not used
    for n in ("q", "k", "qo", "ko", "cs", "wq", "wk"):
        assert fwd(L, **{n: None}) == NULL, n
    assert fwd(L, k=None, Hk=0, wk=None, ko=None) == CUDA     # queries alone
    assert fwd(L, cs=None, R=0) == CUDA                       # norm alone
    assert fwd(L, rows=5) == SHAPE and fwd(L, rows=0) == SHAPE and fwd(L, rows=4) == CUDA
    assert fwd(L, ldcs=126) == SHAPE and fwd(L, rows=1, ldcs=0) == CUDA
    assert fwd(L, T=0, q=None, k=None, qo=None, ko=None, cs=None) == OK
    assert fwd(L, q=A + 1) == ALIGN and fwd(L, cs=A + 4 * G + 2) == ALIGN and fwd(L, wq=A + 2 * G + 1) == ALIGN
    assert fwd(L, wd=1, wq=A + 2 * G + 2) == ALIGN
    assert fwd(L, q=A + 2) == CUDA and fwd(L, D=126, R=126) == CUDA   # the element-wise form


def test_fwd_strides(L):
    assert fwd(L, hsq=64) == SHAPE and fwd(L, ldq=64) == SHAPE        # heads, tokens overlap
    assert fwd(L, ldq=512) == SHAPE                                   # tokens inside one another
    assert fwd(L, ldq=0) == SHAPE and fwd(L, ldq=-1024) == SHAPE
    assert fwd(L, ldqo=512) == SHAPE
    assert fwd(L, ldq=128, hsq=16 * 128) == CUDA                      # [H, T, D]
    assert fwd(L, ldq=128, hsq=15 * 128) == SHAPE
    assert fwd(L, ldq=2048, hsq=256) == CUDA                          # beside a gate
    assert fwd(L, ldq=(1 << 40) + 8) == SHAPE
    assert fwd(L, T=1, rows=1, ldq=0, ldqo=0, ldk=0, ldko=0) == CUDA  # one token: no token stride


def test_fwd_alias(L):
    assert fwd(L, qo=A) == CUDA and fwd(L, ko=A + G) == CUDA          # in place
    assert fwd(L, qo=A, ldqo=1152) == ALIAS and fwd(L, qo=A + 256) == ALIAS
    assert fwd(L, qo=A + G) == ALIAS and fwd(L, ko=A + 5 * G) == ALIAS
    assert fwd(L, qo=A + 4 * G) == ALIAS and fwd(L, qo=A + 2 * G) == ALIAS
    # q, k and q_out as slices of one packed buffer of 20 heads.
    packed = dict(ldq=20 * 128, ldk=20 * 128, k=A + 8 * 256, ldqo=20 * 128, ldko=20 * 128)
    assert fwd(L, **packed, qo=A + 10 * 256, ko=A + 18 * 256) == CUDA
    assert fwd(L, **packed, qo=A + 9 * 256, ko=A + 18 * 256) == ALIAS
    # Heads that alternate: q, k of [T, H, 2, D].
    mixed = dict(Hk=8, ldq=2048, hsq=256, ldk=2048, hsk=256, k=A + 256)
    assert fwd(L, **mixed, qo=A, ldqo=2048, hsqo=256, ko=A + 256, ldko=2048, hsko=256) == CUDA
    assert fwd(L, **mixed, qo=A + 256, ldqo=2048, hsqo=256, ldko=1024) == ALIAS


def bwd(L, **kw):
    d = dict(HEADS, gq=A + 7 * G, ldgq=1024, hsgq=128, gk=A + 8 * G, ldgk=256, hsgk=128, dq=A + 9 * G, lddq=1024, hsdq=128,
             dk=A + 10 * G, lddk=256, hsdk=128, dwq=A + 11 * G, dwk=A + 12 * G, ws=A + 13 * G, wsn=1 << 24)
    return call(L, "qk_rmsnorm_rope_bwd", Bwd, d, kw)


def test_bwd_refusals(L):
    assert bwd(L) == CUDA
    assert bwd(L, Hq=0) == SHAPE and bwd(L, D=1) == UNSUP
    for n in ("gq", "gk", "q", "k", "dq", "dk", "dwq", "dwk", "ws", "cs"):
        assert bwd(L, **{n: None}) == NULL, n
    # Without weights: the rotation's transpose alone.
    none = dict(wq=None, wk=None, q=None, k=None, dwq=None, dwk=None, ws=None, wsn=0)
    assert bwd(L, **none) == CUDA
    assert bwd(L, gk=None, k=None, Hk=0, dk=None, dwk=None, wk=None) == CUDA
    assert bwd(L, dwq=A + 11 * G + 2) == ALIGN and bwd(L, wsn=0) == WS
    assert bwd(L, dq=A + 7 * G) == CUDA                    # in place over the gradient
    assert bwd(L, dq=A) == ALIAS and bwd(L, dwq=A + 12 * G) == ALIAS and bwd(L, ws=A + 9 * G) == ALIAS
    assert L.qk_rmsnorm_rope_bwd_workspace_bytes(127, 0) == 0
    assert L.qk_rmsnorm_rope_bwd_workspace_bytes(514, 0) == 0


def append(L, **kw):
    d = dict(HEADS, v=A + 7 * G, ldv=256, hsv=128, kc=A + 8 * G, kps=4096, kss=256, khs=128, vc=A + 9 * G, vps=4096, vss=256,
             vhs=128, kind=0, pages=10, page=16, slots=A + 10 * G, sd=1, ks=None, vs=None)
    return call(L, "qk_rmsnorm_rope_append", Append, d, kw)


def test_append_refusals(L):
    assert append(L) == CUDA
    assert append(L, q=None, Hq=0, qo=None, wq=None) == CUDA          # the cache alone
    assert append(L, Hk=0) == SHAPE
    for n in ("q", "k", "v", "qo", "kc", "vc", "slots"):
        assert append(L, **{n: None}) == NULL, n
    assert append(L, kind=3) == DTYPE and append(L, sd=2) == DTYPE
    assert append(L, kind=1) == NULL                                  # an FP8 cache needs scales
    fp8 = dict(ks=A + 11 * G, vs=A + 12 * G)
    assert append(L, kind=1, **fp8) == CUDA and append(L, kind=2, **fp8) == CUDA
    assert append(L, kind=1, ks=A + 11 * G + 2, vs=A + 12 * G) == ALIGN
    assert append(L, pages=-1) == SHAPE and append(L, page=0) == SHAPE
    assert append(L, pages=1 << 20, page=1 << 12) == SHAPE            # 2^31 slots and more
    assert append(L, pages=0, kc=None, vc=None) == CUDA               # no page: nothing to write to
    assert append(L, slots=A + 10 * G + 4) == ALIGN and append(L, sd=0, slots=A + 10 * G + 4) == CUDA
    # Overlapping slots, heads or pages.
    assert append(L, kss=128) == SHAPE and append(L, khs=64) == SHAPE and append(L, vps=2048) == SHAPE
    assert append(L, kss=0) == SHAPE
    # Heads before slots; keys and values of one buffer.
    assert append(L, kss=128, khs=16 * 128, vss=128, vhs=16 * 128) == CUDA
    assert append(L, kps=8192, vps=8192, vc=A + 8 * G + 8192) == CUDA
    assert append(L, kps=8192, vps=8192, kss=512, vss=512, vc=A + 8 * G + 512) == CUDA
    assert append(L, vc=A + 8 * G) == ALIAS and append(L, kc=A + 7 * G) == ALIAS and append(L, qo=A + 8 * G) == ALIAS
    assert append(L, T=0, q=None, k=None, v=None, qo=None, slots=None) == OK


class Rope(ctypes.Structure):
    _fields_ = fields("p:pos l:ldp i:pd i:axes i:s0 i:s1 i:s2 i:s3 i:mixed f:scaling p:freq l:T l:R p:out l:ldo")


def rope(L, parts=(), **kw):
    d = dict(pos=A, pd=1, ldp=16, axes=1, mixed=0, freq=A + G, scaling=1.0, T=16, R=128, out=A + 2 * G, ldo=128)
    d.update((f"s{i}", n) for i, n in enumerate((*parts, 0, 0, 0, 0)[:4]))
    return call(L, "rope_cos_sin", Rope, d, kw)


def test_rope_refusals(L):
    assert rope(L) == CUDA and rope(L, parts=[64]) == CUDA and rope(L, parts=[63]) == SHAPE
    assert L.rope_cos_sin(None, None) == NULL
    assert rope(L, R=0) == SHAPE and rope(L, R=127) == SHAPE and rope(L, R=514, ldo=514) == SHAPE
    assert rope(L, axes=0) == SHAPE and rope(L, axes=5) == SHAPE and rope(L, axes=3) == SHAPE
    assert rope(L, axes=3, parts=[16, 24, 24]) == CUDA and rope(L, axes=3, parts=[16, 24, 23]) == SHAPE
    assert rope(L, axes=3, parts=[-8, 48, 24]) == SHAPE and rope(L, axes=3, parts=[0, 40, 24]) == CUDA
    assert rope(L, axes=3, parts=[24, 20, 20], mixed=1) == CUDA
    assert rope(L, axes=3, parts=[16, 24, 24], mixed=1) == SHAPE      # 24 columns of axis 1 do not fit
    assert rope(L, axes=3, parts=[22, 21, 21], mixed=1) == CUDA
    assert rope(L, axes=3, parts=[21, 22, 21], mixed=1) == SHAPE
    assert rope(L, pd=2) == DTYPE and rope(L, scaling=float("inf")) == ARG
    for n in ("pos", "freq", "out"):
        assert rope(L, **{n: None}) == NULL, n
        assert rope(L, **{n: None}, T=0) == OK
    assert rope(L, ldo=126) == SHAPE and rope(L, axes=3, parts=[16, 24, 24], ldp=15) == SHAPE
    assert rope(L, pos=A + 4) == ALIGN and rope(L, pos=A + 4, pd=0) == CUDA and rope(L, out=A + 2 * G + 2) == ALIGN
    assert rope(L, out=A) == ALIAS and rope(L, out=A + G - 8) == ALIAS


def test_supports(L):
    assert L.rmsnorm_supports(128, 0, 8) == OK and L.rmsnorm_supports(512, 1, 8) == OK
    assert L.rmsnorm_supports(514, 0, 8) == UNSUP and L.rmsnorm_supports(127, 0, 8) == UNSUP
    assert L.rmsnorm_supports(0, 0, 8) == SHAPE and L.rmsnorm_supports(128, 2, 8) == DTYPE


def test_head_layouts():
    z = torch.zeros
    assert B.as_heads(z(5, 3, 16)) == (5, 3, 16, 48, 16)
    assert B.as_heads(z(2, 5, 3, 16)) == (10, 3, 16, 48, 16)
    assert B.as_heads(z(5, 9, 16)[:, 3:6]) == (5, 3, 16, 144, 16)            # of a packed projection
    assert B.as_heads(z(5, 3, 32)[..., :16]) == (5, 3, 16, 96, 32)           # beside a gate
    assert B.as_heads(z(3, 5, 16).transpose(0, 1)) == (5, 3, 16, 16, 80)     # [H, T, D]
    assert B.as_heads(z(1, 3, 5, 16).transpose(1, 2)) == (5, 3, 16, 16, 80)
    with pytest.raises(ValueError):
        B.as_heads(z(2, 3, 5, 16).transpose(1, 2))                           # two sequences: no one token stride
    with pytest.raises(ValueError):
        B.as_heads(z(5, 16))
    with pytest.raises(ValueError):
        B.as_heads(z(5, 16, 3).transpose(1, 2))


def test_readable_heads():
    z = torch.zeros
    for t in (z(5, 3, 16), z(5, 9, 16)[:, 3:6], z(3, 5, 16).transpose(0, 1), z(5, 3, 32)[..., 16:]):
        assert ag._readable_heads(t) is t
    for t in (z(1, 1, 1).expand(5, 3, 16), z(1, 3, 16).expand(5, 3, 16), z(5, 1, 16).expand(5, 3, 16),
              z(2, 3, 5, 16).transpose(1, 2), z(5, 16, 3).transpose(1, 2), z(96).as_strided((5, 3, 16), (16, 8, 1))):
        c = ag._readable_heads(t)
        assert c is not t and c.is_contiguous() and torch.equal(c, t)


def test_cpu_tensors_are_refused():
    q, w = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        crm.qk_rmsnorm_rope_fwd(q, q, w, w, None)
    with pytest.raises(TypeError):
        crm.qk_rmsnorm_rope_bwd(q, q, q, q, w, w, None)
    with pytest.raises(TypeError):
        crm.qk_rmsnorm_rope_append(q, q, q, w, w, None, q, q, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(TypeError):
        crm.rope_cos_sin(torch.arange(4), torch.ones(32))


def test_rope_takes_the_same_positions_on_every_axis(L):
    assert rope(L, axes=3, parts=[16, 24, 24], ldp=0) == CUDA
    assert rope(L, axes=3, parts=[16, 24, 24], ldp=-16) == SHAPE and rope(L, axes=3, parts=[16, 24, 24], ldp=1) == SHAPE


def test_calls_run_on_their_tensors_device(monkeypatch):
    # The C call is made with the tensors' device current and on that
    # device's current stream, whichever device is current outside.
    seen, current = [], [0]

    class Lib:
        def rope_cos_sin(self, *args):
            seen.append((current[0], args))
            return 0

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.old, current[0] = current[0], self.dev

        def __exit__(self, *exc):
            current[0] = self.old

    monkeypatch.setattr(B, "_lib", Lib)
    monkeypatch.setattr(B, "_current_device", lambda: current[0])
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(torch.cuda, "device", Device)
    B._enqueue("rope_cos_sin", 0, 7)
    B._enqueue("rope_cos_sin", 3, 7)
    assert seen == [(0, (7, 100)), (3, (7, 103))] and current == [0]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("weight", [True, False])
@pytest.mark.parametrize("R", [0, 6, 10])
def test_reference_gradient_against_differences(pairs, weight, R):
    gen = torch.Generator().manual_seed(R)
    T, H, D, eps, bias = 4, 3, 10, 1e-3, 0.5
    x, g = torch.randn(T, H, D, generator=gen, dtype=torch.float64), torch.randn(T, H, D, generator=gen, dtype=torch.float64)
    w = torch.randn(D, generator=gen, dtype=torch.float64) if weight else None
    cs = qk_ref.angles(torch.arange(2)[None], torch.rand(R // 2, generator=gen)) if R else None
    dx, _, dw, _ = qk_ref.backward(g, x, w, cs, eps, bias, pairs)

    def loss(x, w):
        return float((qk_ref.forward(x, w, cs, eps, bias, pairs)[0] * g).sum())

    # Central differences: error h^2 times third derivatives (below 1e3 here)
    # and rounding 1e-15 / h.
    h = 1e-5
    for t, d, at in ((x, dx, (1, 2, 3)), (x, dx, (3, 0, 9)), (x, dx, (0, 1, 0))) + (((w, dw, (4,)), (w, dw, (9,))) if weight else ()):
        e = torch.zeros_like(t)
        e[at] = h
        up = loss(x + e, w) if t is x else loss(x, w + e)
        down = loss(x - e, w) if t is x else loss(x, w - e)
        assert abs((up - down) / (2 * h) - float(d[at])) < 1e-6


def test_reference_axes():
    assert qk_ref.axis_of(8, [2, 3, 3], False) == [0, 0, 1, 1, 1, 2, 2, 2]
    assert qk_ref.axis_of(8, [4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert qk_ref.axis_of(8, [0, 5, 3], False) == [1] * 5 + [2] * 3


def test_heads_with_dimensions_of_size_one():
    # A dimension of size 1 says nothing about its neighbours, whatever its
    # own stride: single frames with cut-off padding have no one token stride.
    z = torch.zeros
    cut = z(2, 1, 8, 3, 16)[:, :, :5]
    assert cut.stride(0) == cut.stride(1) * cut.size(1)                      # as if contiguous
    for t in (cut, z(2, 1, 8, 3, 16)[:, :, 1:7], z(2, 1, 1, 8, 3, 16)[:, :, :, :5], z(4, 1, 2, 8, 3, 16)[:, :, :, :5]):
        with pytest.raises(ValueError):
            B.as_heads(t)
        c = ag._readable_heads(t)
        assert c is not t and c.is_contiguous() and torch.equal(c, t)
    assert B.as_heads(z(2, 1, 5, 3, 16)) == (10, 3, 16, 48, 16)
    assert B.as_heads(z(2, 5, 1, 3, 16)) == (10, 3, 16, 48, 16)
    assert B.as_heads(z(2, 1, 5, 6, 16)[..., 3:, :]) == (10, 3, 16, 96, 16)
    # One token of each sequence, heads before tokens; the first token of each.
    one = z(4, 3, 1, 16).transpose(1, 2)
    assert B.as_heads(one) == (4, 3, 16, 48, 16) and ag._readable_heads(one) is one
    assert B.as_heads(z(4, 7, 3, 16)[:, :1]) == (4, 3, 16, 7 * 48, 16)
    assert B.as_heads(z(1, 1, 3, 16)) == (1, 3, 16, 48, 16)
    assert B.as_heads(z(0, 7, 3, 16)[:, :5])[:3] == (0, 3, 16)
    assert B.as_heads(z(1, 5, 3, 16).expand(1, 5, 3, 16)) == (5, 3, 16, 48, 16)
    with pytest.raises(ValueError):
        B.as_heads(z(1, 5, 3, 16).expand(2, 5, 3, 16))                       # a repeated sequence
