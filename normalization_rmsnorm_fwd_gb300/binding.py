"""PyTorch-facing binding of the C ABI: argument marshalling only.

Heads (the query / key functions) are ``[..., heads, D]`` with a contiguous D,
one stride between heads and one between tokens: slices of a packed
projection, heads beside a gate, ``[heads, T, D]`` storage transposed.

Each function has the name of the C entry point it calls, takes CUDA tensors,
turns them into pointers, row counts and row strides, allocates outputs the
caller did not pass (``torch.empty``), and enqueues the call on the current
stream of the tensors' device.  Every step of the computation runs in the
CUDA library; a failing status raises :class:`CrmsnError`.

Row tensors are ``[..., H]`` with a contiguous feature dimension.  Leading
dimensions collapse into rows when each is contiguous with the next in
row-major order (``stride(i) == stride(i+1) * size(i+1)``, dimensions of size 1
aside), so a ``[T, heads, H]`` slice of a wider ``[T, heads, W]`` buffer is
read in place as ``T*heads`` rows of stride ``W``
("cake_rmsnorm_det_train_forward" Parameters/x); any other layout raises
``ValueError``.
"""
from __future__ import annotations

import contextlib
import math

import torch

from . import _abi
from ._abi import BF16, E4M3, E5M2, F32, CrmsnError, check  # noqa: F401

_FP8 = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}


def _lib():
    return _abi.load()


# The raw handle of the current stream without building a Stream object
# (a few microseconds a call); the public query where it is missing.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor) -> int:
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


_SAME_DEVICE = contextlib.nullcontext()


def _on_device(t: torch.Tensor):
    """A context making t's device current; nothing to do when it already is."""
    idx = t.get_device()
    if idx == torch.cuda.current_device():
        return _SAME_DEVICE
    return torch.cuda.device(idx)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_cuda(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")


def _collapsed(shape, st, name, what) -> tuple[int, int]:
    """(count, stride) of the rows that leading dimensions collapse into.  A
    dimension of size 1 has no say, whatever its stride; every other one must
    step over all rows of those inside it."""
    n, ld = 1, st[-1]
    if 0 in shape:
        return 0, ld
    for size, step in zip(reversed(shape), reversed(st)):
        if size == 1:
            continue
        if n == 1:
            ld = step
        elif step != ld * n:
            raise ValueError(f"{name}: leading dimensions must be contiguous with one another "
                             f"(stride(i) == stride(i+1) * size(i+1)) to collapse into {what}")
        n *= size
    return n, ld


def as_rows(t: torch.Tensor, name: str = "x") -> tuple[int, int, int]:
    """(rows, H, row stride in elements) of a row-collapsible tensor."""
    shape = t.shape
    nd = len(shape)
    if nd < 1:
        raise ValueError(f"{name}: needs at least one dimension")
    st = t.stride()
    H = shape[-1]
    if H > 1 and st[-1] != 1:
        raise ValueError(f"{name}: the feature dimension must be contiguous")
    if nd == 1:
        return 1, H, H
    rows, ld = (shape[0], st[0]) if nd == 2 else _collapsed(shape[:-1], st[:-1], name, "rows")
    return rows, H, ld if rows > 1 else max(H, ld)


def _bf16(t, name):
    _need_cuda(t, name)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")


def _weight(w):
    _need_cuda(w, "w")
    if w.dtype == torch.bfloat16:
        kind = BF16
    elif w.dtype == torch.float32:
        kind = F32
    else:
        raise TypeError(f"w must be bfloat16 or float32, got {w.dtype}")
    if w.dim() != 1 or (w.numel() > 1 and w.stride(0) != 1):
        raise ValueError("w must be a contiguous 1-D tensor")
    return kind


def _scale_tensor(scale, device):
    if isinstance(scale, torch.Tensor):
        s = scale.to(device=device, dtype=torch.float32)
        return s.reshape(1).contiguous()
    return torch.tensor([float(scale)], dtype=torch.float32, device=device)


# ---------------------------------------------------------------- forward --

def rmsnorm_fwd(x, w, eps: float = 1e-6, residual=None, weight_bias: float = 0.0,
                y=None, rstd=None, h_new=None, want_rstd: bool = True):
    """y = bf16((h * rstd) * f32(w + weight_bias)) with h = x or
    h_new = bf16(x + residual).  Returns (y, rstd, h_new)."""
    _bf16(x, "x")
    kind = _weight(w)
    T, H, ldx = as_rows(x, "x")
    ldr = 0
    if residual is not None:
        _bf16(residual, "residual")
        if residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        _, _, ldr = as_rows(residual, "residual")
        if h_new is None:
            h_new = torch.empty_like(x, memory_format=torch.contiguous_format)
    if y is None:
        y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    if rstd is None and want_rstd:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _, _, ldy = as_rows(y, "y")
    ldh = as_rows(h_new, "h_new")[2] if h_new is not None else 0
    with _on_device(x):
        st = _lib().rmsnorm_fwd(_ptr(x), ldx, _ptr(residual), ldr, _ptr(w), kind,
                                float(weight_bias), float(eps), T, H, _ptr(y), ldy, _ptr(rstd),
                                _ptr(h_new), ldh, _stream(x))
    check("rmsnorm_fwd", st)
    return y, rstd, h_new


def rmsnorm_quant(out, x, w, scale, eps: float = 1e-6, weight_bias: float = 0.0, rstd=None):
    """out = fp8(RMSNorm(x) * w / scale) (no residual)."""
    return fused_add_rmsnorm_quant(out, x, None, w, scale, eps, weight_bias, rstd)


def fused_add_rmsnorm_quant(out, x, residual, w, scale, eps: float = 1e-6,
                            weight_bias: float = 0.0, rstd=None):
    """residual <- bf16(x + residual) in place (when given); out = fp8 of the
    normalised value divided by the static FP32 scale."""
    _bf16(x, "x")
    _need_cuda(out, "out")
    if out.dtype not in _FP8:
        raise TypeError("out must be float8_e4m3fn or float8_e5m2")
    kind = _weight(w)
    T, H, ldx = as_rows(x, "x")
    ldr = 0
    if residual is not None:
        _bf16(residual, "residual")
        _, _, ldr = as_rows(residual, "residual")
    _, _, ldo = as_rows(out, "out")
    s = _scale_tensor(scale, x.device)
    with _on_device(x):
        st = _lib().fused_add_rmsnorm_quant(_ptr(out), ldo, _FP8[out.dtype], _ptr(x), ldx,
                                            _ptr(residual), ldr, _ptr(w), kind,
                                            float(weight_bias), _ptr(s), float(eps), T, H,
                                            _ptr(rstd), _stream(x))
    check("fused_add_rmsnorm_quant", st)
    return out


def fused_add_rmsnorm_fp8_block_quant(out, block_scale, normed_out, x, residual, w,
                                      eps: float = 1e-6):
    """residual <- bf16(x + residual); normed_out = bf16(RMSNorm * w);
    out / block_scale = its 1x128 E4M3 quantisation, block_scale being
    (H/128, ldT) column-major with ldT = block_scale.shape[1] >= T."""
    for t, n in ((x, "x"), (residual, "residual"), (normed_out, "normed_out")):
        _bf16(t, n)
    _need_cuda(out, "out")
    if out.dtype != torch.float8_e4m3fn:
        raise TypeError("out must be float8_e4m3fn")
    if block_scale.dtype != torch.float32 or not block_scale.is_contiguous():
        raise TypeError("block_scale must be a contiguous float32 tensor")
    if _weight(w) != BF16:
        raise TypeError("w must be bfloat16")
    T, H, ldx = as_rows(x, "x")
    _, _, ldr = as_rows(residual, "residual")
    if not (out.is_contiguous() and normed_out.is_contiguous()):
        raise ValueError("out and normed_out must be contiguous")
    if block_scale.dim() != 2 or block_scale.shape[0] != H // 128:
        raise ValueError("block_scale must be (H/128, ldT)")
    ldT = block_scale.shape[1]
    with _on_device(x):
        st = _lib().fused_add_rmsnorm_fp8_block_quant(_ptr(out), _ptr(block_scale), ldT,
                                                      _ptr(normed_out), _ptr(x), ldx,
                                                      _ptr(residual), ldr, _ptr(w), float(eps),
                                                      T, H, _stream(x))
    check("fused_add_rmsnorm_fp8_block_quant", st)
    return out, block_scale, normed_out


def ada_rms_norm_style(x, w, style, eps: float = 1e-6, out=None, gate_out=None):
    """AdaRMSNorm: bf16(RMSNorm(x, w) * (1 + scale) + shift); gate_out is the
    style's last third.  style is (rows, 3*dim) or (1, 3*dim)."""
    _bf16(x, "x")
    _bf16(style, "style")
    if _weight(w) != BF16:
        raise TypeError("w must be bfloat16")
    if not (x.is_contiguous() and style.is_contiguous()):
        raise ValueError("x and style must be contiguous")
    T, D = x.shape
    if out is None:
        out = torch.empty_like(x)
    if gate_out is None:
        gate_out = torch.empty_like(x)
    with _on_device(x):
        st = _lib().ada_rms_norm_style(_ptr(x), _ptr(w), _ptr(style), style.shape[0],
                                       float(eps), T, D, _ptr(out), _ptr(gate_out), _stream(x))
    check("ada_rms_norm_style", st)
    return out, gate_out


def gate_residual_ada_norm_fp8(residual, x, gate, w, style, scale, eps: float = 1e-6,
                               out=None, gate_out=None):
    """residual <- bf16(residual + bf16(x * gate)); out = e4m3 of the
    AdaRMSNorm of the new residual divided by scale.  Returns
    (residual, out, gate_out)."""
    for t, n in ((residual, "residual"), (x, "x"), (gate, "gate"), (style, "style")):
        _bf16(t, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if _weight(w) != BF16:
        raise TypeError("w must be bfloat16")
    T, D = x.shape
    if out is None:
        out = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=x.device)
    if gate_out is None:
        gate_out = torch.empty_like(x)
    s = _scale_tensor(scale, x.device)
    with _on_device(x):
        st = _lib().gate_residual_ada_norm_fp8(_ptr(residual), _ptr(x), _ptr(gate), _ptr(w),
                                               _ptr(style), style.shape[0], _ptr(s),
                                               float(eps), T, D, _ptr(out), _ptr(gate_out),
                                               _stream(x))
    check("gate_residual_ada_norm_fp8", st)
    return residual, out, gate_out



def fused_rmsnorm_silu(x, w, eps: float = 1e-6, weight_bias: float = 0.0, out=None,
                       scale=None, rstd=None):
    """SiLU(RMSNorm(x) * w_eff): out is BF16 (default, allocated when None) or
    a float8_e4m3fn tensor, which receives e4m3(silu / scale) (scale None:
    no scale).  Returns out."""
    _bf16(x, "x")
    kind = _weight(w)
    T, H, ldx = as_rows(x, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _need_cuda(out, "out")
    if out.dtype == torch.bfloat16:
        fmt = _abi.OUT_BF16
    elif out.dtype == torch.float8_e4m3fn:
        fmt = _abi.OUT_E4M3
    else:
        raise TypeError("out must be bfloat16 or float8_e4m3fn")
    _, _, ldo = as_rows(out, "out")
    s = _scale_tensor(scale, x.device) if (scale is not None and fmt == _abi.OUT_E4M3) else None
    with _on_device(x):
        st = _lib().fused_rmsnorm_silu(_ptr(out), ldo, fmt, _ptr(x), ldx, _ptr(w), kind,
                                       float(weight_bias), _ptr(s), float(eps), T, H,
                                       _ptr(rstd), _stream(x))
    check("fused_rmsnorm_silu", st)
    return out


def _ln_params(x, gamma, beta):
    _bf16(x, "x")
    for t, name in ((gamma, "gamma"), (beta, "beta")):
        _need_cuda(t, name)
        if t.dtype != torch.float32 or t.dim() != 1 or (t.numel() > 1 and t.stride(0) != 1):
            raise TypeError(f"{name} must be a contiguous 1-D float32 tensor")
    return as_rows(x, "x")


def layernorm(x, gamma, beta, eps: float = 1e-5, out=None, mean=None, rstd=None):
    """bf16((x - E[x]) / sqrt(Var[x] + eps) * gamma + beta) with the
    population variance; gamma and beta FP32.  Returns out."""
    T, H, ldx = _ln_params(x, gamma, beta)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _bf16(out, "out")
    _, _, ldo = as_rows(out, "out")
    with _on_device(x):
        st = _lib().layernorm(_ptr(out), ldo, _ptr(x), ldx, _ptr(gamma), _ptr(beta), float(eps),
                              T, H, _ptr(mean), _ptr(rstd), _stream(x))
    check("layernorm", st)
    return out


def layernorm_quant(out, x, gamma, beta, scale, eps: float = 1e-5, mean=None, rstd=None):
    """out = fp8(layernorm(x) / scale) with out float8_e4m3fn or
    float8_e5m2.  Returns out."""
    T, H, ldx = _ln_params(x, gamma, beta)
    _need_cuda(out, "out")
    if out.dtype not in _FP8:
        raise TypeError("out must be float8_e4m3fn or float8_e5m2")
    _, _, ldo = as_rows(out, "out")
    s = _scale_tensor(scale, x.device)
    with _on_device(x):
        st = _lib().layernorm_quant(_ptr(out), ldo, _FP8[out.dtype], _ptr(x), ldx, _ptr(gamma),
                                    _ptr(beta), _ptr(s), float(eps), T, H, _ptr(mean), _ptr(rstd),
                                    _stream(x))
    check("layernorm_quant", st)
    return out

# --------------------------------------------------------------- backward --

def rmsnorm_bwd_workspace_bytes(rows: int, hidden: int, device=None, residual: bool = False) -> int:
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    n = _lib().rmsnorm_bwd_workspace_bytes(int(rows), int(hidden), idx, int(bool(residual)))
    if n == 0:
        raise CrmsnError("rmsnorm_bwd_workspace_bytes", 3, "invalid hidden size or device")
    return n


def rmsnorm_bwd_workspace(rows: int, hidden: int, device=None) -> torch.Tensor:
    """A zero-filled uint8 workspace of rmsnorm_bwd_workspace_bytes() bytes
    (the caching allocator returns 512-byte aligned blocks)."""
    dev = torch.device(device) if device is not None else torch.device("cuda")
    return torch.zeros(rmsnorm_bwd_workspace_bytes(rows, hidden, dev), dtype=torch.uint8,
                       device=dev)


def rmsnorm_bwd(g, x, w, rstd, weight_bias: float = 0.0, g_residual=None, workspace=None,
                dx=None, dw=None):
    """dx = bf16(rstd*g*w_eff - x*rstd^3*mean(g*w_eff*x) (+ g_residual)) and the
    deterministic FP32 dw = sum_t g*x*rstd.  Returns (dx, dw)."""
    _bf16(g, "g")
    _bf16(x, "x")
    kind = _weight(w)
    T, H, ldx = as_rows(x, "x")
    if g.shape != x.shape:
        raise ValueError("g must have x's shape")
    _, _, ldg = as_rows(g, "g")
    ldgr = 0
    if g_residual is not None:
        _bf16(g_residual, "g_residual")
        _, _, ldgr = as_rows(g_residual, "g_residual")
    if rstd.dtype != torch.float32 or not rstd.is_contiguous() or rstd.numel() != T:
        raise ValueError("rstd must be a contiguous float32 tensor with one value per row")
    if dx is None:
        dx = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _, _, lddx = as_rows(dx, "dx")
    if dw is None:
        dw = torch.empty(H, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(rmsnorm_bwd_workspace_bytes(T, H, x.device), dtype=torch.uint8,
                                device=x.device)
    with _on_device(x):
        st = _lib().rmsnorm_bwd(_ptr(g), ldg, _ptr(x), ldx, _ptr(w), kind, float(weight_bias),
                                _ptr(rstd), _ptr(g_residual), ldgr, T, H, _ptr(dx), lddx,
                                _ptr(dw), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(x))
    check("rmsnorm_bwd", st)
    return dx, dw


def rmsnorm_bwd_noalloc(g, x, w, rstd, weight_bias: float = 0.0, g_residual=None, dx=None,
                        dw=None):
    """rmsnorm_bwd for callers that cannot provide a workspace: the library's
    built-in 16 MiB scratch is used instead, shared by every call on the
    device (overlapping calls race).  Returns (dx, dw)."""
    _bf16(g, "g")
    _bf16(x, "x")
    kind = _weight(w)
    T, H, ldx = as_rows(x, "x")
    _, _, ldg = as_rows(g, "g")
    ldgr = 0
    if g_residual is not None:
        _bf16(g_residual, "g_residual")
        _, _, ldgr = as_rows(g_residual, "g_residual")
    if dx is None:
        dx = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    _, _, lddx = as_rows(dx, "dx")
    if dw is None:
        dw = torch.empty(H, dtype=torch.float32, device=x.device)
    with _on_device(x):
        st = _lib().rmsnorm_bwd_noalloc(_ptr(g), ldg, _ptr(x), ldx, _ptr(w), kind,
                                        float(weight_bias), _ptr(rstd), _ptr(g_residual), ldgr, T,
                                        H, _ptr(dx), lddx, _ptr(dw), _stream(x))
    check("rmsnorm_bwd_noalloc", st)
    return dx, dw


# ------------------------------------------------- queries, keys and cache --

_INDEX = {torch.int32: _abi.I32, torch.int64: _abi.I64}
_CACHE = {torch.bfloat16: _abi.CACHE_BF16, torch.float8_e4m3fn: _abi.CACHE_E4M3,
          torch.float8_e5m2: _abi.CACHE_E5M2}


def as_heads(t: torch.Tensor, name: str = "q") -> tuple[int, int, int, int, int]:
    """(tokens, heads, D, token stride, head stride in elements) of a
    [..., heads, D] tensor whose leading dimensions collapse into tokens."""
    shape, st = t.shape, t.stride()
    nd = len(shape)
    if nd < 3:
        raise ValueError(f"{name}: needs [tokens, heads, D]")
    H, D = shape[-2:]
    if D > 1 and st[-1] != 1:
        raise ValueError(f"{name}: D must be contiguous")
    if nd == 3:
        return shape[0], H, D, st[0], st[1]
    T, ld = _collapsed(shape[:-2], st[:-2], name, "tokens")
    return T, H, D, ld, st[-2]


_BF16 = torch.bfloat16
_F32 = torch.float32
# The current device without torch.cuda's checks (a call costs 0.07 instead of
# 0.3 us), where the tensors have shown that CUDA is up.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


_ABSENT = (0, 0, 0)           # a tensor that is not given


def _head_tensor(t, name, dev, shape):
    """(pointer, token stride, head stride) of a BF16 tensor of this shape on
    CUDA device `dev`."""
    if t.dtype is not _BF16 or t.get_device() != dev:
        raise TypeError(f"{name} must be bfloat16 on cuda:{dev}, got {t.dtype} on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if len(shape) == 3:
        ld, hs, one = t.stride()
        if one == 1 or shape[2] <= 1:
            return t.data_ptr(), ld, hs
    return (t.data_ptr(), *as_heads(t, name)[3:])


def _first_head_tensor(t, name):
    """(device, shape, tokens, heads, D) of the tensor that the others of a
    call are measured by."""
    _need_cuda(t, name)
    shape = t.shape
    if len(shape) == 3:
        T, H, D = shape
    else:
        T, H, D = as_heads(t, name)[:3]
    return t.get_device(), shape, T, H, D


def _new_heads(t, H, D):
    """A new contiguous tensor of t's shape and dtype, and what _head_tensor
    says of it."""
    n = torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)
    return n, (n.data_ptr(), H * D, D)


def _kv_shape(shape, t, name):
    """The shape that t must have, `shape` with t's own heads, and those."""
    own = t.shape
    if len(own) != len(shape):
        raise ValueError(f"{name} must have {len(shape)} dimensions")
    H = own[-2]
    if len(own) == 3:
        return (shape[0], H, shape[2]), H
    return (*shape[:-2], H, shape[-1]), H


def _weight_ptr(w, name, D, dev):
    if w.get_device() != dev or w.shape != (D,) or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{D}] tensor on cuda:{dev}")
    return w.data_ptr()


def _head_weights(wq, wk, D, dev, has_q, has_k):
    """(pointers, w_dtype) of the two weights."""
    if wq is None and wk is None:
        return 0, 0, 0
    if (has_q and wq is None) or (has_k and wk is None):
        raise ValueError("wq and wk: both or neither")
    one = wq if has_q else wk
    dtype = one.dtype
    if dtype is not _BF16 and dtype is not _F32:
        raise TypeError(f"wq and wk must be bfloat16 or float32, got {dtype}")
    if has_q and has_k and wk.dtype is not dtype:
        raise TypeError("wq and wk must have the same dtype")
    return (_weight_ptr(wq, "wq", D, dev) if has_q else 0, _weight_ptr(wk, "wk", D, dev) if has_k else 0,
            BF16 if dtype is _BF16 else F32)


def _rotation(cos_sin, dev):
    """(pointer, row stride, rows, R) of the cosines and sines; None: none."""
    if cos_sin is None:
        return 0, 0, 1, 0
    if cos_sin.dtype is not _F32 or cos_sin.get_device() != dev:
        raise TypeError(f"cos_sin must be float32 on cuda:{dev}, got {cos_sin.dtype} on {cos_sin.device}")
    if cos_sin.dim() == 2:
        rows, R = cos_sin.shape
        ld, one = cos_sin.stride()
        if one == 1 or R <= 1:
            return cos_sin.data_ptr(), ld, rows, R
    rows, R, ld = as_rows(cos_sin, "cos_sin")
    return cos_sin.data_ptr(), ld, rows, R


def _enqueue(name, dev, *args):
    """The C call `name`, its last argument being the current stream of `dev`,
    with that device current."""
    fn = getattr(_lib(), name)
    stream = _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    if dev == _current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st:
        check(name, st)


_ALL_COLUMNS = (0, 0, 0, 0)     # of the one axis


def rope_cos_sin(positions, inv_freq, sections=None, interleaved_axes: bool = False,
                 scaling: float = 1.0, out=None):
    """Cosines and sines of rotary positions, FP32 [..., R] (R/2 cosines, then
    R/2 sines) with R = 2 * inv_freq.numel(): positions is [...] (int32 or
    int64), or [axes, ...] (possibly expanded) when `sections` (the columns of each
    axis) names more than one axis.  One call serves every layer.  Returns out."""
    _need_cuda(positions, "positions")
    dev = positions.get_device()
    kind = _INDEX.get(positions.dtype)
    if kind is None:
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    if inv_freq.dtype is not _F32 or inv_freq.get_device() != dev:
        raise TypeError(f"inv_freq must be float32 on cuda:{dev}")
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous 1-D tensor")
    R = 2 * inv_freq.shape[0]
    shape, ldp, axes, parts = positions.shape, 0, 1, _ALL_COLUMNS
    if sections is not None:
        axes = len(sections)
        if not 1 <= axes <= 4:
            raise ValueError("sections must name one to four axes")
        parts = (*sections, 0, 0, 0)[:4]
    if axes > 1:
        if len(shape) < 2 or shape[0] != axes:
            raise ValueError(f"positions must be [{axes}, ...]")
        shape, ldp = shape[1:], positions.stride(0)
        if not positions.is_contiguous() and not positions[0].is_contiguous():
            raise ValueError("positions: each axis must be contiguous")
    elif not positions.is_contiguous():
        raise ValueError("positions must be contiguous")
    whole = (*shape, R)
    if out is None:
        out = torch.empty(whole, dtype=_F32, device=positions.device)
        ldo = R
    else:
        if out.dtype is not _F32 or out.get_device() != dev or out.shape != whole:
            raise TypeError(f"out must be float32 {whole} on cuda:{dev}")
        ldo = as_rows(out, "out")[2]
    T = shape[0] if len(shape) == 1 else math.prod(shape)
    _enqueue("rope_cos_sin", dev,
             _abi.ROPE_CALL.pack(positions.data_ptr(), ldp, kind, axes, *parts, interleaved_axes, scaling,
                                 inv_freq.data_ptr(), T, R, out.data_ptr(), ldo))
    return out


def qk_rmsnorm_rope_fwd(q, k, wq, wk, cos_sin, eps: float = 1e-6, weight_bias: float = 0.0,
                        interleaved: bool = False, q_out=None, k_out=None):
    """Per-head RMSNorm of q [..., Hq, D] (weight wq) and k [..., Hk, D] (wk)
    and the rotation by cos_sin, one rounding to BF16.  k None: queries alone;
    wq = wk = None: no norm; cos_sin None: no rotation.  cos_sin [P, R] serves
    token t with row t % P.  q_out may be q, k_out may be k.  Returns
    (q_out, k_out)."""
    dev, shape, T, Hq, D = _first_head_tensor(q, "q")
    qp = _head_tensor(q, "q", dev, shape)
    if q_out is None:
        q_out, qo = _new_heads(q, Hq, D)
    else:
        qo = _head_tensor(q_out, "q_out", dev, shape)
    Hk, kp, ko = 0, _ABSENT, _ABSENT
    if k is not None:
        kshape, Hk = _kv_shape(shape, k, "k")
        kp = _head_tensor(k, "k", dev, kshape)
        if k_out is None:
            k_out, ko = _new_heads(k, Hk, D)
        else:
            ko = _head_tensor(k_out, "k_out", dev, kshape)
    elif k_out is not None:
        raise ValueError("k_out without k")
    wqp, wkp, kind = _head_weights(wq, wk, D, dev, True, k is not None)
    _enqueue("qk_rmsnorm_rope_fwd", dev,
             _abi.QK_FWD_CALL.pack(T, D, Hq, Hk, wqp, wkp, kind, interleaved, weight_bias, eps, *_rotation(cos_sin, dev),
                                   *qp, *kp, *qo, *ko))
    return q_out, k_out


def qk_rmsnorm_rope_bwd_workspace_bytes(D: int, device=None) -> int:
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    n = _lib().qk_rmsnorm_rope_bwd_workspace_bytes(int(D), idx)
    if n == 0:
        raise CrmsnError("qk_rmsnorm_rope_bwd_workspace_bytes", 3, "invalid head size or device")
    return n


def _dw_tensor(dw, name, D, like):
    if dw is None:
        return torch.empty(D, dtype=_F32, device=like.device)
    if dw.dtype is not _F32 or dw.device != like.device or dw.shape != (D,) or not dw.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 [{D}] tensor on {like.device}")
    return dw


def qk_rmsnorm_rope_bwd(gq, gk, q, k, wq, wk, cos_sin, eps: float = 1e-6, weight_bias: float = 0.0,
                        interleaved: bool = False, dq=None, dk=None, dwq=None, dwk=None, workspace=None):
    """Gradients of qk_rmsnorm_rope_fwd from gq, gk (of its outputs) and its
    inputs q, k: dq, dk (BF16) and the FP32 dwq, dwk, added in a fixed order.
    Without weights q and k may be None and dwq, dwk are None.  Returns
    (dq, dk, dwq, dwk)."""
    dev, shape, T, Hq, D = _first_head_tensor(gq, "gq")
    gqp = _head_tensor(gq, "gq", dev, shape)
    if dq is None:
        dq, dqp = _new_heads(gq, Hq, D)
    else:
        dqp = _head_tensor(dq, "dq", dev, shape)
    Hk, gkp, dkp, qp, kp = 0, _ABSENT, _ABSENT, _ABSENT, _ABSENT
    if gk is not None:
        kshape, Hk = _kv_shape(shape, gk, "gk")
        gkp = _head_tensor(gk, "gk", dev, kshape)
        if dk is None:
            dk, dkp = _new_heads(gk, Hk, D)
        else:
            dkp = _head_tensor(dk, "dk", dev, kshape)
    elif dk is not None or dwk is not None:
        raise ValueError("dk or dwk without gk")
    wqp, wkp, kind = _head_weights(wq, wk, D, dev, True, gk is not None)
    dwqp = dwkp = wsp = wsn = 0
    if wq is not None:
        if q is None or (gk is not None and k is None):
            raise ValueError("q and k are needed with weights")
        qp = _head_tensor(q, "q", dev, shape)
        dwq = _dw_tensor(dwq, "dwq", D, gq)
        dwqp = dwq.data_ptr()
        if gk is not None:
            kp = _head_tensor(k, "k", dev, kshape)
            dwk = _dw_tensor(dwk, "dwk", D, gq)
            dwkp = dwk.data_ptr()
        if workspace is None:
            wsn = _lib().qk_rmsnorm_rope_bwd_workspace_bytes(D, dev)
            workspace = torch.empty(wsn, dtype=torch.uint8, device=gq.device)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on cuda:{dev}")
        else:
            wsn = workspace.numel() * workspace.element_size()
        wsp = workspace.data_ptr()
    elif dwq is not None or dwk is not None:
        raise ValueError("dwq or dwk without weights")
    _enqueue("qk_rmsnorm_rope_bwd", dev,
             _abi.QK_BWD_CALL.pack(T, D, Hq, Hk, wqp, wkp, kind, interleaved, weight_bias, eps, *_rotation(cos_sin, dev),
                                   *gqp, *gkp, *qp, *kp, *dqp, *dkp, dwqp, dwkp, wsp, wsn))
    return dq, dk, dwq, dwk


def _cache_scale(scale, name, fp8, dev):
    if not fp8:
        if scale is not None:
            raise ValueError(f"{name} without an FP8 cache")
        return 0
    if not isinstance(scale, torch.Tensor) or scale.dtype is not _F32 or scale.get_device() != dev or scale.numel() != 1:
        raise TypeError(f"{name} must be a float32 tensor of one value on cuda:{dev}")
    return scale.data_ptr()


def qk_rmsnorm_rope_append(q, k, v, wq, wk, cos_sin, k_cache, v_cache, slots, eps: float = 1e-6,
                           weight_bias: float = 0.0, interleaved: bool = False, k_scale=None, v_scale=None,
                           q_out=None):
    """qk_rmsnorm_rope_fwd with the keys, and the values v, written to a paged
    cache: k_cache, v_cache are [pages, page_size, Hk, D] views (any strides
    with a contiguous D, e.g. a transposed [pages, Hk, page_size, D]) in BF16
    or FP8 (x / scale, k_scale and v_scale being float32 tensors of one
    value).  Token t goes to slot slots[t] = page * page_size + row (int32 or
    int64); a negative or too large slot writes nothing.  Slots must differ.
    q None: the cache alone.  Returns q_out."""
    dev, kshape, T, Hk, D = _first_head_tensor(k, "k")
    kp, vp = _head_tensor(k, "k", dev, kshape), _head_tensor(v, "v", dev, kshape)
    Hq, qp, qo = 0, _ABSENT, _ABSENT
    if q is not None:
        shape, Hq = _kv_shape(kshape, q, "q")
        qp = _head_tensor(q, "q", dev, shape)
        if q_out is None:
            q_out, qo = _new_heads(q, Hq, D)
        else:
            qo = _head_tensor(q_out, "q_out", dev, shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    wqp, wkp, kind = _head_weights(wq, wk, D, dev, q is not None, True)
    ck = _CACHE.get(k_cache.dtype)
    if ck is None or v_cache.dtype is not k_cache.dtype or k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise TypeError(f"k_cache and v_cache must be bfloat16, float8_e4m3fn or float8_e5m2, both, on cuda:{dev}")
    cshape = k_cache.shape
    if len(cshape) != 4 or cshape != v_cache.shape or cshape[2] != Hk or cshape[3] != D:
        raise ValueError(f"k_cache and v_cache must be [pages, page_size, {Hk}, {D}]")
    kps, kss, khs, k1 = k_cache.stride()
    vps, vss, vhs, v1 = v_cache.stride()
    if D > 1 and (k1 != 1 or v1 != 1):
        raise ValueError("k_cache and v_cache: D must be contiguous")
    sk = _INDEX.get(slots.dtype)
    if sk is None or slots.get_device() != dev:
        raise TypeError(f"slots must be int32 or int64 on cuda:{dev}, got {slots.dtype} on {slots.device}")
    if slots.numel() != T or not slots.is_contiguous():
        raise ValueError("slots must be contiguous with one slot per token")
    fp8 = ck != _abi.CACHE_BF16
    _enqueue("qk_rmsnorm_rope_append", dev,
             _abi.QK_APPEND_CALL.pack(T, D, Hq, Hk, wqp, wkp, kind, interleaved, weight_bias, eps,
                                      *_rotation(cos_sin, dev), *qp, *kp, *vp, *qo, k_cache.data_ptr(), kps, kss, khs,
                                      v_cache.data_ptr(), vps, vss, vhs, ck, sk, cshape[0], cshape[1], slots.data_ptr(),
                                      _cache_scale(k_scale, "k_scale", fp8, dev),
                                      _cache_scale(v_scale, "v_scale", fp8, dev)))
    return q_out


# -------------------------------------------------------------- attention --

def attention_workspace_bytes(D: int, device=None) -> int:
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    n = _lib().attention_workspace_bytes(int(D), idx)
    if n == 0:
        raise CrmsnError("attention_workspace_bytes", 3, "invalid head size or device")
    return n


def attention_status(device=None) -> None:
    """Waits for `device` (default: the current one); raises CrmsnError if a
    wait inside an attention kernel has run out there since the last call of
    this function (rows of NaN, which no input causes)."""
    with torch.cuda.device(device):
        check("attention_status", _lib().attention_status(None))


_I32 = torch.int32


def _int32_vector(t, name, n, dev):
    if t.dtype is not _I32 or t.get_device() != dev:
        raise TypeError(f"{name} must be int32 on cuda:{dev}, got {t.dtype} on {t.device}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor")
    return t.data_ptr()


def _attention(q, shape, T, Hq, D, Hk, B, keys, dev, starts, scale, causal, window, out, lse, workspace):
    """(out, workspace, the fields of crmsn_attention): what the two attention
    functions share.  keys: the most that a sequence can have."""
    qp = _head_tensor(q, "q", dev, shape)
    if Hk < 1 or Hq % Hk:
        raise ValueError(f"{Hq} query heads are no multiple of {Hk} key heads")
    if out is None:
        out, op = _new_heads(q, Hq, D)
    else:
        op = _head_tensor(out, "out", dev, shape)
    lp = 0
    if lse is not None:
        if lse.dtype is not _F32 or lse.get_device() != dev or lse.shape != shape[:-1] or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 {tuple(shape[:-1])} tensor on cuda:{dev}")
        lp = lse.data_ptr()
    wsp = wsn = 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on cuda:{dev}")
        wsp, wsn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif keys > _abi.ATTENTION_SHORT:
        wsn = _lib().attention_workspace_bytes(D, dev)
        workspace = torch.empty(wsn, dtype=torch.uint8, device=q.device)
        wsp = workspace.data_ptr()
    return out, workspace, (T, D, Hq, Hk, B, *qp, *op, lp, 0 if starts is None else _int32_vector(starts, "starts", B + 1, dev),
                            D ** -0.5 if scale is None else scale, bool(causal), window, wsp, wsn)


def prompt_attention(q, k, v, starts=None, scale=None, causal: bool = True, window: int = 0, out=None, lse=None,
                     workspace=None):
    """Attention of every token of q [..., Hq, D] over the keys k and values v
    [..., Hk, D] of its own sequence: causal, over the last `window` keys
    (0: all), or over all of them.  Head h reads key head h // (Hq // Hk).
    starts (int32 [B + 1], on the device): the first token of each packed
    sequence, and the end of the last; None: [T, H, D] is one sequence, [B, S,
    H, D] holds B.  scale: of the scores, D ** -0.5 by default.  lse (float32
    [..., Hq]) receives the logarithms of the sums.  Forward only; a call in
    which gradients would be recorded is refused.  Returns out."""
    dev, shape, T, Hq, D = _first_head_tensor(q, "q")
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad):
        raise RuntimeError("prompt_attention has no gradient: call it under torch.no_grad()")
    kshape, Hk = _kv_shape(shape, k, "k")
    kp, vp = _head_tensor(k, "k", dev, kshape), _head_tensor(v, "v", dev, kshape)
    if starts is not None:
        if starts.dim() != 1 or starts.numel() < 1:
            raise ValueError("starts must be a contiguous [sequences + 1] tensor")
        B = starts.shape[0] - 1
    else:
        B = 1 if len(shape) == 3 else math.prod(shape[:-3])
    out, workspace, packed = _attention(q, shape, T, Hq, D, Hk, B, T // B if starts is None and B else T, dev, starts, scale, causal, window, out, lse, workspace)
    _enqueue("prompt_attention", dev, _abi.PROMPT_ATTENTION_CALL.pack(*packed, *kp, *vp))
    return out


def paged_attention(q, k_cache, v_cache, page_table, lens, starts=None, scale=None, causal: bool = True,
                    window: int = 0, k_scale=None, v_scale=None, out=None, lse=None, workspace=None):
    """Attention of new tokens q [..., Hq, D] over a paged cache (k_cache,
    v_cache and their scales as qk_rmsnorm_rope_append fills them; the new
    tokens' own keys among them).  Sequence b has lens[b] keys (int32), in the
    pages page_table[b] (int32 [B, pages]; what lies behind its last key is not
    read), and its new tokens are the last of them: starts (int32 [B + 1])
    names the first of each sequence, None: the tokens are shared out evenly
    (one each: a decode step).  The rest as in prompt_attention."""
    dev, shape, T, Hq, D = _first_head_tensor(q, "q")
    if torch.is_grad_enabled() and (q.requires_grad or k_cache.requires_grad or v_cache.requires_grad or
                                    any(s is not None and s.requires_grad for s in (k_scale, v_scale))):
        raise RuntimeError("paged_attention has no gradient: call it under torch.no_grad()")
    ck = _CACHE.get(k_cache.dtype)
    if ck is None or v_cache.dtype is not k_cache.dtype or k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise TypeError(f"k_cache and v_cache must be bfloat16, float8_e4m3fn or float8_e5m2, both, on cuda:{dev}")
    cshape = k_cache.shape
    if len(cshape) != 4 or cshape != v_cache.shape or cshape[3] != D:
        raise ValueError(f"k_cache and v_cache must be [pages, page_size, heads, {D}]")
    kps, kss, khs, k1 = k_cache.stride()
    vps, vss, vhs, v1 = v_cache.stride()
    if D > 1 and (k1 != 1 or v1 != 1):
        raise ValueError("k_cache and v_cache: D must be contiguous")
    if lens.dim() != 1:
        raise ValueError("lens must be a contiguous [sequences] tensor")
    B = lens.shape[0]
    lp = _int32_vector(lens, "lens", B, dev)
    if starts is None and (T % B if B else T):
        raise ValueError(f"{T} tokens cannot be shared out evenly over {B} sequences: give starts")
    if page_table.dtype is not _I32 or page_table.get_device() != dev:
        raise TypeError(f"page_table must be int32 on cuda:{dev}, got {page_table.dtype} on {page_table.device}")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be [{B}, pages]")
    ldt, t1 = page_table.stride()
    if page_table.shape[1] > 1 and t1 != 1:
        raise ValueError("page_table: a sequence's pages must be contiguous")
    out, workspace, packed = _attention(q, shape, T, Hq, D, cshape[2], B, page_table.shape[1] * cshape[1], dev, starts, scale,
                                        causal, window, out, lse, workspace)
    fp8 = ck != _abi.CACHE_BF16
    _enqueue("paged_attention", dev,
             _abi.PAGED_ATTENTION_CALL.pack(*packed, k_cache.data_ptr(), kps, kss, khs, v_cache.data_ptr(), vps, vss, vhs,
                                            cshape[0], cshape[1], page_table.data_ptr(), ldt, page_table.shape[1], lp,
                                            _cache_scale(k_scale, "k_scale", fp8, dev),
                                            _cache_scale(v_scale, "v_scale", fp8, dev), ck, 0))
    return out


def rmsnorm_supports(H: int, w_dtype: int = BF16, op: int = _abi.OP_FWD) -> int:
    return _lib().rmsnorm_supports(int(H), int(w_dtype), int(op))
