"""PyTorch autograd for the RMSNorm forward / backward kernels.

Source: "FlashInfer normalization operator guide" 6.2 and 6.4, and the
flashinfer.norm API index entries for cake_rmsnorm and CakeRMSNormFunction:
the function keeps only three tensors for the backward -- the tensor that was
normalised (x, or h_new = bf16(x + residual) on the residual route), the
weight and the FP32 rstd per row -- and returns the weight gradient, which
the kernel accumulates in FP32, in the weight's dtype.  On the residual route
the forward also returns h_new, and the gradient of x and of the residual is
the same tensor: the normalisation gradient plus the gradient flowing
straight into h_new.

Layouts: a tensor whose rows the kernels can read in place (row-collapsible,
contiguous features, ld >= H, 4-byte aligned, even stride) is passed as is;
any other layout (an expanded gradient, a transposed view, an odd offset) is
copied to a contiguous tensor once.

``qk_rmsnorm_rope`` is the same for queries and keys with their rotation: it
keeps q, k and the weights (rstd is computed again) and gives each weight's
gradient in the weight's dtype.
"""
from __future__ import annotations

import threading
import weakref

import torch

from . import binding
from .binding import qk_rmsnorm_rope_bwd, qk_rmsnorm_rope_fwd, rmsnorm_bwd, rmsnorm_fwd


def _readable(t: torch.Tensor) -> torch.Tensor:
    """t itself when the kernels can read its rows in place, else a
    contiguous copy."""
    try:
        rows, H, ld = binding.as_rows(t, "tensor")
    except ValueError:
        return t.contiguous()
    if (rows > 1 and (ld < H or ld % 2)) or t.data_ptr() % 4:
        # A fresh allocation (contiguous() would return a misaligned but
        # contiguous tensor unchanged).
        return t.clone(memory_format=torch.contiguous_format)
    return t


class RMSNormFunction(torch.autograd.Function):
    """y = RMSNorm(x) * (w + weight_bias), or (y, h_new) with a residual."""

    @staticmethod
    def forward(ctx, x, w, residual, eps, weight_bias):
        x = _readable(x)
        if residual is not None:
            residual = _readable(residual)
        y, rstd, h_new = rmsnorm_fwd(x, w, eps, residual=residual, weight_bias=weight_bias)
        ctx.save_for_backward(h_new if residual is not None else x, w, rstd)
        ctx.weight_bias = float(weight_bias)
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        if residual is not None:
            return y, h_new
        return y

    @staticmethod
    def backward(ctx, gy, gh=None):
        xn, w, rstd = ctx.saved_tensors
        if gy is None:
            gy = torch.zeros_like(xn)
        gy = _readable(gy)
        g_res = _readable(gh) if gh is not None else None
        dx, dw = rmsnorm_bwd(gy, xn, w, rstd.reshape(-1), weight_bias=ctx.weight_bias,
                             g_residual=g_res)
        dw = dw.to(w.dtype)
        if ctx.has_residual:
            return dx, dw, dx, None, None
        return dx, dw, None, None, None


def rmsnorm(x: torch.Tensor, w: torch.Tensor, eps: float = 1e-6, residual=None,
            weight_bias: float = 0.0):
    """Autograd-enabled RMSNorm: y (BF16, x's shape), or (y, h_new) when a
    residual is given (h_new = bf16(x + residual), the updated residual
    stream).  w is BF16 (weight_bias 1 for Gemma) or FP32 (weight_bias 1 for
    the zero-centred form)."""
    return RMSNormFunction.apply(x, w, residual, eps, weight_bias)


# The eager graphs of qk_rmsnorm_rope that are alive, each with its stream and
# its leaves.  A leaf's gradient is accumulated on the stream on which its
# first living graph was recorded; a captured backward pass that has to wait
# for another stream than its own ends the process, so such a capture is
# refused while it is still an ordinary call: at its forward, which cannot know
# whether a backward will follow.
_eager = weakref.WeakSet()
_eager_lock = threading.Lock()


def _note_graph(ctx, inputs):
    leaves = [t for t in inputs if t is not None and t.requires_grad and t.is_leaf and t.is_cuda]
    if not leaves:
        return
    stream = binding._stream(leaves[0])
    with _eager_lock:
        if not torch.cuda.is_current_stream_capturing():
            ctx.graph_stream, ctx.graph_leaves = stream, tuple(weakref.ref(t) for t in leaves)
            _eager.add(ctx)
            return
        held = [r() for c in _eager if c.graph_stream != stream for r in c.graph_leaves]
    if any(h is t for h in held for t in leaves):
        raise RuntimeError("qk_rmsnorm_rope: a graph recorded outside this capture, on another stream, still holds "
                           "one of these leaves; drop it (its outputs and losses) before capturing, or capture a forward "
                           "alone under torch.no_grad()")


def _readable_heads(t: torch.Tensor) -> torch.Tensor:
    """t itself when the kernels can read its heads in place, else a
    contiguous copy."""
    try:
        T, H, D, ld, hs = binding.as_heads(t, "tensor")
    except ValueError:
        return t.contiguous() if t.dim() >= 3 else t
    apart = (T <= 1 or ld >= D) and (H <= 1 or hs >= D)
    if apart and T > 1 and H > 1:
        apart = ld >= (H - 1) * hs + D or hs >= (T - 1) * ld + D
    return t if apart else t.clone(memory_format=torch.contiguous_format)


class QKRMSNormRopeFunction(torch.autograd.Function):
    """(q_out, k_out) of qk_rmsnorm_rope_fwd (k_out None without k);
    recording: whether gradients are being recorded (forward() itself always
    runs without)."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, cos_sin, eps, weight_bias, interleaved, recording):
        if cos_sin is not None and cos_sin.requires_grad:
            raise ValueError("cos_sin takes no gradient")
        if recording:
            _note_graph(ctx, (q, k, wq, wk))
        q = _readable_heads(q)
        k = None if k is None else _readable_heads(k)
        q_out, k_out = qk_rmsnorm_rope_fwd(q, k, wq, wk, cos_sin, eps, weight_bias, interleaved)
        norm = wq is not None
        ctx.save_for_backward(q if norm else None, k if norm else None, wq, wk, cos_sin)
        ctx.how = (eps, weight_bias, interleaved)
        ctx.shapes = (q.shape, None if k is None else k.shape)
        ctx.set_materialize_grads(False)
        return q_out, k_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        q, k, wq, wk, cos_sin = ctx.saved_tensors
        like = gq if gq is not None else gk
        if like is None:
            return (None,) * 9
        g = [None if shape is None else like.new_zeros(shape) if t is None else _readable_heads(t)
             for t, shape in zip((gq, gk), ctx.shapes)]
        dq, dk, dwq, dwk = qk_rmsnorm_rope_bwd(g[0], g[1], q, k, wq, wk, cos_sin, *ctx.how)
        return (dq, dk, None if dwq is None else dwq.to(wq.dtype), None if dwk is None else dwk.to(wk.dtype),
                None, None, None, None, None)


def qk_rmsnorm_rope(q: torch.Tensor, k, wq, wk, cos_sin, eps: float = 1e-6, weight_bias: float = 0.0,
                    interleaved: bool = False):
    """Autograd-enabled per-head RMSNorm and rotation of q [..., Hq, D] and k
    [..., Hk, D] (arguments as qk_rmsnorm_rope_fwd): (q_out, k_out).  cos_sin
    (rope_cos_sin) takes no gradient.  The gradients of all other inputs are
    worked out together, whichever are asked for.  Heads that no one token
    stride describes ([B, heads, S, D] storage with B > 1, gradients among
    them) are copied to a contiguous tensor once.

    To capture a training step, record the forward and the backward in one
    graph and let no eager graph of the same leaves live from another stream.
    One of this function's is seen, and the captured forward refused with
    RuntimeError while gradients are being recorded, with or without a
    backward to come (capture a forward alone under torch.no_grad()); graphs
    in which other operators hold the leaves are not seen."""
    return QKRMSNormRopeFunction.apply(q, k, wq, wk, cos_sin, eps, weight_bias, interleaved,
                                       torch.is_grad_enabled())
