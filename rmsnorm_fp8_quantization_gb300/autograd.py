"""torch.autograd functions over the C ABI.

``layer_norm`` / ``rms_norm`` run the library's fused forward (saving mu and
rsigma) and, on backward, its fused backward.  ``*_with_residual`` also return
the input itself as a second, "extra" output (the residual branch of a
pre-norm block); when both outputs receive gradients, the backward adds the
residual's gradient inside the norm's backward kernel instead of in a
separate add ("Implementation:NVIDIA TransformerEngine Ops Fused Backward Add
RMSNorm", Description and I/O Contract: grad_input = norm backward +
residual gradient, plus grad_weight).

``rope`` rotates q and k to their positions in one launch; its backward is
the transposed rotation of both gradients in one launch, and saves nothing but
the positions and frequencies.

``attention`` runs the attention over whole sequences and saves its output and the
rows' logarithms of their sums; its backward computes the probabilities again.
``dropout`` (with the residual's addition) saves two numbers; its backward draws
the mask again.

Shapes (norms): x is [..., hidden], contiguous, on a CUDA device; gamma (and beta)
[hidden].  The outputs have x's dtype; weight gradients have the weights'
dtype.  Every step runs in the library's kernels; this module only reshapes
and marshals.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import ops

__all__ = ["layer_norm", "rms_norm", "layer_norm_with_residual", "rms_norm_with_residual", "rope",
           "attention", "dropout"]


def _rows(x: torch.Tensor, hidden: int) -> torch.Tensor:
    if x.shape[-1] != hidden:
        raise ValueError(f"last dimension {x.shape[-1]} != hidden {hidden}")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    return x.view(-1, hidden)


class _Norm(torch.autograd.Function):
    """Outputs (y, residual); residual is x passed through (or None)."""

    @staticmethod
    def forward(ctx, x, gamma, beta, norm, eps, zero_centered_gamma, sm_margin, residual):
        hidden = gamma.shape[0]
        x2 = _rows(x, hidden)
        o = ops.norm_fwd(x2, gamma, beta, norm=norm, eps=eps,
                         zero_centered_gamma=zero_centered_gamma, sm_margin=sm_margin,
                         training=True)
        ctx.save_for_backward(x2, gamma, o["mu"], o["rsigma"])
        ctx.norm, ctx.zcg, ctx.sm_margin = norm, zero_centered_gamma, sm_margin
        ctx.shape, ctx.has_beta = x.shape, beta is not None
        y = o["out"].view(x.shape)
        if not residual:
            return y, None
        # A new tensor object sharing x's storage: the extra output.
        return y, x.view(x.shape)

    @staticmethod
    def backward(ctx, dy, dres):
        x2, gamma, mu, rsigma = ctx.saved_tensors
        hidden = gamma.shape[0]
        if dy is None:
            dy = torch.zeros(ctx.shape, dtype=x2.dtype, device=x2.device)
        dz = dy.contiguous().view(-1, hidden)
        dr = None if dres is None else dres.contiguous().view(-1, hidden)
        dx, dg, db = ops.norm_bwd(dz, x2, mu, rsigma, gamma, dr, norm=ctx.norm,
                                  zero_centered_gamma=ctx.zcg, sm_margin=ctx.sm_margin)
        return (dx.view(ctx.shape), dg, db if ctx.has_beta else None,
                None, None, None, None, None)


def layer_norm(x, gamma, beta, eps=1e-5, zero_centered_gamma=False, sm_margin=0):
    """LayerNorm over the last dimension: (x - mu) * rsigma * g' + beta."""
    return _Norm.apply(x, gamma, beta, "layernorm", eps, zero_centered_gamma, sm_margin,
                       False)[0]


def rms_norm(x, gamma, eps=1e-6, zero_centered_gamma=False, sm_margin=0):
    """RMSNorm over the last dimension: x * rsigma * g'."""
    return _Norm.apply(x, gamma, None, "rmsnorm", eps, zero_centered_gamma, sm_margin, False)[0]


def layer_norm_with_residual(x, gamma, beta, eps=1e-5, zero_centered_gamma=False, sm_margin=0):
    """(layer_norm(x), x); the backward adds the second output's gradient to
    dx inside the norm's backward kernel."""
    return _Norm.apply(x, gamma, beta, "layernorm", eps, zero_centered_gamma, sm_margin, True)


def rms_norm_with_residual(x, gamma, eps=1e-6, zero_centered_gamma=False, sm_margin=0):
    """(rms_norm(x), x); the backward adds the second output's gradient to dx
    inside the norm's backward kernel (the fused backward-add)."""
    return _Norm.apply(x, gamma, None, "rmsnorm", eps, zero_centered_gamma, sm_margin, True)


def _no_gradient(name, value, where):
    if isinstance(value, torch.Tensor) and value.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, and {where} has none for it")


class _Rope(torch.autograd.Function):
    """(q, k) rotated; k may be None."""

    @staticmethod
    def forward(ctx, q, k, inv_freq, positions, layout, mscale):
        ctx.save_for_backward(inv_freq, positions)
        ctx.layout, ctx.mscale = layout, mscale
        ctx.set_materialize_grads(False)  # an unused output costs nothing
        return ops.rope_fwd(q, k, inv_freq, positions, layout=layout, mscale=mscale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        inv_freq, positions = ctx.saved_tensors
        dq, dk = (t if need else None for t, need in zip((dq, dk), ctx.needs_input_grad))
        # A gradient whose head elements are not contiguous (an expanded or
        # transposed view) is copied; other strides are taken as they are.
        dq, dk = (t if t is None or t.stride(-1) == 1 else t.contiguous() for t in (dq, dk))
        if dq is None and dk is None:
            return (None,) * 6
        dq, dk = ops.rope_bwd(dq, dk, inv_freq, positions, layout=ctx.layout, mscale=ctx.mscale)
        return dq, dk, None, None, None, None


def rope(q, k, inv_freq, positions=None, layout="half", mscale=1.0):
    """Rotary positions of q and k [batch, seq, heads, head_dim] (k may be
    None): ``ops.rope_fwd`` with its gradient, for q and k alone (inv_freq is refused
    where it requires one)."""
    _no_gradient("inv_freq", inv_freq, "rope")
    return _Rope.apply(q, k, inv_freq, positions, layout, mscale)


def _whole_rows(t):
    """t, or a copy where its strides are not what the attention takes."""
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0
    for n, st in zip(t.shape[:-1], t.stride()):
        ok = ok and (n <= 1 or st > 0 and st * t.element_size() % 16 == 0)
    if ok and t.dim() == 4 and t.shape[0] > 1 and t.shape[1] > 1:
        ok = t.stride(0) == t.shape[1] * t.stride(1)
    return t if ok else t.clone(memory_format=torch.contiguous_format)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, cu_seqlens_k, kw):
        q, k, v = (_whole_rows(t) for t in (q, k, v))
        # Padding rows are not written: zeros there, and in their gradients.
        out = None if cu_seqlens is None else torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        out, lse = ops.attention_fwd(q, k, v, cu_seqlens=cu_seqlens, cu_seqlens_k=cu_seqlens_k,
                                     out=out, **kw)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens, cu_seqlens_k)
        ctx.kw = kw
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, cu, cu_k = ctx.saved_tensors
        d = (None,) * 3
        if cu is not None:
            d = tuple(torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        dq, dk, dv = ops.attention_bwd(_whole_rows(dout), q, k, v, out, lse, cu_seqlens=cu,
                                       cu_seqlens_k=cu_k, dq=d[0], dk=d[1], dv=d[2], **ctx.kw)
        return dq, dk, dv, None, None, None


def attention(q, k, v, *, cu_seqlens=None, cu_seqlens_k=None, max_q=None, max_k=None, scale=None,
              causal=True, window=0):
    """``ops.attention_fwd`` with its gradient, for q, k and v; returns its output.  Padding rows
    of packed tensors get 0, in the output and in the gradients.  Tensors whose strides the
    kernels do not take are copied.  ``scale`` gets no gradient (a tensor that requires one is
    refused: multiply q by it)."""
    _no_gradient("scale", scale, "attention")
    kw = dict(max_q=max_q, max_k=max_k, scale=scale, causal=causal, window=window)
    return _Attention.apply(q, k, v, cu_seqlens, cu_seqlens_k, kw)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, rng, residual):
        # The caller's is advanced in place before the backward runs.
        rng = rng.clone()
        ctx.save_for_backward(rng)
        ctx.p = p
        return ops.dropout_fwd(x, p, rng, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        dx = None
        if ctx.needs_input_grad[0]:
            rng, = ctx.saved_tensors
            dx = ops.dropout_bwd(dout.contiguous(), ctx.p, rng)
        return dx, None, None, dout if ctx.needs_input_grad[3] else None


def dropout(x, p, rng, residual=None):
    """``ops.dropout_fwd`` with its gradient, for x and residual.  rng (seed, offset) is copied:
    the caller may advance it in place."""
    _no_gradient("p", p, "dropout")
    return _Dropout.apply(x, p, rng, residual)
