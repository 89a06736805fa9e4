"""torch.autograd bindings of the block and of varlen attention, so that the
library's forward and backward calls can sit inside a training step
("DanLing NestedTensor" section 4.1 and Appendix A.1: the measured step is
forward, the sample-weighted loss and the backward).  Argument marshalling
only: the forward and the backward of each Function are the C-ABI calls of
``nt``.

    z_t, s_out = pair_block(part, s, W_a, W_b, ln_gamma, ln_beta, W1, b1, W2, b2, W_g, b_g)
    o = varlen_attention(q, k, v, cu_seqlens, max_len)

``pair_block`` is the ReLU block of Eq. 1 on a square partition (the
forward: nt_pair_broadcast, nt_pair_transition, nt_pair_reduce; the
backward: nt_pair_block_backward, whose gradients are fp32 and are returned
in the dtype of each input).  ``varlen_attention`` is non-causal or causal
self-attention over cu_seqlens segments (the forward keeps the natural-log
LSE; the backward is nt_varlen_attn_bwd).  ``qk_norm_rope`` gives packed
queries and keys their norms and positions before it (nt_qk_norm_rope; the
backward is nt_qk_norm_rope_bwd):

    q, k = qk_norm_rope(q, k, turns, cu_seqlens=cu_seqlens, q_gamma=g_q, k_gamma=g_k)
"""
from __future__ import annotations

from types import SimpleNamespace
from typing import Optional

import torch

from . import nt


class _FirstOnly(torch.autograd.Function):
    """Passes gradients on, as copies (views of its inputs could not be
    changed in place); raises when they are differentiated."""

    @staticmethod
    def forward(ctx, name, n, *tensors):
        ctx.name = name
        return tuple(t.clone() for t in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name} has first derivatives only")


def _first_only(name, grads, *of):
    """The gradients a Function's backward returns, computed by the library
    from the tensors ``of``.  The calls are opaque to autograd, so with
    create_graph the gradients would pass for constants; here they depend on
    ``of`` through a node that raises.  (torch's once_differentiable looks at
    the upstream gradients only, and lets a constant one through.)"""
    if not torch.is_grad_enabled() or not any(t is not None and t.requires_grad for t in of):
        return grads
    at = [i for i, g in enumerate(grads) if g is not None]
    kept = _FirstOnly.apply(name, len(at), *(grads[i] for i in at), *of)
    out = list(grads)
    for i, g in zip(at, kept):
        out[i] = g
    return tuple(out)


class PairBlock(torch.autograd.Function):
    @staticmethod
    def forward(ctx, part, s, W_a, W_b, ln_gamma, ln_beta, W1, b1, W2, b2, W_g, b_g, ln_eps):
        w = SimpleNamespace(W_a=W_a, W_b=W_b, ln_gamma=ln_gamma, ln_beta=ln_beta, W1=W1, b1=b1, W2=W2, b2=b2,
                            W_g=W_g, b_g=b_g)
        z_t, m, s_out = nt.block_forward(part, s, w, ln_eps=ln_eps)
        ctx.part = part
        ctx.ln_eps = ln_eps
        ctx.has_b = (b1 is not None, b2 is not None, b_g is not None)
        ctx.save_for_backward(s, W_a, W_b, ln_gamma, ln_beta, W1, b1 if b1 is not None else s.new_empty(0),
                              W2, b2 if b2 is not None else s.new_empty(0), W_g,
                              b_g if b_g is not None else s.new_empty(0), m)
        return z_t, s_out

    @staticmethod
    def backward(ctx, dz_t, ds_out):
        s, W_a, W_b, ln_gamma, ln_beta, W1, b1, W2, b2, W_g, b_g, m = ctx.saved_tensors
        has_b1, has_b2, has_bg = ctx.has_b
        w = SimpleNamespace(W_a=W_a, W_b=W_b, ln_gamma=ln_gamma, ln_beta=ln_beta, W1=W1,
                            b1=b1 if has_b1 else None, W2=W2, b2=b2 if has_b2 else None, W_g=W_g,
                            b_g=b_g if has_bg else None)
        f32 = lambda t: None if t is None else t.float().contiguous()
        if ds_out is None:
            ds_out = torch.zeros(s.shape[0], W_g.shape[0], dtype=torch.float32, device=s.device)
        g = nt.nt_pair_block_backward(ctx.part, s, w, m, f32(ds_out), f32(dz_t), ln_eps=ctx.ln_eps)
        like = lambda grad, t: grad.to(t.dtype)
        grads = (like(g["ds"], s), like(g["dW_a"], W_a), like(g["dW_b"], W_b), like(g["dgamma"], ln_gamma),
                 like(g["dbeta"], ln_beta), like(g["dW1"], W1), like(g["db1"], b1) if has_b1 else None,
                 like(g["dW2"], W2), like(g["db2"], b2) if has_b2 else None, like(g["dW_g"], W_g),
                 like(g["db_g"], b_g) if has_bg else None)
        return (None, *_first_only("pair_block", grads, dz_t, ds_out, s, W_a, W_b, ln_gamma, ln_beta, W1, b1, W2, b2,
                                   W_g, b_g), None)


def pair_block(part: "nt.Partition", s: torch.Tensor, W_a, W_b, ln_gamma, ln_beta, W1, b1, W2, b2, W_g, b_g,
               ln_eps: float = 1e-5):
    """The ReLU block of Eq. 1 with autograd: returns (z~, s_out).  First
    derivatives only: differentiating the gradients raises."""
    return PairBlock.apply(part, s, W_a, W_b, ln_gamma, ln_beta, W1, b1, W2, b2, W_g, b_g, ln_eps)


class VarlenAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, max_len, causal, scale):
        o, lse = nt.nt_varlen_attn_qk(q, k, v, cu_seqlens, cu_seqlens, max_len, scale=scale, causal=causal,
                                      want_lse=True)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.max_len, ctx.causal, ctx.scale = max_len, causal, scale
        return o

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, o, lse, cu = ctx.saved_tensors
        dq, dk, dv = nt.nt_varlen_attn_bwd(q, k, v, o, d_o.to(q.dtype).contiguous(), lse, cu, None, ctx.max_len,
                                           scale=ctx.scale, causal=ctx.causal)
        dq, dk, dv = _first_only("varlen_attention", (dq, dk, dv), d_o, q, k, v)
        return dq, dk, dv, None, None, None, None


def varlen_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, max_len: int,
                     causal: bool = False, scale: Optional[float] = None):
    """Self-attention within each cu_seqlens segment, with autograd.  First
    derivatives only: differentiating the gradients raises."""
    return VarlenAttention.apply(q, k, v, cu_seqlens, max_len, causal, scale)


class QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, turns, q_gamma, k_gamma, cu_seqlens, positions, pos0, eps, interleaved, rot_scale):
        q_gamma = None if q is None else q_gamma       # a gamma without its side takes no part
        k_gamma = None if k is None else k_gamma
        q_out, k_out = nt.nt_qk_norm_rope(q, k, turns, cu_seqlens=cu_seqlens, positions=positions, pos0=pos0,
                                          q_gamma=q_gamma, k_gamma=k_gamma, eps=eps, interleaved=interleaved,
                                          rot_scale=rot_scale)
        ctx.save_for_backward(q if q_gamma is not None else None, k if k_gamma is not None else None, turns, q_gamma,
                              k_gamma, cu_seqlens, positions, pos0)
        ctx.args = eps, interleaved, rot_scale
        return q_out, k_out

    @staticmethod
    def backward(ctx, dq_out, dk_out):
        q, k, turns, q_gamma, k_gamma, cu_seqlens, positions, pos0 = ctx.saved_tensors
        eps, interleaved, rot_scale = ctx.args
        uq, uk = (None if g is None else g.contiguous() for g in (dq_out, dk_out))
        dq, dk, dqg, dkg = nt.nt_qk_norm_rope_bwd(uq, uk, turns, q=q, k=k,
                                                  cu_seqlens=cu_seqlens, positions=positions, pos0=pos0,
                                                  q_gamma=q_gamma, k_gamma=k_gamma, eps=eps, interleaved=interleaved,
                                                  rot_scale=rot_scale)
        dq, dk, dqg, dkg = _first_only("qk_norm_rope", (dq, dk, dqg, dkg), dq_out, dk_out, q, k, q_gamma, k_gamma)
        return dq, dk, None, dqg, dkg, None, None, None, None, None, None


def qk_norm_rope(q: Optional[torch.Tensor], k: Optional[torch.Tensor], turns: Optional[torch.Tensor], cu_seqlens=None, positions=None,
                 pos0=None, q_gamma: Optional[torch.Tensor] = None, k_gamma: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, interleaved: bool = False, rot_scale: float = 1.0):
    """Per-head norm and rotary positions of packed q and k with autograd
    (:func:`nt.nt_qk_norm_rope`): returns (q_out, k_out), ready for
    :func:`varlen_attention`.  The gammas are fp32 leaves.  First derivatives
    only: differentiating the gradients raises."""
    return QKNormRope.apply(q, k, turns, q_gamma, k_gamma, cu_seqlens, positions, pos0, eps, interleaved, rot_scale)
