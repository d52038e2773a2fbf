"""The two ends of a language model's training step as torch functions: embedding, linear cross
entropy and gradient clipping (the library's embed_*, linear_ce_* and grad_* calls).

    Y = embedding(ids, E, scale)              # rows of E, differentiable in E
    loss = linear_cross_entropy(X, W, t)      # mean over targets inside [0, V), differentiable in X and W
    norm = clip_grad_norm(params, max_norm)   # scales .grad in place, returns the norm before

ids and targets outside [0, V) take no part: padding rows are zero and masked tokens (-100, say)
cost nothing and get zero gradients.  Second derivatives pass through embedding; the gradients of
linear_cross_entropy have none, and differentiating them raises an error.  Nothing here reads back to the host, so a step made of these
can be captured in a HIP graph; as with any autograd capture, drop the losses and gradients of eager
steps on the same parameters first (their graph holds the parameters' accumulation nodes on the
eager stream).

Argument marshalling only: every step runs in the HIP library.
"""
from __future__ import annotations

import torch

from . import binding as csp


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, E, ids, scale):
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale = E.shape[0], scale
        return csp.embed_fwd(E, ids, scale)

    @staticmethod
    def backward(ctx, dY):
        (ids,) = ctx.saved_tensors
        return _EmbeddingGrad.apply(dY.contiguous(), ids, ctx.vocab, ctx.scale), None, None


class _EmbeddingGrad(torch.autograd.Function):
    """dE of dY, which is linear in it: its own gradient is the lookup."""

    @staticmethod
    def forward(ctx, dY, ids, vocab, scale):
        ctx.save_for_backward(ids)
        ctx.scale = scale
        return csp.embed_bwd(dY, ids, vocab, scale)

    @staticmethod
    def backward(ctx, ddE):
        (ids,) = ctx.saved_tensors
        return _Embedding.apply(ddE.contiguous(), ids, ctx.scale), None, None, None


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, targets):
        loss, lse, total = csp.linear_ce_fwd(X, W, targets)
        ctx.save_for_backward(X, W, targets, lse, total)
        return total[2].clone()  # the backward reads total; the caller may change its loss in place

    @staticmethod
    def backward(ctx, dmean):
        X, W, targets, lse, total = ctx.saved_tensors
        need = ctx.needs_input_grad[:2]
        dX, dW = _LinearCrossEntropyGrad.apply(X, W, targets, lse, dmean.reshape(1).contiguous(), total, need)
        return dX, dW, None


class _LinearCrossEntropyGrad(torch.autograd.Function):
    """dX and dW.  Under create_graph=True they hang on X, W and dmean, so that differentiating them (a penalty
    on a gradient, say) arrives here; otherwise they would pass for constants and their part be dropped."""

    @staticmethod
    def forward(ctx, X, W, targets, lse, dmean, total, need):
        args = X, W, targets, lse, dmean, total
        if all(need):
            return csp.linear_ce_bwd(*args)
        return (csp.linear_ce_bwd_input(*args), None) if need[0] else (None, csp.linear_ce_bwd_weight(*args))

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the gradients of linear_cross_entropy cannot be differentiated")


def embedding(ids, E, scale: float = 1.0):
    """scale * E[ids] as [*ids.shape, D]; a zero row for an id outside [0, V)."""
    Y = _Embedding.apply(E, ids.reshape(-1).contiguous(), float(scale))
    return Y.view(*ids.shape, E.shape[1])


def linear_cross_entropy(X, W, targets):
    """Mean cross entropy of the logits X W^T [..., V] (never stored) against targets [...], as an fp32
    scalar; the mean is over the targets inside [0, V), and 0 if there are none."""
    if tuple(X.shape[:-1]) != tuple(targets.shape):
        raise ValueError(f"X is {tuple(X.shape)} but targets are {tuple(targets.shape)}")
    return _LinearCrossEntropy.apply(X.reshape(-1, X.shape[-1]).contiguous(), W, targets.reshape(-1).contiguous())


@torch.no_grad()
def clip_grad_norm(params, max_norm: float):
    """Scale the gradients of the parameters (or of the one parameter) in place by min(1, max_norm / (norm +
    1e-6)); returns the norm over all of them before that, as an fp32 tensor [1].  A parameter listed twice
    is an error."""
    params = [params] if isinstance(params, torch.Tensor) else params
    grads = [p.grad for p in params if p.grad is not None]
    norm = csp.grad_clip(grads, max_norm)
    torch.autograd.graph.increment_version(grads)  # a write in place that torch did not see
    return norm
