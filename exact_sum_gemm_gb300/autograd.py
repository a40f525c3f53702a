"""Layer norm, attention and token log probabilities as differentiable functions.

With DetLinear they make a decoder's training step whose every forward and
backward operation repeats bit for bit.  There are no second derivatives: asking
for one raises.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .training import (det_attention_backward, det_attention_forward, det_layer_norm_backward,
                       det_layer_norm_forward, det_token_logprobs_backward,
                       det_token_logprobs_forward)


class _LayerNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = det_layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, mean, rstd, weight, bias)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight, bias = ctx.saved_tensors
        dx, dweight, dbias = det_layer_norm_backward(
            dy.to(x.dtype), x, mean, rstd, weight, bias if ctx.needs_input_grad[2] else None,
            need_dx=ctx.needs_input_grad[0])
        return dx, dweight, dbias, None


def det_layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over x's last axis, differentiable (see det_layer_norm_forward)."""
    return _LayerNormFn.apply(x, weight, bias, eps)


class DetLayerNorm(torch.nn.Module):
    """Layer norm over the last axis with a learned weight and, by default, bias."""

    def __init__(self, width, eps=1e-5, bias=True, device=None, dtype=torch.float32):
        super().__init__()
        self.width, self.eps = int(width), float(eps)
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        if bias:
            self.bias = torch.nn.Parameter(torch.zeros(width, device=device, dtype=dtype))
        else:
            self.register_parameter("bias", None)

    def forward(self, x):
        if x.shape[-1] != self.width:
            raise ValueError(f"expected last dim {self.width}, got {x.shape[-1]}")
        return det_layer_norm(x, self.weight, self.bias, self.eps)

    def extra_repr(self):
        return f"width={self.width}, eps={self.eps}, bias={self.bias is not None}"


class _AttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale, k_lengths):
        o, lse = det_attention_forward(q, k, v, causal, scale, k_lengths)
        ctx.save_for_backward(q, k, v, o, lse, k_lengths)
        ctx.causal, ctx.scale = causal, scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, k_lengths = ctx.saved_tensors
        need_q, need_k, need_v = ctx.needs_input_grad[:3]
        dq, dk, dv = det_attention_backward(do.to(q.dtype), q, k, v, o, lse, ctx.causal, ctx.scale,
                                            k_lengths, need_dq=need_q, need_dkv=need_k or need_v)
        return dq, dk if need_k else None, dv if need_v else None, None, None, None


def det_attention(q, k, v, causal=False, scale=None, k_lengths=None):
    """softmax(scale q k^T) v, differentiable (see det_attention_forward)."""
    return _AttentionFn.apply(q, k, v, causal, scale, k_lengths)


class _TokenLogprobsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens):
        logprobs, entropy, stats, _, _ = det_token_logprobs_forward(logits, tokens)
        ctx.save_for_backward(logits, tokens, entropy, stats)
        ctx.set_materialize_grads(False)
        return logprobs, entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogprobs, dentropy):
        if dlogprobs is None and dentropy is None:
            return None, None
        logits, tokens, entropy, stats = ctx.saved_tensors
        return det_token_logprobs_backward(dlogprobs, dentropy, logits, tokens, entropy, stats), None


def det_token_logprobs(logits, tokens):
    """(logprobs, entropy) of logits [..., vocab] and tokens [...], differentiable.

    A negative token marks a place without one: its log probability is 0 and
    has no gradient.
    """
    if logits.dim() < 1 or logits.shape[-1] < 1:
        raise ValueError(f"logits must be [..., vocab], got {tuple(logits.shape)}")
    if tokens.shape != logits.shape[:-1]:
        raise ValueError(f"tokens must have shape {tuple(logits.shape[:-1])}, got {tuple(tokens.shape)}")
    vocab = logits.shape[-1]
    logprobs, entropy = _TokenLogprobsFn.apply(logits.reshape(-1, vocab), tokens.reshape(-1))
    return logprobs.reshape(tokens.shape), entropy.reshape(tokens.shape)
