"""Operators of the training step over torch tensors.

The work runs in the CUDA kernels behind the C ABI (``include/muon_adamw.h``,
"Operators of the training step", which has the formulas); arguments are
checked and results allocated by the extension module ``lib/_torch_ops.so``
(``csrc/torch_ops.cpp``). Outputs are new tensors, allocated on the current
stream, on which the work is queued; nothing here waits for the GPU.

``embedding``, ``qk_norm_rope``, ``window_attention``, ``dropout``,
``residual_norm``, ``expert_matmul`` and ``token_logprobs`` each have a
``_backward`` function, and an ``_autograd`` form that torch's autograd
differentiates with it, once: a second derivative raises. The plain forms
record no graph, whatever their arguments require: a result that a loss is to
reach the parameters through comes from an ``_autograd`` form. Queries, keys,
values, experts' inputs, weights and tables start every row on a 16-byte
boundary and are refused otherwise (MA_ERR_ALIGN); the rows of the residual
stream and of logits may start anywhere; gradients and saved outputs may lie in
any layout, at the price of a copy where the kernels cannot read it. Refused
arguments raise TypeError or ValueError, or MuonAdamWError with the library's
status.
"""
from __future__ import annotations

import functools
import importlib.machinery
import importlib.util
import os
from typing import Optional

import torch

from . import LibraryNotBuilt, _check, load_library
from . import build as _build


def _load():
    load_library()  # raises LibraryNotBuilt where nothing has been built
    path = _build.torch_ops_path()
    if not os.path.exists(path):
        raise LibraryNotBuilt(f"{path} is missing: build it with muon_adamw_hybrid_grad_gb300.build.build()\n"
                              f"{_build.torch_ops_problem()}".rstrip())
    loader = importlib.machinery.ExtensionFileLoader("_torch_ops", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_torch_ops", path, loader=loader))
    loader.exec_module(module)
    module.set_check(_check)
    return module


_ext = _load()


def embedding(weight, ids, *, scale: float = 1.0, dtype: Optional[torch.dtype] = None):
    """scale * weight[ids], a row of zeros where an id is outside the vocabulary.
    Records no graph, as no plain form does.

    weight: [vocab, width] fp32 or bf16, rows may be strided; ids: any shape,
    int32 or int64; dtype: the result's (the weight's by default)."""
    return _ext.embedding(weight, ids, scale, dtype)


def embedding_backward(dout, ids, grad, *, scale: float = 1.0, accumulate: bool = False):
    """The lookup's dense gradient, written into `grad` ([vocab, width] fp32 or
    bf16, e.g. the buffer registered with the optimizer) or, with
    `accumulate`, added to it. Returns `grad`."""
    return _ext.embedding_backward(dout, ids, grad, scale, accumulate)


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6, neighbours: bool = False):
    """RMS norm of every head of q and k, then the rotation by the token's
    position. q, k: [token, head, head_dim] fp32 or bf16 (e.g. slices of one
    projection's output); weights and the tables [position, rotated pairs]
    fp32; positions int32 or int64. Returns contiguous (q_out, k_out), which
    carry no graph."""
    return _ext.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6,
                          neighbours: bool = False):
    """(dq, dk, dq_weight, dk_weight) from the outputs' gradients and the
    forward call's inputs; the weights' gradients are fp32."""
    return _ext.qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)


def window_attention(q, k, v, *, window: Optional[int], sinks: int = 0, scale: Optional[float] = None,
                     cu_seqlens=None):
    """Causal attention of packed samples: a query sees the `window` last keys
    of its sample (itself among them; None: all) and the sample's first
    `sinks` keys. q: [token, head, head_dim] bf16; k, v: [token, kv head,
    head_dim]; cu_seqlens: int32 bounds of the samples on the GPU (None: one
    sample); scale: 1 / sqrt(head_dim) by default. Returns (out, lse): out like
    q, lse [head, token] fp32; they carry no graph."""
    return _ext.window_attention(q, k, v, window, sinks, scale, cu_seqlens)


def window_attention_backward(dout, q, k, v, out, lse, *, window: Optional[int], sinks: int = 0,
                              scale: Optional[float] = None, cu_seqlens=None):
    """(dq, dk, dv) from the output's gradient, the forward call's inputs and
    what it returned."""
    return _ext.window_attention_backward(dout, q, k, v, out, lse, window, sinks, scale, cu_seqlens)


def dropout(x, p: float, rng, *, site: int = 0):
    """x / (1 - p) where an element is kept, 0 where it is dropped; p counts in
    steps of 2^-16. No mask is stored: it follows from `rng`, two int64 values
    on the GPU (seed and step), and `site`, the number of the call within a
    step. x: any shape, fp32 or bf16. The values are read when the work runs:
    a captured call whose step is counted up in the graph drops others at
    every replay."""
    return _ext.dropout(x, p, rng, site)


def dropout_backward(dout, p: float, rng, *, site: int = 0):
    """The gradient: the same elements are kept. `rng` holds the values of the forward call."""
    return _ext.dropout(dout, p, rng, site)


def residual_norm(x, residual, weight, *, eps: float = 1e-6, p: float = 0.0, rng=None, site: int = 0,
                  eight_bit: bool = False):
    """(y, res): res = residual + dropout(x), y its RMS norm times `weight`,
    normalised before res is rounded. x: [..., width] fp32 or bf16; residual:
    the same shape, x's type or fp32, or None (then, without dropout, res is x
    itself); weight: fp32; p, rng, site: as of ``dropout`` over x's elements.
    With `eight_bit` (y, scales, res): y in float8_e4m3fn, scales [...] fp32 the
    values' factor for each row, its largest magnitude / 448."""
    return _ext.residual_norm(x, residual, weight, eps, p, rng, site, eight_bit)


def residual_norm_backward(dy, dres, res, weight, *, eps: float = 1e-6, p: float = 0.0, rng=None, site: int = 0):
    """(dx, dresidual, dweight) from the gradients of y and of res (None: no
    other use of it) and from res as the forward call returned it. dx is
    dresidual itself where no dropout and no change of type lies between them."""
    return _ext.residual_norm_backward(dy, dres, res, weight, eps, p, rng, site)


def expert_matmul(x, weight, offsets):
    """out[t] = weight[e] @ x[t] for the tokens t of expert e, which lie
    together: offsets[e] to offsets[e + 1] - 1. x: [token, inner] bf16; weight:
    [expert, outer, inner] bf16; offsets: int32 on the GPU, ascending from 0.
    Tokens behind the last expert's get rows of zeros."""
    return _ext.expert_matmul(x, weight, offsets)


def expert_matmul_backward(dout, x, weight, offsets, grad, *, accumulate: bool = False, input_grad: bool = True):
    """(dx, grad): the gradient of x (None without `input_grad`) and the
    weights', written into `grad` ([expert, outer, inner] fp32 or bf16, whose
    matrices can be the buffers registered with the optimizer) or, with
    `accumulate`, added to it. grad None: not formed."""
    return _ext.expert_matmul_backward(dout, x, weight, offsets, grad, accumulate, input_grad)


def token_logprobs(logits, ids, *, scale: float = 1.0, top: int = 0):
    """(logprobs, entropy, lse, top_logprobs, top_ids) of softmax(scale *
    logits): the log probability of each given token (0 where its id is outside
    the vocabulary), the entropy and the log of the sum in fp32, and the `top`
    (at most 32) likeliest tokens, the lowest id first among equal ones. logits:
    [..., vocab] fp32 or bf16; ids: [...] int32 or int64."""
    return _ext.token_logprobs(logits, ids, scale, top)


def token_logprobs_backward(dlogprobs, dentropy, logits, ids, entropy, lse, *, scale: float = 1.0):
    """The logits' gradient, in their type, from the gradients of logprobs and
    of entropy (either may be None) and what the forward call took and returned."""
    return _ext.token_logprobs_backward(dlogprobs, dentropy, logits, ids, entropy, lse, scale)


def check() -> None:
    """Wait for the current stream; raises if a bounded wait of an operator's
    kernel has run out (a fault of the machine or of the library)."""
    _check(load_library().muon_adamw_operators_check(torch.cuda.current_stream().cuda_stream))


# ---- forms for autograd ----

class _FirstOrder(torch.autograd.Function):
    """The gradients, unchanged, as a function of what they were formed from: differentiating them raises. Left
    without a graph they would count as constants."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(x.view_as(x) for x in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the operators have no second derivative")


def _first_order(backward):
    """For the backward functions below, whose kernels record no graph of their own."""
    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            outputs = backward(ctx, *grads)
        if not torch.is_grad_enabled():  # no create_graph
            return outputs
        formed_from = [x for x in (*grads, *ctx.saved_tensors) if x is not None and x.requires_grad]
        if not formed_from:
            return outputs
        some = [x for x in outputs if x is not None]
        some = iter(_FirstOrder.apply(len(some), *some, *formed_from))
        return tuple(None if x is None else next(some) for x in outputs)
    return run


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, dtype):
        ctx.save_for_backward(ids)
        ctx.like, ctx.scale = (weight.shape, weight.dtype, weight.device), scale
        return embedding(weight, ids, scale=scale, dtype=dtype)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        (ids,) = ctx.saved_tensors
        shape, dtype, dev = ctx.like
        grad = torch.empty(shape, dtype=dtype, device=dev)
        return embedding_backward(dout, ids, grad, scale=ctx.scale), None, None, None


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.how = {"eps": eps, "neighbours": neighbours}
        return qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, **ctx.how)

    @staticmethod
    @_first_order
    def backward(ctx, dq_out, dk_out):
        return (*qk_norm_rope_backward(dq_out, dk_out, *ctx.saved_tensors, **ctx.how), None, None, None, None, None)


class _WindowAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, window, sinks, scale):
        ctx.how = {"window": window, "sinks": sinks, "scale": scale}
        out, lse = window_attention(q, k, v, cu_seqlens=cu_seqlens, **ctx.how)
        # the bounds too: autograd then refuses a gradient behind a write to them
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        return out

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        *saved, cu_seqlens = ctx.saved_tensors
        return (*window_attention_backward(dout, *saved, cu_seqlens=cu_seqlens, **ctx.how), None, None, None, None)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, rng, site):
        ctx.save_for_backward(rng)  # autograd then refuses a gradient behind a new step
        ctx.how = (p, site)
        return dropout(x, p, rng, site=site)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        (rng,) = ctx.saved_tensors
        return dropout_backward(dout, ctx.how[0], rng, site=ctx.how[1]), None, None, None


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, p, rng, site):
        ctx.how = {"eps": eps, "p": p, "site": site}
        y, res = residual_norm(x, residual, weight, rng=rng, **ctx.how)
        ctx.save_for_backward(res, weight, rng)
        ctx.dtype = y.dtype
        ctx.set_materialize_grads(False)
        ctx.alone = res is x
        return y if ctx.alone else (y, res)

    @staticmethod
    @_first_order
    def backward(ctx, dy, dres=None):
        res, weight, rng = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(res.shape, dtype=ctx.dtype, device=res.device)
        dx, dresidual, dweight = residual_norm_backward(dy, dres, res, weight, rng=rng, **ctx.how)
        return dx, dresidual if ctx.needs_input_grad[1] else None, dweight, None, None, None, None


class _ExpertMatmul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, offsets):
        ctx.save_for_backward(x, weight, offsets)
        return expert_matmul(x, weight, offsets)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        x, weight, offsets = ctx.saved_tensors
        grad = torch.empty(weight.shape, dtype=weight.dtype, device=weight.device) if ctx.needs_input_grad[1] else None
        dx, grad = expert_matmul_backward(dout, x, weight, offsets, grad, input_grad=ctx.needs_input_grad[0])
        return dx, grad, None


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, scale, top):
        logprobs, entropy, lse, top_logprobs, top_ids = token_logprobs(logits, ids, scale=scale, top=top)
        ctx.save_for_backward(logits, ids, entropy, lse)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(top_logprobs, top_ids)
        return logprobs, entropy, top_logprobs, top_ids

    @staticmethod
    @_first_order
    def backward(ctx, dlogprobs, dentropy, *_):
        if dlogprobs is None and dentropy is None:
            return None, None, None, None
        return token_logprobs_backward(dlogprobs, dentropy, *ctx.saved_tensors, scale=ctx.scale), None, None, None


def embedding_autograd(weight, ids, *, scale: float = 1.0, dtype: Optional[torch.dtype] = None):
    """``embedding`` whose gradient reaches `weight` (dense, in its type)."""
    return _Embedding.apply(weight, ids, scale, dtype)


def qk_norm_rope_autograd(q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6,
                          neighbours: bool = False):
    """``qk_norm_rope`` whose gradients reach q, k and the two weights."""
    return _QkNormRope.apply(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)


def window_attention_autograd(q, k, v, *, window: Optional[int], sinks: int = 0, scale: Optional[float] = None,
                              cu_seqlens=None):
    """``window_attention`` (its output alone) whose gradients reach q, k and v."""
    return _WindowAttention.apply(q, k, v, cu_seqlens, window, sinks, scale)


def dropout_autograd(x, p: float, rng, *, site: int = 0):
    """``dropout`` whose gradient reaches x. `rng` is not to change before the gradient has been formed."""
    return _Dropout.apply(x, p, rng, site)


def residual_norm_autograd(x, residual, weight, *, eps: float = 1e-6, p: float = 0.0, rng=None, site: int = 0):
    """``residual_norm`` (without 8 bits) whose gradients reach x, residual and the weight."""
    got = _ResidualNorm.apply(x, residual, weight, eps, p, rng, site)
    return got if isinstance(got, tuple) else (got, x)


def expert_matmul_autograd(x, weight, offsets):
    """``expert_matmul`` whose gradients reach x and the weights (dense, in their type)."""
    return _ExpertMatmul.apply(x, weight, offsets)


def token_logprobs_autograd(logits, ids, *, scale: float = 1.0, top: int = 0):
    """``token_logprobs`` (without lse) whose gradients reach the logits from logprobs and entropy; the alternatives
    have none."""
    return _TokenLogprobs.apply(logits, ids, scale, top)
