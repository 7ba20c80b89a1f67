"""Operators of the training step over torch tensors.

The work runs in the CUDA kernels behind the C ABI (``include/muon_adamw.h``,
"Operators of the training step", which has the formulas); arguments are
checked and results allocated by the extension module ``lib/_torch_ops.so``
(``csrc/torch_ops.cpp``). Outputs are new tensors, allocated on the current
stream, on which the work is queued; nothing here waits for the GPU.

``embedding``, ``qk_norm_rope`` and ``window_attention`` each have a
``_backward`` function, and an ``_autograd`` form that torch's autograd
differentiates with it, once: a second derivative raises. The plain forms
record no graph, whatever their arguments require: a result that a loss is to
reach the parameters through comes from an ``_autograd`` form. Queries, keys,
values, weights and tables start every row on a 16-byte boundary and are
refused otherwise (MA_ERR_ALIGN); gradients and saved outputs may lie in any
layout, at the price of a copy where the kernels cannot read it. Refused arguments raise TypeError or ValueError, or
MuonAdamWError with the library's status.
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
