"""Operators of the training step over torch tensors.

Argument checks and marshalling only: the work runs in the CUDA kernels behind
the C ABI (``include/muon_adamw.h``, "Operators of the training step", which
has the formulas). Outputs are new tensors, allocated on the current stream,
on which the work is queued; nothing here waits for the GPU.

``embedding``, ``qk_norm_rope`` and ``window_attention`` each have a
``_backward`` function, and an ``_autograd`` form that torch's autograd
differentiates with it.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import MA_DT_BF16, MA_DT_F32, QkNormRope, WindowAttention, _check, load_library

_DT = {torch.float32: MA_DT_F32, torch.bfloat16: MA_DT_BF16}


def _on_gpu(first, **tensors) -> torch.device:
    """The device that every given tensor lies on."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError(f"the operators take CUDA tensors, not {dev.type} ones")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, not {dev}")
    return dev


def _dtype(name: str, t) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be fp32 or bf16, not {t.dtype}")
    return dt


def _call(dev, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream."""
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            _check(fn(*args, torch.cuda.current_stream().cuda_stream))
    else:
        _check(fn(*args, torch.cuda.current_stream().cuda_stream))


def _scratch(dev, fn, *args):
    """A workspace of as many bytes as fn(*args, &bytes) asks for."""
    n = ctypes.c_int64()
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            _check(fn(*args, ctypes.byref(n)))
    else:
        _check(fn(*args, ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=dev), n.value


# ---- embedding ----

def _ids(ids):
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, not {ids.dtype}")
    return ids if ids.is_contiguous() else ids.contiguous(), 8 if ids.dtype == torch.int64 else 4


def _rows(name: str, t, width: int):
    """(tensor, row stride) of `t` seen as rows of `width` elements."""
    if t.shape[-1] != width:
        raise ValueError(f"{name} has rows of {t.shape[-1]} elements, not {width}")
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= width:
        return t, t.stride(0)
    return t if t.is_contiguous() else t.contiguous(), width


def embedding(weight, ids, *, scale: float = 1.0, dtype: Optional[torch.dtype] = None):
    """scale * weight[ids], a row of zeros where an id is outside the vocabulary.

    weight: [vocab, width] fp32 or bf16, rows may be strided; ids: any shape,
    int32 or int64; dtype: the result's (the weight's by default)."""
    dev = _on_gpu(weight, ids=ids)
    if weight.dim() != 2 or (weight.shape[1] > 1 and weight.stride(1) != 1):
        raise ValueError("weight must be [vocab, width] with consecutive elements in a row")
    vocab, width = weight.shape
    ids, id_bytes = _ids(ids)
    out = torch.empty((*ids.shape, width), dtype=dtype or weight.dtype, device=dev)
    _call(dev, load_library().muon_adamw_embedding, weight.data_ptr(), _dtype("weight", weight),
          weight.stride(0) if vocab > 1 else width, vocab, width, ids.data_ptr(), id_bytes, ids.numel(), float(scale),
          out.data_ptr(), _dtype("out", out), width)
    return out


def embedding_backward(dout, ids, grad, *, scale: float = 1.0, accumulate: bool = False):
    """The lookup's dense gradient, written into `grad` ([vocab, width] fp32 or
    bf16, e.g. the buffer registered with the optimizer) or, with
    `accumulate`, added to it. Returns `grad`."""
    dev = _on_gpu(grad, ids=ids, dout=dout)
    if grad.dim() != 2 or (grad.shape[1] > 1 and grad.stride(1) != 1):
        raise ValueError("grad must be [vocab, width] with consecutive elements in a row")
    vocab, width = grad.shape
    ids, id_bytes = _ids(ids)
    if dout.shape[:-1] != ids.shape:
        raise ValueError(f"dout {tuple(dout.shape)} does not belong to ids {tuple(ids.shape)}")
    dout, dstride = _rows("dout", dout, width)
    lib = load_library()
    ws, n = _scratch(dev, lib.muon_adamw_embedding_backward_workspace, ids.numel(), vocab, width)
    _call(dev, lib.muon_adamw_embedding_backward, dout.data_ptr(), _dtype("dout", dout), dstride, ids.data_ptr(),
          id_bytes, ids.numel(), float(scale), grad.data_ptr(), _dtype("grad", grad),
          grad.stride(0) if vocab > 1 else width, vocab, width, 1 if accumulate else 0, ws.data_ptr(), n)
    return grad


# ---- norm and rotation of queries and keys ----

def _heads(name: str, t, dim: Optional[int] = None):
    """`t` as [token, head, head_dim] whose elements of a head are consecutive."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [token, head, head_dim], not {tuple(t.shape)}")
    if dim is not None and t.shape[2] != dim:
        raise ValueError(f"{name} has heads of {t.shape[2]} elements, not {dim}")
    return t if t.stride(2) == 1 or t.shape[2] == 1 else t.contiguous()


def _strides(t):
    """(token stride, head stride); 0 for a single token or head, whose stride says nothing."""
    return t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if t.shape[1] > 1 else 0


def _qk(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours):
    dev = _on_gpu(q, k=k, q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin, positions=positions)
    q = _heads("q", q)
    n, h, dim = q.shape
    k = _heads("k", k, dim)
    if k.shape[0] != n:
        raise ValueError(f"q has {n} tokens and k has {k.shape[0]}")
    if k.dtype != q.dtype:
        raise TypeError(f"q is {q.dtype} and k is {k.dtype}")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w.dtype != torch.float32 or w.shape != (dim,) or not w.is_contiguous():
            raise ValueError(f"{name} must be {dim} contiguous fp32 values")
    if (cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.dim() != 2 or cos.shape != sin.shape
            or not cos.is_contiguous() or not sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous fp32 tables of one shape [position, rotated pairs]")
    if positions.dtype not in (torch.int32, torch.int64) or positions.shape != (n,) or not positions.is_contiguous():
        raise ValueError(f"positions must be {n} contiguous int32 or int64 values")
    d = QkNormRope(n, h, k.shape[1], dim, 2 * cos.shape[1], _dtype("q", q), 1 if neighbours else 0,
                   8 if positions.dtype == torch.int64 else 4, 0, float(eps), q.data_ptr(), k.data_ptr(), *_strides(q),
                   *_strides(k), q_weight.data_ptr(), k_weight.data_ptr(), cos.data_ptr(),
                   sin.data_ptr(), cos.shape[0], positions.data_ptr())
    return dev, q, k, d


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6, neighbours: bool = False):
    """RMS norm of every head of q and k, then the rotation by the token's
    position. q, k: [token, head, head_dim] fp32 or bf16 (e.g. slices of one
    projection's output); weights and tables fp32. Returns contiguous
    (q_out, k_out)."""
    dev, q, k, d = _qk(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    k_out = torch.empty(k.shape, dtype=q.dtype, device=dev)
    _call(dev, load_library().muon_adamw_qk_norm_rope, d, q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6,
                          neighbours: bool = False):
    """(dq, dk, dq_weight, dk_weight) from the outputs' gradients and the
    forward call's inputs; the weights' gradients are fp32."""
    dev, q, k, d = _qk(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)
    _on_gpu(q, dq_out=dq_out, dk_out=dk_out)
    if dq_out.shape != q.shape or dk_out.shape != k.shape or dq_out.dtype != q.dtype or dk_out.dtype != q.dtype:
        raise ValueError("dq_out and dk_out must have the shapes and the type of q and k")
    dq_out, dk_out = _heads("dq_out", dq_out), _heads("dk_out", dk_out)
    lib = load_library()
    ws, n = _scratch(dev, lib.muon_adamw_qk_norm_rope_backward_workspace, d)
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
    dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
    dw = torch.empty((2, q.shape[2]), dtype=torch.float32, device=dev)
    dqw, dkw = dw[0], dw[1]
    _call(dev, lib.muon_adamw_qk_norm_rope_backward, d, dq_out.data_ptr(), *_strides(dq_out),
          dk_out.data_ptr(), *_strides(dk_out), dq.data_ptr(), dk.data_ptr(), dqw.data_ptr(),
          dkw.data_ptr(), ws.data_ptr(), n)
    return dq, dk, dqw, dkw


# ---- attention ----

def _apart(name: str, t, dim: Optional[int] = None):
    """``_heads``, with no two heads on the same elements (as in an expanded tensor)."""
    t = _heads(name, t, dim)
    return t.contiguous() if any(t.shape[i] > 1 and t.stride(i) < t.shape[2] for i in (0, 1)) else t


def _attention(q, k, v, window, sinks, scale, cu_seqlens):
    dev = _on_gpu(q, k=k, v=v, cu_seqlens=cu_seqlens)
    q = _apart("q", q)
    n, h, dim = q.shape
    k, v = _apart("k", k, dim), _apart("v", v, dim)
    if k.shape[0] != n or v.shape != k.shape:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not fit together")
    if q.dtype != torch.bfloat16 or k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("q, k and v must be bf16")
    n_seqs, cu = 0, None
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() \
                or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be at least 2 contiguous int32 values")
        n_seqs, cu = cu_seqlens.numel() - 1, cu_seqlens.data_ptr()
    d = WindowAttention(n, h, k.shape[1], dim, int(sinks), n if window is None else int(window),
                        1.0 / math.sqrt(dim) if scale is None else float(scale), cu, n_seqs, 0, q.data_ptr(),
                        k.data_ptr(), v.data_ptr(), *_strides(q), *_strides(k), *_strides(v))
    return dev, q, k, v, d


def window_attention(q, k, v, *, window: Optional[int], sinks: int = 0, scale: Optional[float] = None,
                     cu_seqlens=None):
    """Causal attention of packed samples: a query sees the `window` last keys
    of its sample (itself among them; None: all) and the sample's first
    `sinks` keys. q: [token, head, head_dim] bf16; k, v: [token, kv head,
    head_dim]; cu_seqlens: int32 bounds of the samples on the GPU (None: one
    sample); scale: 1 / sqrt(head_dim) by default. Returns (out, lse): out like
    q, lse [head, token] fp32."""
    dev, q, k, v, d = _attention(q, k, v, window, sinks, scale, cu_seqlens)
    out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=dev)
    _call(dev, load_library().muon_adamw_window_attention, d, out.data_ptr(), lse.data_ptr())
    return out, lse


def window_attention_backward(dout, q, k, v, out, lse, *, window: Optional[int], sinks: int = 0,
                              scale: Optional[float] = None, cu_seqlens=None):
    """(dq, dk, dv) from the output's gradient, the forward call's inputs and
    what it returned."""
    dev, q, k, v, d = _attention(q, k, v, window, sinks, scale, cu_seqlens)
    _on_gpu(q, dout=dout, out=out, lse=lse)
    if dout.shape != q.shape or out.shape != q.shape or dout.dtype != q.dtype or out.dtype != q.dtype:
        raise ValueError("dout and out must have the shape and the type of q")
    if lse.shape != (q.shape[1], q.shape[0]) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [head, token]")
    dout = _apart("dout", dout)
    out = out if out.is_contiguous() else out.contiguous()
    lib = load_library()
    ws, n = _scratch(dev, lib.muon_adamw_window_attention_backward_workspace, d)
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
    dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
    dv = torch.empty(k.shape, dtype=q.dtype, device=dev)
    _call(dev, lib.muon_adamw_window_attention_backward, d, dout.data_ptr(), *_strides(dout),
          out.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), n)
    return dq, dk, dv


def check() -> None:
    """Wait for the current stream; raises if a bounded wait of an attention
    kernel has run out (a fault of the machine or of the library)."""
    _check(load_library().muon_adamw_window_attention_check(torch.cuda.current_stream().cuda_stream))


# ---- forms for autograd ----

class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, dtype):
        ctx.save_for_backward(ids)
        ctx.like, ctx.scale = (weight.shape, weight.dtype, weight.device), scale
        return embedding(weight, ids, scale=scale, dtype=dtype)

    @staticmethod
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
    def backward(ctx, dq_out, dk_out):
        return (*qk_norm_rope_backward(dq_out, dk_out, *ctx.saved_tensors, **ctx.how), None, None, None, None, None)


class _WindowAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, window, sinks, scale):
        ctx.how = {"window": window, "sinks": sinks, "scale": scale, "cu_seqlens": cu_seqlens}
        out, lse = window_attention(q, k, v, **ctx.how)
        ctx.save_for_backward(q, k, v, out, lse)
        return out

    @staticmethod
    def backward(ctx, dout):
        return (*window_attention_backward(dout, *ctx.saved_tensors, **ctx.how), None, None, None, None)


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
