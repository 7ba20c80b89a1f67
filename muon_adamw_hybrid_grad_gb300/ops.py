"""Operators of the training step over torch tensors.

Argument checks and marshalling only: the work runs in the CUDA kernels behind
the C ABI (``include/muon_adamw.h``, "Operators of the training step", which
has the formulas). Outputs are new tensors, allocated on the current stream,
on which the work is queued; nothing here waits for the GPU.

``embedding``, ``qk_norm_rope`` and ``window_attention`` each have a
``_backward`` function, and an ``_autograd`` form that torch's autograd
differentiates with it.

The smallest calls take a few microseconds on the GPU, so what the host does
for a call counts: sizes, strides and devices are read once each, and the
workspace sizes, which depend on sizes alone, are kept per combination.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch

from . import MA_DT_BF16, MA_DT_F32, QkNormRope, WindowAttention, _check, load_library

_empty = torch.empty
_F32, _BF16, _I32, _I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64
_DT = {_F32: MA_DT_F32, _BF16: MA_DT_BF16}
_device_now = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    _stream = torch._C._cuda_getCurrentRawStream
else:
    def _stream(dev: int) -> int:
        return torch.cuda.current_stream(dev).cuda_stream


def _apart_devices(names, tensors) -> None:
    """Raise for tensors that do not all lie on one GPU."""
    first = tensors[0].device
    if first.type != "cuda":
        raise ValueError(f"the operators take CUDA tensors, not {first.type} ones")
    for name, t in zip(names, tensors):
        if t.device != first:
            raise ValueError(f"{name} is on {t.device}, not {first}")


def _dtype(name: str, t) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be fp32 or bf16, not {t.dtype}")
    return dt


def _call(dev: int, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream."""
    if dev == _device_now():
        st = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    if st:
        _check(st)


def _bytes_of(dev: int, fn, *args) -> int:
    n = ctypes.c_int64()
    with torch.cuda.device(dev):
        _check(fn(*args, ctypes.byref(n)))
    return n.value


# ---- embedding ----

@functools.lru_cache(maxsize=1024)
def _embedding_bytes(dev: int, n: int, vocab: int, width: int) -> int:
    return _bytes_of(dev, load_library().muon_adamw_embedding_backward_workspace, n, vocab, width)


def _ids(ids):
    dt = ids.dtype
    if dt is not _I64 and dt is not _I32:
        raise TypeError(f"ids must be int32 or int64, not {dt}")
    return ids if ids.is_contiguous() else ids.contiguous(), 8 if dt is _I64 else 4


def _table(name: str, t):
    """(vocab, width, row stride) of a table whose rows' elements are consecutive."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [vocab, width], not {tuple(t.shape)}")
    vocab, width = t.shape
    stride, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{name} must have consecutive elements in a row")
    return vocab, width, stride if vocab > 1 else width


def embedding(weight, ids, *, scale: float = 1.0, dtype: Optional[torch.dtype] = None):
    """scale * weight[ids], a row of zeros where an id is outside the vocabulary.

    weight: [vocab, width] fp32 or bf16, rows may be strided; ids: any shape,
    int32 or int64; dtype: the result's (the weight's by default)."""
    dev = weight.get_device()
    if dev < 0 or ids.get_device() != dev:
        _apart_devices(("weight", "ids"), (weight, ids))
    vocab, width, stride = _table("weight", weight)
    ids, id_bytes = _ids(ids)
    out = _empty((*ids.shape, width), dtype=dtype or weight.dtype, device=weight.device)
    _call(dev, load_library().muon_adamw_embedding, weight.data_ptr(), _dtype("weight", weight), stride, vocab, width,
          ids.data_ptr(), id_bytes, ids.numel(), scale, out.data_ptr(), _dtype("out", out), width)
    return out


def embedding_backward(dout, ids, grad, *, scale: float = 1.0, accumulate: bool = False):
    """The lookup's dense gradient, written into `grad` ([vocab, width] fp32 or
    bf16, e.g. the buffer registered with the optimizer) or, with
    `accumulate`, added to it. Returns `grad`."""
    dev = grad.get_device()
    if dev < 0 or ids.get_device() != dev or dout.get_device() != dev:
        _apart_devices(("grad", "ids", "dout"), (grad, ids, dout))
    vocab, width, gstride = _table("grad", grad)
    ids, id_bytes = _ids(ids)
    shape = dout.shape
    if shape[:-1] != ids.shape:
        raise ValueError(f"dout {tuple(shape)} does not belong to ids {tuple(ids.shape)}")
    if shape[-1] != width:
        raise ValueError(f"dout has rows of {shape[-1]} elements, not {width}")
    dstride = width
    if not dout.is_contiguous():
        if len(shape) == 2 and dout.stride(1) == 1 and dout.stride(0) >= width:
            dstride = dout.stride(0)
        else:
            dout = dout.contiguous()
    n = ids.numel()
    size = _embedding_bytes(dev, n, vocab, width)
    ws = _empty(size, dtype=torch.uint8, device=grad.device)
    _call(dev, load_library().muon_adamw_embedding_backward, dout.data_ptr(), _dtype("dout", dout), dstride,
          ids.data_ptr(), id_bytes, n, scale, grad.data_ptr(), _dtype("grad", grad), gstride, vocab, width,
          1 if accumulate else 0, ws.data_ptr(), size)
    return grad


# ---- norm and rotation of queries and keys ----

def _heads(name: str, t, dim: Optional[int] = None):
    """(t, shape, token stride, head stride) of [token, head, head_dim] whose
    heads' elements are consecutive. The stride of a single token or head says
    nothing and counts as 0."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [token, head, head_dim], not {tuple(shape)}")
    n, h, d = shape
    if dim is not None and d != dim:
        raise ValueError(f"{name} has heads of {d} elements, not {dim}")
    ts, hs, one = t.stride()
    if one != 1 and d > 1:
        t = t.contiguous()
        ts, hs, one = t.stride()
    return t, shape, ts if n > 1 else 0, hs if h > 1 else 0


def _qk(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours):
    dev = q.get_device()
    if (dev < 0 or k.get_device() != dev or q_weight.get_device() != dev or k_weight.get_device() != dev
            or cos.get_device() != dev or sin.get_device() != dev or positions.get_device() != dev):
        _apart_devices(("q", "k", "q_weight", "k_weight", "cos", "sin", "positions"),
                       (q, k, q_weight, k_weight, cos, sin, positions))
    q, (n, h, dim), q_ts, q_hs = _heads("q", q)
    k, (nk, g, _), k_ts, k_hs = _heads("k", k, dim)
    if nk != n:
        raise ValueError(f"q has {n} tokens and k has {nk}")
    if k.dtype is not q.dtype:
        raise TypeError(f"q is {q.dtype} and k is {k.dtype}")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w.dtype is not _F32 or w.shape != (dim,) or not w.is_contiguous():
            raise ValueError(f"{name} must be {dim} contiguous fp32 values")
    table = cos.shape
    if (cos.dtype is not _F32 or sin.dtype is not _F32 or len(table) != 2 or table != sin.shape
            or not cos.is_contiguous() or not sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous fp32 tables of one shape [position, rotated pairs]")
    pt = positions.dtype
    if (pt is not _I32 and pt is not _I64) or positions.shape != (n,) or not positions.is_contiguous():
        raise ValueError(f"positions must be {n} contiguous int32 or int64 values")
    d = QkNormRope(n, h, g, dim, 2 * table[1], _dtype("q", q), 1 if neighbours else 0, 8 if pt is _I64 else 4, 0, eps,
                   q.data_ptr(), k.data_ptr(), q_ts, q_hs, k_ts, k_hs, q_weight.data_ptr(), k_weight.data_ptr(),
                   cos.data_ptr(), sin.data_ptr(), table[0], positions.data_ptr())
    return dev, q, k, d


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6, neighbours: bool = False):
    """RMS norm of every head of q and k, then the rotation by the token's
    position. q, k: [token, head, head_dim] fp32 or bf16 (e.g. slices of one
    projection's output); weights and tables fp32. Returns contiguous
    (q_out, k_out)."""
    dev, q, k, d = _qk(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)
    dtype, device = q.dtype, q.device
    q_out, k_out = _empty(q.shape, dtype=dtype, device=device), _empty(k.shape, dtype=dtype, device=device)
    _call(dev, load_library().muon_adamw_qk_norm_rope, d, q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def _qk_bytes(dev: int, dim: int) -> int:
    return _bytes_of(dev, load_library().muon_adamw_qk_norm_rope_backward_workspace, QkNormRope(head_dim=dim))


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, cos, sin, positions, *, eps: float = 1e-6,
                          neighbours: bool = False):
    """(dq, dk, dq_weight, dk_weight) from the outputs' gradients and the
    forward call's inputs; the weights' gradients are fp32."""
    dev, q, k, d = _qk(q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours)
    if dq_out.get_device() != dev or dk_out.get_device() != dev:
        _apart_devices(("q", "dq_out", "dk_out"), (q, dq_out, dk_out))
    dtype, device = q.dtype, q.device
    if dq_out.shape != q.shape or dk_out.shape != k.shape or dq_out.dtype is not dtype or dk_out.dtype is not dtype:
        raise ValueError("dq_out and dk_out must have the shapes and the type of q and k")
    dq_out, shape, dq_ts, dq_hs = _heads("dq_out", dq_out)
    dk_out, _, dk_ts, dk_hs = _heads("dk_out", dk_out)
    dim = shape[2]
    size = _qk_bytes(dev, dim)
    ws = _empty(size, dtype=torch.uint8, device=device)
    dq, dk = _empty(shape, dtype=dtype, device=device), _empty(k.shape, dtype=dtype, device=device)
    dw = _empty((2, dim), dtype=_F32, device=device)
    at = dw.data_ptr()
    _call(dev, load_library().muon_adamw_qk_norm_rope_backward, d, dq_out.data_ptr(), dq_ts, dq_hs, dk_out.data_ptr(),
          dk_ts, dk_hs, dq.data_ptr(), dk.data_ptr(), at, at + 4 * dim, ws.data_ptr(), size)
    dqw, dkw = dw.unbind(0)
    return dq, dk, dqw, dkw


# ---- attention ----

def _apart(name: str, t, dim: Optional[int] = None):
    """``_heads``, with no two heads on the same elements (as in an expanded tensor)."""
    r = _heads(name, t, dim)
    n, h, d = r[1]
    if (n > 1 and r[2] < d) or (h > 1 and r[3] < d):
        return _heads(name, t.contiguous(), dim)
    return r


def _attention(q, k, v, window, sinks, scale, cu_seqlens):
    dev = q.get_device()
    if dev < 0 or k.get_device() != dev or v.get_device() != dev or (
            cu_seqlens is not None and cu_seqlens.get_device() != dev):
        _apart_devices(("q", "k", "v", "cu_seqlens"), (q, k, v) if cu_seqlens is None else (q, k, v, cu_seqlens))
    q, (n, h, dim), q_ts, q_hs = _apart("q", q)
    k, ks, k_ts, k_hs = _apart("k", k, dim)
    v, vs, v_ts, v_hs = _apart("v", v, dim)
    if ks[0] != n or vs != ks:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(ks)} and v {tuple(vs)} do not fit together")
    if q.dtype is not _BF16 or k.dtype is not _BF16 or v.dtype is not _BF16:
        raise TypeError("q, k and v must be bf16")
    n_seqs, cu = 0, None
    if cu_seqlens is not None:
        n_seqs, cu = cu_seqlens.numel() - 1, cu_seqlens.data_ptr()
        if cu_seqlens.dtype is not _I32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() or n_seqs < 1:
            raise ValueError("cu_seqlens must be at least 2 contiguous int32 values")
    g, sinks = ks[1], int(sinks)
    d = WindowAttention(n, h, g, dim, sinks, n if window is None else window,
                        1.0 / math.sqrt(dim) if scale is None else scale, cu, n_seqs, 0, q.data_ptr(), k.data_ptr(),
                        v.data_ptr(), q_ts, q_hs, k_ts, k_hs, v_ts, v_hs)
    return dev, q, k, v, d, (n, h, g, dim, sinks, n_seqs)


def window_attention(q, k, v, *, window: Optional[int], sinks: int = 0, scale: Optional[float] = None,
                     cu_seqlens=None):
    """Causal attention of packed samples: a query sees the `window` last keys
    of its sample (itself among them; None: all) and the sample's first
    `sinks` keys. q: [token, head, head_dim] bf16; k, v: [token, kv head,
    head_dim]; cu_seqlens: int32 bounds of the samples on the GPU (None: one
    sample); scale: 1 / sqrt(head_dim) by default. Returns (out, lse): out like
    q, lse [head, token] fp32."""
    dev, q, k, v, d, size = _attention(q, k, v, window, sinks, scale, cu_seqlens)
    out = _empty(q.shape, dtype=_BF16, device=q.device)
    lse = _empty((size[1], size[0]), dtype=_F32, device=q.device)
    _call(dev, load_library().muon_adamw_window_attention, d, out.data_ptr(), lse.data_ptr())
    return out, lse


@functools.lru_cache(maxsize=1024)
def _attention_bytes(dev: int, n: int, h: int, g: int, dim: int, sinks: int, n_seqs: int) -> int:
    at = 256  # any address will do: the size depends on the counts alone
    d = WindowAttention(n, h, g, dim, sinks, 0, 1.0, at if n_seqs else None, n_seqs, 0, at, at, at,
                        h * dim, dim, g * dim, dim, g * dim, dim)
    return _bytes_of(dev, load_library().muon_adamw_window_attention_backward_workspace, d)


def window_attention_backward(dout, q, k, v, out, lse, *, window: Optional[int], sinks: int = 0,
                              scale: Optional[float] = None, cu_seqlens=None):
    """(dq, dk, dv) from the output's gradient, the forward call's inputs and
    what it returned."""
    dev, q, k, v, d, size = _attention(q, k, v, window, sinks, scale, cu_seqlens)
    if dout.get_device() != dev or out.get_device() != dev or lse.get_device() != dev:
        _apart_devices(("q", "dout", "out", "lse"), (q, dout, out, lse))
    shape, device = q.shape, q.device
    if dout.shape != shape or out.shape != shape or dout.dtype is not _BF16 or out.dtype is not _BF16:
        raise ValueError("dout and out must have the shape and the type of q")
    if lse.shape != (size[1], size[0]) or lse.dtype is not _F32 or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [head, token]")
    dout, _, do_ts, do_hs = _apart("dout", dout)
    if not out.is_contiguous():
        out = out.contiguous()
    need = _attention_bytes(dev, *size)
    ws = _empty(need, dtype=torch.uint8, device=device)
    dq, dk, dv = (_empty(shape, dtype=_BF16, device=device), _empty(k.shape, dtype=_BF16, device=device),
                  _empty(k.shape, dtype=_BF16, device=device))
    _call(dev, load_library().muon_adamw_window_attention_backward, d, dout.data_ptr(), do_ts, do_hs, out.data_ptr(),
          lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), need)
    return dq, dk, dv


def check() -> None:
    """Wait for the current stream; raises if a bounded wait of an operator's
    kernel has run out (a fault of the machine or of the library)."""
    torch.cuda.init()
    _check(load_library().muon_adamw_operators_check(_stream(_device_now())))


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
