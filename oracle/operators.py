"""fp64 definitions of the training step's operators (test infrastructure).

The embedding lookup, the norm and rotation of queries and keys, and causal
attention with a sliding window and sinks, each with its gradient, step by
step in numpy. Each gradient is pinned to differences of its forward
definition. The ``*_bound`` results say how far a computation may lie from the
exact one, element by element, when it

  * holds sums and statistics in fp32 (unit roundoff U32 = 2^-24), a sum of n
    terms being off by at most about n U32 times the sum of their magnitudes;
  * rounds softmax weights and score gradients to bf16 (UB = 2^-8) before they
    enter a product, as tensor cores want them;
  * rounds its results once to their type.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24
UB = 2.0 ** -8


def embedding(weight, ids, scale):
    out = np.zeros((len(ids), weight.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < len(weight):
            out[t] = scale * weight[i]
    return out


def embedding_backward(dout, ids, vocab, scale):
    """(grad, sum of the terms' magnitudes, number of terms of each row)."""
    grad, mag, count = (np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1])), np.zeros((vocab, 1)))
    for t, i in enumerate(ids):
        if 0 <= i < vocab:
            grad[i] += scale * dout[t]
            mag[i] += abs(scale) * np.abs(dout[t])
            count[i] += 1
    return grad, mag, count


def _pairs(rot, neighbours):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)


def norm_rope(x, w, cos, sin, eps, neighbours):
    """x [token, head, D], cos/sin [token, rot / 2] -> (y, bound of an fp32 computation's error)."""
    d, rot = x.shape[-1], 2 * cos.shape[-1]
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    z = x * r * w
    y, mag = z.copy(), np.abs(z)
    a, b = _pairs(rot, neighbours)
    c, s = cos[:, None], sin[:, None]
    y[..., a] = z[..., a] * c - z[..., b] * s
    y[..., b] = z[..., b] * c + z[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(z[..., a]) + np.abs(z[..., b])
    return y, (d + 16) * U32 * mag


def norm_rope_backward(dy, x, w, cos, sin, eps, neighbours):
    """(dx, dw, bound of dx, bound of dw)."""
    d, rot = x.shape[-1], 2 * cos.shape[-1]
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    z = x * r
    dn, mag = dy.copy(), np.abs(dy)
    a, b = _pairs(rot, neighbours)
    c, s = cos[:, None], sin[:, None]
    dn[..., a] = dy[..., a] * c + dy[..., b] * s
    dn[..., b] = dy[..., b] * c - dy[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(dy[..., a]) + np.abs(dy[..., b])
    g = dn * w
    dx = r * (g - z * np.mean(g * z, -1, keepdims=True))
    gm = mag * np.abs(w)
    bx = (2 * d + 32) * U32 * r * (gm + np.abs(z) * np.mean(gm * np.abs(z), -1, keepdims=True))
    bw = (x.shape[0] * x.shape[1] + d + 32) * U32 * (mag * np.abs(z)).sum((0, 1))
    return dx, (dn * z).sum((0, 1)), bx, bw


def visible(n, lengths, window, sinks):
    """[query, key] truth values; tokens behind the last sample see nothing."""
    see = np.zeros((n, n), bool)
    at = 0
    for m in lengths:
        for i in range(m):
            for j in range(i + 1):
                see[at + i, at + j] = i - j < window or j < sinks
        at += m
    return see


def window_attention(q, k, v, see, scale):
    """q [token, head, D], k and v [token, kv head, D] -> out, lse [head, token], and bounds of both."""
    n, heads, d = q.shape
    out, lse = np.zeros(q.shape), np.full((heads, n), -np.inf)
    bo, bl = np.zeros(q.shape), np.zeros((heads, n))
    per = heads // k.shape[1]
    for h in range(heads):
        kk, vv = k[:, h // per], v[:, h // per]
        for i in range(n):
            j = np.flatnonzero(see[i])
            if not len(j):
                continue
            s = scale * kk[j] @ q[i, h]
            top = s.max()
            p = np.exp(s - top)
            total = p.sum()
            p /= total
            lse[h, i] = top + np.log(total)
            out[i, h] = p @ vv[j]
            ds = (d + 8) * U32 * (abs(scale) * np.abs(kk[j]) @ np.abs(q[i, h])).max() + 2.0 ** -20
            bl[h, i] = 2 * ds + len(j) * U32 + 4 * U32 * abs(lse[h, i])
            bo[i, h] = (UB + 2 * (2 * ds + (len(j) + 16) * U32)) * (p @ np.abs(vv[j]))
    return out, lse, bo, bl


def window_attention_backward(dout, q, k, v, see, scale):
    """((dq, dk, dv), bounds of the three). The bounds hold for a computation
    that takes delta_i = dout_i . out_i from an out rounded to bf16."""
    n, heads, d = q.shape
    per = heads // k.shape[1]
    grads = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    bounds = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    out, _, bo, _ = window_attention(q, k, v, see, scale)
    for h in range(heads):
        g = h // per
        kk, vv, qq, dd = k[:, g], v[:, g], q[:, h], dout[:, h]
        s = np.where(see, scale * qq @ kk.T, -np.inf)
        rows = see.any(1)
        p = np.zeros((n, n))
        p[rows] = np.exp(s[rows] - s[rows].max(1, keepdims=True))
        p[rows] /= p[rows].sum(1, keepdims=True)
        dp = dd @ vv.T
        delta = (p * dp).sum(1, keepdims=True)
        ds = p * (dp - delta)
        # relative error of a softmax weight from its score and from lse
        es = np.where(see, (d + 8) * U32 * abs(scale) * np.abs(qq) @ np.abs(kk).T, 0)
        ep = (2 * es + 2 * es.max(1, keepdims=True) + 2.0 ** -19 + (n + 16) * U32)
        # dp is a sum of D terms; delta takes an out that is off by its own bound and its rounding
        ed = (d + 8) * U32 * np.abs(dd) @ np.abs(vv).T + (
            np.abs(dd) * (bo[:, h] + (1 + UB) * UB * np.abs(out[:, h]) + (d + 8) * U32 * np.abs(out[:, h]))
        ).sum(1, keepdims=True)
        eds = (UB + ep) * np.abs(ds) + (1 + UB) * p * ed
        grads[0][:, h] += scale * ds @ kk
        grads[1][:, g] += scale * ds.T @ qq
        grads[2][:, g] += p.T @ dd
        m = (n * per + 16) * U32
        bounds[0][:, h] += abs(scale) * (eds + m * np.abs(ds)) @ np.abs(kk)
        bounds[1][:, g] += abs(scale) * (eds + m * np.abs(ds)).T @ np.abs(qq)
        bounds[2][:, g] += ((UB + ep + m) * p).T @ np.abs(dd)
    return tuple(grads), tuple(bounds)
