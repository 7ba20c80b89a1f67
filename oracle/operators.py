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


# ---- dropout, residual and norm, products grouped by expert, log probabilities ----

def philox(counter, key):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): counter [..., 4] and key [2] of 32-bit words -> [..., 4]."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), q & low, (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def dropout_factors(n, p, seed, step, site, first=0):
    """The factors of elements `first` to `first` + n - 1 (`first` a multiple of 8): 0 or 1 / (1 - p), p in steps of 2^-16."""
    t = int(np.floor(p * 65536 + 0.5))
    group = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    counter = np.stack([group, np.full_like(group, site), np.full_like(group, step & 0xFFFFFFFF),
                        np.full_like(group, step >> 32 & 0xFFFFFFFF)], -1)
    words = philox(counter, (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF))
    bits = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], -1).reshape(-1)[:n]
    return np.where(bits >= t, 65536 / max(65536 - t, 1), 0.0)


def residual_norm(x, residual, w, eps, factors):
    """x, residual [row, width] -> (y, r, bounds of both in an fp32 computation)."""
    d = x.shape[-1]
    drop = np.where(factors == 0, 0, x) * factors
    r = residual + drop
    er = 3 * U32 * (np.abs(residual) + np.abs(drop))
    sq = np.sum(r * r, -1, keepdims=True)
    rstd = 1 / np.sqrt(sq / d + eps)
    # relative error of rstd: that of the sum, and of a reciprocal root good to two steps
    e = np.sum(np.abs(r) * er, -1, keepdims=True) / np.maximum(sq, 1e-300) + (d / 2 + 16) * U32
    y = r * rstd * w
    return y, r, e * np.abs(y) + er * rstd * np.abs(w), er


def residual_norm_backward(dy, dres, r, w, eps, factors):
    """(dx, dresidual, dw) and their bounds."""
    n, d = r.shape
    rstd = 1 / np.sqrt(np.mean(r * r, -1, keepdims=True) + eps)
    e = (d / 2 + 16) * U32
    g = dy * w
    c = np.mean(g * r, -1, keepdims=True) * rstd ** 3
    ec = (d + 16) * U32 * np.mean(np.abs(g * r), -1, keepdims=True) * rstd ** 3 + 3 * e * np.abs(c)
    dr = dres + rstd * g - c * r
    er = 6 * U32 * (np.abs(dres) + np.abs(rstd * g) + np.abs(c * r)) + e * np.abs(rstd * g) + ec * np.abs(r)
    terms = dy * r * rstd
    dx = np.where(factors == 0, 0, dr) * factors
    ex = factors * er + 2 * U32 * np.abs(dx)
    return (dx, dr, terms.sum(0)), (ex, er, ((n + 16) * U32 + e) * np.abs(terms).sum(0))


E4M3_UNIT, E4M3_TINY = 2.0 ** -4, 2.0 ** -10  # half a step, relative for normal numbers and absolute below them


def expert_matmul(x, w, offsets):
    """(out, sum of the terms' magnitudes): tokens offsets[e] to offsets[e + 1] - 1 by w[e]."""
    out, mag = np.zeros((len(x), w.shape[1])), np.zeros((len(x), w.shape[1]))
    for e in range(len(w)):
        rows = slice(offsets[e], offsets[e + 1])
        out[rows], mag[rows] = x[rows] @ w[e].T, np.abs(x[rows]) @ np.abs(w[e]).T
    return out, mag


def expert_matmul_backward(dout, x, w, offsets):
    """((dx, dw), (magnitudes of both))."""
    dx, dw = np.zeros(x.shape), np.zeros(w.shape)
    mx, mw = np.zeros(x.shape), np.zeros(w.shape)
    for e in range(len(w)):
        rows = slice(offsets[e], offsets[e + 1])
        dx[rows], mx[rows] = dout[rows] @ w[e], np.abs(dout[rows]) @ np.abs(w[e])
        dw[e], mw[e] = dout[rows].T @ x[rows], np.abs(dout[rows]).T @ np.abs(x[rows])
    return (dx, dw), (mx, mw)


EX2 = 2.0 ** -22  # relative error of the hardware's power of two


def token_logprobs(z, ids, scale, top):
    """z [row, vocab] -> (logprobs, entropy, lse, top_logprobs, top_ids) and bounds of the four numbers in an fp32
    computation relative to each row's maximum. Rows of -infinity alone have lse and log probabilities -infinity."""
    n, v = z.shape
    m = z.max(-1, keepdims=True)
    empty = m[:, 0] == -np.inf
    with np.errstate(invalid="ignore", divide="ignore"):
        a = np.where(z == -np.inf, 0, (z - m) * scale)
        p = np.where(z == -np.inf, 0.0, np.exp(a))
    p[empty] = 0
    a[empty] = 0
    s = np.where(empty, 1, p.sum(-1))
    p /= s[:, None]
    inside = (ids >= 0) & (ids < v)
    given = z[np.arange(n), np.where(inside, ids, 0)]
    logs = np.log(s)
    # an exponent is off by 4 roundings of itself; sums of v / 512 terms a thread, their joins, and new maxima
    ee = 4 * U32 * np.abs(a) + EX2
    es = (p * ee).sum(-1) + (v / 512 + 64) * U32 + (v / 8192 + 16) * 2 * EX2
    mean = (p * a).sum(-1)
    eu = (p * np.abs(a) * (ee + 4 * U32)).sum(-1) + np.abs(mean) * ((v / 512 + 64) * U32 + (v / 8192 + 16) * 2 * EX2)
    entropy = np.where(empty, 0, logs - mean)
    with np.errstate(invalid="ignore"):
        lse = np.where(empty, -np.inf, m[:, 0] * scale + logs)
        lp = np.where(inside, np.where(empty, -np.inf, (given - m[:, 0]) * scale - logs), 0)
        order = np.argsort(-z, axis=-1, kind="stable")[:, :top]
        tops = np.take_along_axis(z, order, -1)
        tl = np.where(empty[:, None], -np.inf, (tops - m) * scale - logs[:, None])
    common = es + 2 * U32 * np.abs(logs)
    finite = lambda x: np.where(np.isfinite(x), np.abs(x), 0)  # noqa: E731
    bounds = (common + 6 * U32 * (finite(lp) + logs), common + eu + es * np.abs(mean) + 4 * U32 * np.abs(mean),
              common + 2 * U32 * finite(m[:, 0] * scale), common[:, None] + 6 * U32 * (finite(tl) + logs[:, None]))
    return (lp, entropy, lse, tl, order), bounds


def token_logprobs_backward(dlp, dh, z, ids, entropy, lse, scale):
    """(dlogits, bound), from the row's entropy and lse as they are given. Rows with lse -infinity get zeros."""
    n, v = z.shape
    empty = lse == -np.inf
    shift = np.where(empty, 0, lse)[:, None] / scale
    hidden = (z == -np.inf) | empty[:, None]
    logp = np.where(hidden, 0, (np.where(hidden, 0, z) - shift) * scale)
    p = np.where(hidden, 0, np.exp(logp))
    inside = (ids >= 0) & (ids < v) & ~empty
    l, h = np.where(inside, dlp, 0)[:, None], dh[:, None]
    d = -scale * p * (l + h * (logp + entropy[:, None]))
    mag = scale * p * (np.abs(l) + np.abs(h * logp) + np.abs(h * entropy[:, None]))
    one = np.zeros_like(z)
    one[np.arange(n)[inside], ids[inside]] = scale * dlp[inside]
    ea = 4 * U32 * np.abs(logp) + 2 * U32 * np.abs(shift) * scale
    return d + one, mag * (ea + EX2 + 8 * U32) + scale * p * np.abs(h) * ea + 2 * U32 * np.abs(one)
