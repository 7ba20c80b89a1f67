"""The operators past a warp's first unit, a CTA's first item and 2^31 elements.

Definitions in 64 bits, and element-wise bounds of an fp32 computation, as in
``oracle/operators.py``; the attention's are written here once more over whole
matrices, for samples of thousands of tokens, and held against the oracle's.
"""
import numpy as np
import pytest

from oracle import operators as O

torch = pytest.importorskip("torch")

TINY = 1e-30  # absolute slack for results that are zero
DTYPES = {"fp32": (torch.float32, O.U32), "bf16": (torch.bfloat16, O.UB)}


@pytest.fixture(scope="module")
def ops():
    from muon_adamw_hybrid_grad_gb300 import build

    build.build()
    from muon_adamw_hybrid_grad_gb300 import ops as m

    yield m
    torch.cuda.empty_cache()


def within(got, want, bound, unit):
    """|got - want| <= bound, plus one rounding of a value up to |want| + bound to the result's type."""
    got = got.double()
    want, bound = (torch.as_tensor(x, device=got.device) for x in (want, bound))
    assert got.shape == want.shape and bool(got.isfinite().all())
    over = (got - want).abs() - (bound + unit * (want.abs() + bound) + TINY)
    assert float(over.max()) <= 0, (int((over > 0).sum()), float(over.max()))


def normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32).to(dtype)


# ---- norm and rotation: many units to a warp ----

# 2 * 8 warps an SM (2368 to 2432 on the GPU): 4.9 units to a warp; tokens of two and four units, four and eight to a
# warp; and one unit to most warps and a second to a few
QK = [(12001, 2, 1, 64, 64), (5003, 40, 8, 128, 128), (2500, 3, 2, 80, 48)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,g,d,rot", QK)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("fused", [False, True])
def test_qk_norm_rope_of_many_tokens(ops, n, h, g, d, rot, dt, fused):
    dtype, unit = DTYPES[dt]
    gen = torch.Generator(device="cuda").manual_seed(n + d)
    if fused:
        qkv = normal(gen, n, h + 2 * g, d, dtype=dtype)
        q, k = qkv[:, :h], qkv[:, h:h + g]
    else:
        q, k = normal(gen, n, h, d, dtype=dtype), normal(gen, g, n, d, dtype=dtype).transpose(0, 1)
    qw, kw = (1 + 0.3 * normal(gen, d, dtype=torch.float32) for _ in range(2))
    angle = 3 * normal(gen, 512, rot // 2, dtype=torch.float32)
    cos, sin = angle.cos(), angle.sin()
    pos = torch.randint(0, 512, (n,), generator=gen, device="cuda")
    outs = ops.qk_norm_rope(q, k, qw, kw, cos, sin, pos, eps=1e-5)
    dqo, dko = normal(gen, n, h, d, dtype=dtype), normal(gen, n, g, d, dtype=dtype)
    dq, dk, dqw, dkw = ops.qk_norm_rope_backward(dqo, dko, q, k, qw, kw, cos, sin, pos, eps=1e-5)
    host = lambda x: x.double().cpu().numpy()  # noqa: E731
    cs, sn = host(cos[pos]), host(sin[pos])
    for x, w, y, dy, dx, dw in ((q, qw, outs[0], dqo, dq, dqw), (k, kw, outs[1], dko, dk, dkw)):
        within(y, *O.norm_rope(host(x), host(w), cs, sn, 1e-5, False), unit)
        wx, ww, bx, bw = O.norm_rope_backward(host(dy), host(x), host(w), cs, sn, 1e-5, False)
        within(dx, wx, bx, unit)
        within(dw, ww, bw, O.U32)


# ---- attention: many items to a CTA, long samples ----

def attention(q, k, v, do, window, sinks, scale):
    """One sample in fp64 over whole matrices: (out, lse, dq, dk, dv) and their bounds, as the oracle's."""
    q, k, v, do = (x.double() for x in (q, k, v, do))
    n, heads, d = q.shape
    per = heads // k.shape[1]
    at = torch.arange(n, device=q.device)
    back = at[:, None] - at[None]
    see = (back >= 0) & ((back < window) | (at[None] < sinks))
    seen = see.sum(1, keepdim=True)
    res = [torch.zeros_like(q), q.new_zeros(heads, n), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]
    bnd = [torch.zeros_like(x) for x in res]
    for h in range(heads):
        g = h // per
        qq, kk, vv, dd = q[:, h], k[:, g], v[:, g], do[:, h]
        s = (scale * qq @ kk.T).masked_fill_(~see, -np.inf)
        lse = torch.logsumexp(s, 1, keepdim=True)
        p = torch.exp(s - lse)
        mag = (abs(scale) * qq.abs() @ kk.abs().T).masked_fill_(~see, 0)
        res[0][:, h], res[1][h] = p @ vv, lse[:, 0]
        ds = (d + 8) * O.U32 * mag.amax(1, keepdim=True) + 2.0 ** -20
        bnd[1][h] = (2 * ds + seen * O.U32 + 4 * O.U32 * lse.abs())[:, 0]
        bnd[0][:, h] = (O.UB + 2 * (2 * ds + (seen + 16) * O.U32)) * (p @ vv.abs())
        dp = dd @ vv.T
        dsc = p * (dp - (p * dp).sum(1, keepdim=True))
        es = (d + 8) * O.U32 * mag
        ep = 2 * es + 2 * es.amax(1, keepdim=True) + 2.0 ** -19 + (n + 16) * O.U32
        ed = (d + 8) * O.U32 * dd.abs() @ vv.abs().T + (
            dd.abs() * (bnd[0][:, h] + (1 + O.UB) * O.UB * res[0][:, h].abs() + (d + 8) * O.U32 * res[0][:, h].abs())
        ).sum(1, keepdim=True)
        eds = (O.UB + ep) * dsc.abs() + (1 + O.UB) * p * ed
        m = (n * per + 16) * O.U32
        res[2][:, h] += scale * dsc @ kk
        res[3][:, g] += scale * dsc.T @ qq
        res[4][:, g] += p.T @ dd
        bnd[2][:, h] += abs(scale) * (eds + m * dsc.abs()) @ kk.abs()
        bnd[3][:, g] += abs(scale) * (eds + m * dsc.abs()).T @ qq.abs()
        bnd[4][:, g] += ((O.UB + ep + m) * p).T @ dd.abs()
    return res, bnd


@pytest.mark.parametrize("window,sinks", [(7, 3), (40, 0), (1, 1)])
def test_whole_matrices_agree_with_the_oracle(window, sinks):
    gen = torch.Generator().manual_seed(5)
    q, k, v, do = (normal(gen, 40, x, 8, dtype=torch.float64) for x in (4, 2, 2, 4))
    res, bnd = attention(q, k, v, do, window, sinks, 0.4)
    see = O.visible(40, [40], window, sinks)
    x = [y.numpy() for y in (q, k, v, do)]
    out, lse, bo, bl = O.window_attention(*x[:3], see, 0.4)
    grads, bounds = O.window_attention_backward(x[3], *x[:3], see, 0.4)
    for got, want in zip((*res, *bnd), (out, lse, *grads, bo, bl, *bounds)):
        assert np.abs(got.numpy() - want).max() <= 1e-12 * (1 + np.abs(want).max())


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,g,d,window,sinks", [
    (6001, 2, 1, 128, None, 0), (5121, 2, 2, 64, 1024, 4), (4999, 4, 1, 96, 700, 128), (6144, 1, 1, 64, None, 0)])
def test_window_attention_of_a_long_sample(ops, n, h, g, d, window, sinks):
    gen = torch.Generator(device="cuda").manual_seed(n)
    q, k, v, do = (normal(gen, n, x, d) for x in (h, g, g, h))
    how = {"window": window, "sinks": sinks}
    out, lse = ops.window_attention(q, k, v, **how)
    grads = ops.window_attention_backward(do, q, k, v, out, lse, **how)
    res, bnd = attention(q, k, v, do, n if window is None else window, sinks, 1 / np.sqrt(d))
    for i, x in enumerate((out, lse, *grads)):
        within(x, res[i], bnd[i], O.U32 if i == 1 else O.UB)
    ops.check()


LENGTHS = [513, 250, 1021, 64, 7, 700, 1, 128, 900, 333, 1500, 129, 2, 640, 255, 1100]


@pytest.mark.gpu
@pytest.mark.parametrize("h,g,d,window,sinks", [
    (16, 16, 64, 256, 8), (16, 8, 128, 256, 8), (16, 8, 128, None, 0), (12, 4, 96, 100, 1), (16, 16, 64, 0, 3)])
def test_packed_samples_are_what_each_is_alone(ops, h, g, d, window, sinks):
    """Many items of many samples to a CTA: every sample's outputs and gradients are those of a call of its own."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    n = sum(LENGTHS)
    q, k, v, do = (normal(gen, n, x, d) for x in (h, g, g, h))
    how = {"window": window, "sinks": sinks}
    cu = torch.tensor(np.cumsum([0] + LENGTHS), dtype=torch.int32, device="cuda")
    out, lse = ops.window_attention(q, k, v, cu_seqlens=cu, **how)
    grads = ops.window_attention_backward(do, q, k, v, out, lse, cu_seqlens=cu, **how)
    at = 0
    for m in LENGTHS:
        x = [t[at:at + m] for t in (q, k, v, do)]
        o, l = ops.window_attention(*x[:3], **how)
        assert torch.equal(o, out[at:at + m]) and torch.equal(l, lse[:, at:at + m])
        one = ops.window_attention_backward(x[3], *x[:3], o, l, **how)
        assert all(torch.equal(a, b[at:at + m]) for a, b in zip(one, grads))
        at += m
    ops.check()


# ---- offsets past 2^31 elements ----

@pytest.mark.gpu
def test_embedding_past_2_31_elements(ops):
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows, width = 1_100_000, 2048
    assert rows * width > 2 ** 31
    w = torch.randn(rows, width, generator=gen, device="cuda", dtype=torch.bfloat16)
    ids = torch.randperm(rows, generator=gen, device="cuda")
    out = ops.embedding(w, ids)
    for i in range(0, rows, 100_000):
        assert torch.equal(out[i:i + 100_000], w[ids[i:i + 100_000]])
    # every row once: the gradient puts the rows back
    grad = ops.embedding_backward(out, ids, torch.empty_like(w))
    assert torch.equal(grad, w)
    del out, w, grad
    # one launch for few tokens, into a strided buffer
    base = torch.full((600_000, 4096), 7.0, dtype=torch.bfloat16, device="cuda")
    grad = base[:, :width]
    few = torch.tensor([599_999, 5, 599_998], device="cuda")
    d = torch.randn(3, width, generator=gen, device="cuda", dtype=torch.bfloat16)
    ops.embedding_backward(d, few, grad)
    assert torch.equal(grad[few], d) and int(grad.any(1).sum()) == 3
    assert bool((base[:, width:] == 7).all())


@pytest.mark.gpu
def test_qk_norm_rope_past_2_31_elements(ops):
    gen = torch.Generator(device="cuda").manual_seed(2)
    n, tail, d = 1_100_000, 700, 128
    q, dq = (torch.randn(n, 16, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    assert q.numel() > 2 ** 31
    k, dk = (torch.randn(n, 1, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    w = 1 + 0.1 * normal(gen, d, dtype=torch.float32)
    angle = normal(gen, 4096, d // 2, dtype=torch.float32)
    pos = torch.arange(n, device="cuda") % 4096
    rest = (w, w, angle.cos(), angle.sin())
    outs = ops.qk_norm_rope(q, k, *rest, pos)
    grads = ops.qk_norm_rope_backward(dq, dk, q, k, *rest, pos)
    one = ops.qk_norm_rope(q[-tail:], k[-tail:], *rest, pos[-tail:])
    assert all(torch.equal(a[-tail:], b) for a, b in zip(outs, one))
    one = ops.qk_norm_rope_backward(dq[-tail:], dk[-tail:], q[-tail:], k[-tail:], *rest, pos[-tail:])
    assert all(torch.equal(a[-tail:], b) for a, b in zip(grads[:2], one))


@pytest.mark.gpu
def test_window_attention_past_2_31_elements(ops):
    gen = torch.Generator(device="cuda").manual_seed(3)
    lengths, heads, d = [66_000, 700], 256, 128
    n = sum(lengths)
    q, k, v, do = (torch.randn(n, heads, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    assert lengths[0] * heads * d > 2 ** 31
    how = {"window": 64, "sinks": 2}
    cu = torch.tensor([0, lengths[0], n], dtype=torch.int32, device="cuda")
    out, lse = ops.window_attention(q, k, v, cu_seqlens=cu, **how)
    grads = ops.window_attention_backward(do, q, k, v, out, lse, cu_seqlens=cu, **how)
    x = [t[-lengths[1]:] for t in (q, k, v, do)]
    o, l = ops.window_attention(*x[:3], **how)
    assert torch.equal(o, out[-lengths[1]:]) and torch.equal(l, lse[:, -lengths[1]:])
    one = ops.window_attention_backward(x[3], *x[:3], o, l, **how)
    assert all(torch.equal(a, b[-lengths[1]:]) for a, b in zip(one, grads))
    ops.check()
