"""The training step's operators on the GPU against their fp64 definitions.

Tolerances are element by element and come from the arithmetic alone
(``oracle/operators.py``): the operators' fp32 sums, the bf16 rounding of
softmax weights and score gradients before a product, and one rounding of each
result to its type (UB = 2^-8 relative for bf16, U32 = 2^-24 for fp32).
"""
import numpy as np
import pytest

from oracle import operators as O

pytestmark = pytest.mark.gpu

TINY = 1e-30  # absolute slack for results that are zero


@pytest.fixture(scope="module")
def ops():
    from muon_adamw_hybrid_grad_gb300 import build

    build.build()
    from muon_adamw_hybrid_grad_gb300 import ops as m

    return m


def t_dtype(name):
    import torch

    return {"fp32": torch.float32, "bf16": torch.bfloat16}[name]


def unit(name):
    return O.UB if name == "bf16" else O.U32


def cuda(x, dtype):
    import torch

    return torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda").to(t_dtype(dtype))


def host(x):
    return x.double().cpu().numpy()


def within(got, want, bound, dtype):
    """|got - want| <= bound, plus one rounding of a value up to |want| + bound to the result's type."""
    got = host(got)
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    err, lim = np.abs(got - want), bound + unit(dtype) * (np.abs(want) + bound) + TINY
    bad = err > lim
    assert not bad.any(), (int(bad.sum()), float((err / lim).max()), np.argwhere(bad)[:3].tolist())


def signal(rng, *shape):
    return rng.normal(size=shape)


# ---- embedding ----

EMBED = [(1, 1, 1), (7, 3, 1), (61, 1000, 256), (130, 50, 24), (33, 9, 20), (1000, 17, 264), (5, 300, 2056), (300, 70, 77)]


@pytest.mark.parametrize("tokens,vocab,width", EMBED)
@pytest.mark.parametrize("wt,ot", [("fp32", "bf16"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
def test_embedding(ops, tokens, vocab, width, wt, ot):
    import torch

    rng = np.random.default_rng(tokens + width)
    w = cuda(signal(rng, vocab, width), wt)
    ids = torch.tensor(rng.integers(-2, vocab + 2, tokens), device="cuda")
    for i in (ids, ids.to(torch.int32)):
        got = ops.embedding(w, i, scale=1.7, dtype=t_dtype(ot))
        want = O.embedding(host(w), ids.tolist(), 1.7)
        within(got, want, 3 * O.U32 * np.abs(want), ot)
        assert got.dtype == t_dtype(ot)


@pytest.mark.parametrize("tokens,vocab,width", EMBED)
@pytest.mark.parametrize("dt,gt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_backward(ops, tokens, vocab, width, dt, gt, accumulate):
    import torch

    rng = np.random.default_rng(tokens * 3 + width)
    d = cuda(signal(rng, tokens, width), dt)
    ids = torch.tensor(rng.integers(-2, vocab + 2, tokens), device="cuda")
    before = cuda(signal(rng, vocab, width), gt)
    got = ops.embedding_backward(d, ids, before.clone(), scale=0.7, accumulate=accumulate)
    want, mag, count = O.embedding_backward(host(d), ids.tolist(), vocab, 0.7)
    if accumulate:
        want, mag = want + host(before), mag + np.abs(host(before))
        untouched = count[:, 0] == 0
        assert torch.equal(got[torch.tensor(untouched)], before[torch.tensor(untouched)])
    within(got, want, (count + 4) * O.U32 * mag, gt)


@pytest.mark.parametrize("tokens,vocab,width", [(4500, 40, 264), (4099, 6000, 77), (9000, 3, 16), (4321, 30000, 2056)])
@pytest.mark.parametrize("dt,gt", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_backward_of_many_tokens(ops, tokens, vocab, width, dt, gt, accumulate):
    """Past the one-launch form: sorted tokens, runs within and over the groups."""
    test_embedding_backward(ops, tokens, vocab, width, dt, gt, accumulate)


@pytest.mark.parametrize("n", [777, 4096, 4097])
@pytest.mark.parametrize("ids", ["one", "two", "none", "runs", "sorted", "reversed"])
@pytest.mark.parametrize("vocab", [3, 513, 262145])
def test_embedding_backward_orders(ops, ids, vocab, n):
    """Heavy tokens, runs over many groups, and vocabularies of one to three digits."""
    import torch

    rng = np.random.default_rng(vocab)
    v = {"one": np.full(n, vocab - 1), "two": np.where(np.arange(n) % 2, 0, vocab - 1), "none": np.full(n, -1),
         "runs": np.repeat(rng.integers(0, vocab, n // 100 + 1), 100)[:n],
         "sorted": np.sort(rng.integers(0, vocab, n)), "reversed": np.sort(rng.integers(0, vocab, n))[::-1].copy()}[ids]
    d = cuda(signal(rng, n, 8), "fp32")
    grad = torch.full((vocab, 8), float("nan"), device="cuda")
    got = ops.embedding_backward(d, torch.tensor(v, device="cuda"), grad)
    assert got is grad
    rows = sorted(set(int(x) for x in v if x >= 0))
    where = {r: i for i, r in enumerate(rows)}
    want, mag, count = O.embedding_backward(host(d), [where.get(int(x), -1) for x in v], max(1, len(rows)), 1.0)
    within(got[torch.tensor(rows, dtype=torch.int64)], want[:len(rows)], ((count + 4) * O.U32 * mag)[:len(rows)], "fp32")
    rest = torch.ones(vocab, dtype=torch.bool, device="cuda")
    rest[torch.tensor(rows, dtype=torch.int64)] = False
    assert not got[rest].any()
    again = ops.embedding_backward(d, torch.tensor(v, device="cuda"), torch.empty_like(grad))
    assert torch.equal(got, again)


def test_embedding_strides_and_empty(ops):
    import torch

    rng = np.random.default_rng(5)
    table = cuda(signal(rng, 40, 48), "bf16")
    ids = torch.tensor(rng.integers(0, 40, (3, 7)), device="cuda")
    for part in (table[:, 8:40], table[:, 3:40], table[::2, :16]):
        keep = ids % part.shape[0]
        got = ops.embedding(part, keep, dtype=torch.float32)
        assert got.shape == (3, 7, part.shape[1])
        assert torch.equal(got, part.float()[keep])
    base = torch.full((40, 48), 7.0, device="cuda")
    d = cuda(signal(rng, 3, 7, 32), "bf16")
    ops.embedding_backward(d, ids, base[:, 8:40])
    assert (base[:, :8] == 7).all() and (base[:, 40:] == 7).all()
    want, mag, count = O.embedding_backward(host(d).reshape(21, 32), ids.flatten().tolist(), 40, 1.0)
    within(base[:, 8:40], want, (count + 4) * O.U32 * mag, "fp32")
    # the same gradient from rows that are strided and not on 16-byte boundaries
    wide = cuda(signal(rng, 21, 70), "fp32")
    got = ops.embedding_backward(wide[:, 5:66], ids.flatten(), torch.empty(40, 61, device="cuda"))
    want, mag, count = O.embedding_backward(host(wide)[:, 5:66], ids.flatten().tolist(), 40, 1.0)
    within(got, want, (count + 4) * O.U32 * mag, "fp32")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert ops.embedding(table, none).shape == (0, 48)
    full = torch.full((40, 48), 3.0, device="cuda")
    empty = torch.empty(0, 48, device="cuda")
    assert (ops.embedding_backward(empty, none, full, accumulate=True) == 3).all()
    assert (ops.embedding_backward(empty, none, full) == 0).all()


def test_embedding_keeps_other_rows_clear_of_nonfinite_ones(ops):
    import torch

    w = torch.ones(4, 16, device="cuda")
    w[2] = float("inf")
    got = ops.embedding(w, torch.tensor([1, 2, -1, 9], device="cuda"))
    assert (got[0] == 1).all() and got[1].isinf().all() and (got[2:] == 0).all()
    d = torch.ones(4, 16, device="cuda")
    d[1:3] = float("nan")
    grad = ops.embedding_backward(d, torch.tensor([1, 2, -1, 3], device="cuda"), torch.empty(4, 16, device="cuda"))
    assert (grad[0] == 0).all() and (grad[1] == 1).all() and grad[2].isnan().all() and (grad[3] == 1).all()


# ---- norm and rotation ----

QK = [  # tokens, heads, kv heads, dim, rot
    (1, 1, 1, 16, 16), (50, 16, 16, 64, 64), (3, 16, 8, 128, 128), (37, 12, 4, 80, 48), (5, 5, 5, 96, 32),
    (1300, 2, 1, 128, 128), (2, 3, 1, 256, 256), (9, 40, 1, 64, 0), (11, 1, 70, 24, 16), (4, 2, 2, 8, 0)]


def qk_case(rng, n, h, g, d, rot, dt, fused):
    import torch

    if fused:
        qkv = cuda(signal(rng, n, h + 2 * g, d) * 2, dt)
        q, k = qkv[:, :h], qkv[:, h:h + g]
    else:
        q, k = cuda(signal(rng, n, h, d) * 2, dt), cuda(signal(rng, g, n, d) * 2, dt).transpose(0, 1)
    qw, kw = cuda(1 + 0.3 * signal(rng, d), "fp32"), cuda(1 + 0.3 * signal(rng, d), "fp32")
    ang = rng.normal(size=(64, rot // 2)) * 3
    cos, sin = cuda(np.cos(ang), "fp32"), cuda(np.sin(ang), "fp32")
    pos = torch.tensor(rng.integers(0, 64, n), device="cuda")
    return q, k, qw, kw, cos, sin, pos


@pytest.mark.parametrize("n,h,g,d,rot", QK)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("neighbours,fused", [(False, True), (True, False), (False, False)])
def test_qk_norm_rope(ops, n, h, g, d, rot, dt, neighbours, fused):
    import torch

    rng = np.random.default_rng(n + h + d)
    q, k, qw, kw, cos, sin, pos = qk_case(rng, n, h, g, d, rot, dt, fused)
    args = (q, k, qw, kw, cos, sin)
    qo, ko = ops.qk_norm_rope(*args, pos, eps=1e-5, neighbours=neighbours)
    cs, sn = host(cos)[pos.cpu().numpy()], host(sin)[pos.cpu().numpy()]
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want, bound = O.norm_rope(host(x), host(w), cs, sn, 1e-5, neighbours)
        within(got, want, bound, dt)
        assert got.is_contiguous() and got.dtype == x.dtype
    for p in (pos.to(torch.int32), torch.where(pos == 0, -5, pos)):  # one before the tables reads their first row
        again = ops.qk_norm_rope(*args, p, eps=1e-5, neighbours=neighbours)
        assert torch.equal(again[0], qo) and torch.equal(again[1], ko)


@pytest.mark.parametrize("n,h,g,d,rot", QK)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("neighbours,fused", [(False, True), (True, False), (False, False)])
def test_qk_norm_rope_backward(ops, n, h, g, d, rot, dt, neighbours, fused):
    import torch

    rng = np.random.default_rng(2 * n + h + d)
    q, k, qw, kw, cos, sin, pos = qk_case(rng, n, h, g, d, rot, dt, fused)
    dqo, dko = cuda(signal(rng, n, h, d), dt), cuda(signal(rng, g, n, d), dt).transpose(0, 1)
    run = lambda: ops.qk_norm_rope_backward(dqo, dko, q, k, qw, kw, cos, sin, pos, eps=1e-5, neighbours=neighbours)  # noqa: E731
    dq, dk, dqw, dkw = run()
    cs, sn = host(cos)[pos.cpu().numpy()], host(sin)[pos.cpu().numpy()]
    for dx, dw, dy, x, w in ((dq, dqw, dqo, q, qw), (dk, dkw, dko, k, kw)):
        wx, ww, bx, bw = O.norm_rope_backward(host(dy), host(x), host(w), cs, sn, 1e-5, neighbours)
        within(dx, wx, bx, dt)
        within(dw, ww, bw, "fp32")
    for a, b in zip(run(), (dq, dk, dqw, dkw)):
        assert torch.equal(a, b)


def test_qk_gradient_against_differences(ops):
    """The fp32 kernels' own differences along a direction, for inputs and weights."""
    import torch

    rng = np.random.default_rng(8)
    q, k, qw, kw, cos, sin, pos = qk_case(rng, 33, 4, 2, 64, 32, "fp32", False)
    dqo, dko = cuda(signal(rng, 33, 4, 64), "fp32"), cuda(signal(rng, 33, 2, 64), "fp32")
    f = lambda *x: sum(float((a.double() * b.double()).sum()) for a, b in  # noqa: E731
                       zip(ops.qk_norm_rope(*x, cos, sin, pos), (dqo, dko)))
    grads = ops.qk_norm_rope_backward(dqo, dko, q, k, qw, kw, cos, sin, pos)
    x = (q, k, qw, kw)
    for i, g in enumerate(grads):
        u = cuda(signal(rng, *x[i].shape), "fp32")
        h = 2.0 ** -8
        up = f(*(y + h * u if j == i else y for j, y in enumerate(x)))
        down = f(*(y - h * u if j == i else y for j, y in enumerate(x)))
        want = float((g.double() * u.double()).sum())
        # fp32 outputs: about 1e-7 of 12 k terms of size 1 in quadrature, over 2 h; truncation h^2 / 6 of third
        # derivatives of the size of the slope along u
        assert abs((up - down) / (2 * h) - want) < 1e-2 + 1e-3 * abs(want)


def test_qk_rows_are_independent_of_nonfinite_neighbours(ops):
    import torch

    rng = np.random.default_rng(9)
    args = list(qk_case(rng, 12, 4, 2, 128, 128, "bf16", False))
    clean = ops.qk_norm_rope(*args)
    args[0] = args[0].clone()
    args[0][5, 2, 7] = float("nan")
    dirty = ops.qk_norm_rope(*args)
    assert dirty[0][5, 2].isnan().all() and torch.equal(dirty[1], clean[1])
    same = torch.ones(12, 4, dtype=torch.bool)
    same[5, 2] = False
    assert torch.equal(dirty[0][same], clean[0][same])


# ---- attention ----

ATTN = [  # lengths, tokens behind the last sample, heads, kv heads, dim, window, sinks
    ([1], 0, 1, 1, 64, 4, 0), ([2, 1, 3], 0, 2, 1, 128, 2, 1), ([50], 0, 4, 4, 64, 32, 4), ([129, 64], 3, 2, 2, 64, 64, 4),
    ([128], 0, 2, 1, 128, 128, 0), ([256, 128], 0, 4, 2, 128, 100, 16), ([300], 0, 4, 1, 80, 37, 3),
    ([511, 1, 60], 5, 3, 3, 96, 130, 128), ([700], 0, 2, 2, 128, 700, 0), ([640], 0, 2, 1, 64, 1, 1),
    ([400], 7, 2, 1, 40, 0, 5), ([90, 0, 40], 0, 2, 2, 8, 0, 0), ([385, 257], 0, 6, 2, 128, 256, 64),
    ([900], 0, 2, 1, 64, 128, 130 - 2), ([5] * 60, 0, 2, 2, 64, 3, 2), ([768], 100, 5, 5, 120, 257, 1),
    # several chunks of query tiles that only the sinks reach, in more than one sample
    ([2300, 40, 1500], 0, 2, 1, 64, 64, 6), ([1700], 20, 2, 2, 128, 40, 3)]


def attn_case(rng, lengths, behind, h, g, d):
    import torch

    n = sum(lengths) + behind
    q = signal(rng, n, h, d)
    k = signal(rng, n, g, d)
    if sum(lengths):
        k[np.cumsum([0] + lengths[:-1]).clip(max=n - 1)] *= 2
    cu = torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device="cuda")
    return cuda(q, "bf16"), cuda(k, "bf16"), cuda(signal(rng, n, g, d), "bf16"), cuda(signal(rng, n, h, d), "bf16"), cu


@pytest.mark.parametrize("lengths,behind,h,g,d,window,sinks", ATTN)
def test_window_attention(ops, lengths, behind, h, g, d, window, sinks):
    import torch

    rng = np.random.default_rng(len(lengths) + d + window)
    q, k, v, do, cu = attn_case(rng, lengths, behind, h, g, d)
    scale = 1 / np.sqrt(d)
    how = {"window": window, "sinks": sinks, "cu_seqlens": cu}
    out, lse = ops.window_attention(q, k, v, **how)
    see = O.visible(q.shape[0], lengths, window, sinks)
    want, wl, bo, bl = O.window_attention(host(q), host(k), host(v), see, scale)
    within(out, want, bo, "bf16")
    got = host(lse)
    empty = ~see.any(1)
    assert (got[:, empty] == -np.inf).all()
    assert (np.abs(got[:, ~empty] - wl[:, ~empty]) <= bl[:, ~empty]).all()
    grads = ops.window_attention_backward(do, q, k, v, out, lse, **how)
    exact, bounds = O.window_attention_backward(host(do), host(q), host(k), host(v), see, scale)
    for g_, w_, b_ in zip(grads, exact, bounds):
        within(g_, w_, b_, "bf16")
    again = ops.window_attention(q, k, v, **how)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    for a, b in zip(ops.window_attention_backward(do, q, k, v, out, lse, **how), grads):
        assert torch.equal(a, b)


def test_window_attention_without_bounds_is_one_sample(ops):
    import torch

    rng = np.random.default_rng(11)
    q, k, v, do, cu = attn_case(rng, [333], 0, 4, 2, 64)
    for window in (None, 333, 10 ** 12):
        one = ops.window_attention(q, k, v, window=window, sinks=2)
        two = ops.window_attention(q, k, v, window=333, sinks=0, cu_seqlens=cu)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
        assert all(torch.equal(a, b) for a, b in zip(ops.window_attention_backward(do, q, k, v, *one, window=window),
                                                     ops.window_attention_backward(do, q, k, v, *two, window=333,
                                                                                   cu_seqlens=cu)))


def test_window_attention_strides(ops):
    """Slices of a fused projection, heads before tokens, and a strided gradient give the same bits as copies."""
    import torch

    rng = np.random.default_rng(12)
    n, h, g, d = 200, 4, 2, 64
    qkv = cuda(signal(rng, n, h + 2 * g, d), "bf16")
    q, k, v = qkv[:, :h], qkv[:, h:h + g], cuda(signal(rng, g, n, d), "bf16").transpose(0, 1)
    do = cuda(signal(rng, h, n, d), "bf16").transpose(0, 1)
    how = {"window": 70, "sinks": 3, "scale": 0.3}
    a = ops.window_attention(q, k, v, **how)
    c = [x.contiguous() for x in (q, k, v, do)]
    b = ops.window_attention(*c[:3], **how)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = ops.window_attention_backward(do, q, k, v, *a, **how)
    gb = ops.window_attention_backward(c[3], *c[:3], *b, **how)
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))
    # a gradient that autograd expanded from one number
    ones = torch.ones((), dtype=torch.bfloat16, device="cuda").expand(n, h, d)
    gc = ops.window_attention_backward(ones, q, k, v, *a, **how)
    gd = ops.window_attention_backward(ones.contiguous(), q, k, v, *a, **how)
    assert all(torch.equal(x, y) for x, y in zip(gc, gd))


def test_window_attention_output_strides(ops):
    """The saved output may lie in any layout: heads before tokens, a slice, rows off 16-byte boundaries."""
    import torch

    rng = np.random.default_rng(18)
    n, h, g, d = 200, 4, 2, 64
    q, k, v, do = (cuda(signal(rng, n, x, d), "bf16") for x in (h, g, g, h))
    how = {"window": 70, "sinks": 3, "scale": 0.3}
    out, lse = ops.window_attention(q, k, v, **how)
    want = ops.window_attention_backward(do, q, k, v, out, lse, **how)
    flipped = out.transpose(0, 1).contiguous().transpose(0, 1)
    part = torch.full((n, h + 3, d + 8), float("nan"), dtype=torch.bfloat16, device="cuda")[:, 1:h + 1, 8:]
    odd = torch.full((n, h, d + 1), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :, 1:]
    for other in (flipped, part, odd):
        other.copy_(out)
        got = ops.window_attention_backward(do, q, k, v, other, lse, **how)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_window_attention_samples_do_not_mix(ops):
    """Non-finite values in one sample, or behind the last, reach no other."""
    import torch

    rng = np.random.default_rng(13)
    lengths = [70, 130, 55]
    q, k, v, do, cu = attn_case(rng, lengths, 9, 2, 1, 64)
    how = {"window": 40, "sinks": 2, "cu_seqlens": cu}
    clean = ops.window_attention(q, k, v, **how)
    gclean = ops.window_attention_backward(do, q, k, v, *clean, **how)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = [t.clone() for t in (q, k, v, do)]
        for t in x:
            t[70:200] = bad
            t[255:] = bad
        out, lse = ops.window_attention(*x[:3], **how)
        keep = torch.ones(264, dtype=torch.bool)
        keep[70:200] = False
        assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[:, keep], clean[1][:, keep])
        grads = ops.window_attention_backward(x[3], *x[:3], out, lse, **how)
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(grads, gclean))
        assert (out[255:] == 0).all() and all((a[255:] == 0).all() for a in grads)


def test_window_attention_large_scores(ops):
    """Scores in the thousands: the softmax is one key's, and nothing overflows."""
    rng = np.random.default_rng(14)
    q, k, v, do, cu = attn_case(rng, [150], 0, 2, 1, 64)
    see = O.visible(150, [150], 60, 2)
    out, lse = ops.window_attention(q, k, v, window=60, sinks=2, scale=50.0)
    want, wl, bo, bl = O.window_attention(host(q), host(k), host(v), see, 50.0)
    within(out, want, bo, "bf16")
    assert (np.abs(host(lse) - wl) <= bl).all()
    grads = ops.window_attention_backward(do, q, k, v, out, lse, window=60, sinks=2, scale=50.0)
    exact, bounds = O.window_attention_backward(host(do), host(q), host(k), host(v), see, 50.0)
    for a, w, b in zip(grads, exact, bounds):
        within(a, w, b, "bf16")


# ---- streams, autograd ----

def test_operators_on_another_stream(ops):
    """Inputs made on one stream, the calls on another that waits for it."""
    import torch

    rng = np.random.default_rng(15)
    q, k, v, do, cu = attn_case(rng, [300], 0, 4, 2, 64)
    want = ops.window_attention(q, k, v, window=64)
    gw = ops.window_attention_backward(do, q, k, v, *want, window=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops.window_attention(q, k, v, window=64)
        gg = ops.window_attention_backward(do, q, k, v, *got, window=64)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and all(torch.equal(a, b) for a, b in zip(gg, gw))


def test_operators_in_a_graph(ops):
    """The calls can be captured, and a replay takes the inputs' new values."""
    import torch

    rng = np.random.default_rng(16)
    q, k, v, do, cu = attn_case(rng, [200, 57], 0, 4, 2, 64)
    ids = torch.tensor(rng.integers(0, 30, 257), device="cuda")
    d = cuda(signal(rng, 257, 64), "bf16")
    grad = torch.empty(30, 64, device="cuda")

    def calls():
        o = ops.window_attention(q, k, v, window=64, sinks=2, cu_seqlens=cu)
        return (*o, *ops.window_attention_backward(do, q, k, v, *o, window=64, sinks=2, cu_seqlens=cu),
                ops.embedding_backward(d, ids, grad))

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    q.copy_(cuda(signal(rng, *q.shape), "bf16"))
    d.copy_(cuda(signal(rng, *d.shape), "bf16"))
    graph.replay()
    torch.cuda.synchronize()
    held = [x.clone() for x in held]
    assert all(torch.equal(a, b) for a, b in zip(held, calls()))


def test_autograd_forms(ops):
    import torch

    rng = np.random.default_rng(17)
    n, h, g, d = 60, 4, 2, 64
    w = cuda(signal(rng, 20, h * d), "bf16").requires_grad_()
    ids = torch.tensor(rng.integers(-1, 20, n), device="cuda")
    _, k, qw, kw, cos, sin, pos = qk_case(rng, n, h, g, d, 32, "bf16", False)
    v = cuda(signal(rng, n, g, d), "bf16").requires_grad_()
    k = k.contiguous().requires_grad_()
    qw.requires_grad_(), kw.requires_grad_()
    x = ops.embedding_autograd(w, ids, scale=2.0).view(n, h, d)
    qr, kr = ops.qk_norm_rope_autograd(x, k, qw, kw, cos, sin, pos)
    out = ops.window_attention_autograd(qr, kr, v, window=16, sinks=1)
    do = cuda(signal(rng, n, h, d), "bf16")
    out.backward(do)
    o, lse = ops.window_attention(qr.detach(), kr.detach(), v.detach(), window=16, sinks=1)
    dqr, dkr, dv = ops.window_attention_backward(do, qr.detach(), kr.detach(), v.detach(), o, lse, window=16, sinks=1)
    dx, dk, dqw, dkw = ops.qk_norm_rope_backward(dqr, dkr, x.detach(), k.detach(), qw.detach(), kw.detach(), cos, sin, pos)
    dw = ops.embedding_backward(dx.view(n, h * d), ids, torch.empty_like(w), scale=2.0)
    for got, want in ((w.grad, dw), (k.grad, dk), (qw.grad, dqw), (kw.grad, dkw), (v.grad, dv)):
        assert torch.equal(got, want)


def test_wrappers_refuse(ops):
    """Wrong types, shapes and devices raise before anything is queued."""
    import torch

    from muon_adamw_hybrid_grad_gb300 import MuonAdamWError

    w, ids = torch.zeros(4, 16, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    x = torch.zeros(3, 2, 16, dtype=torch.bfloat16, device="cuda")
    ones, table = torch.ones(16, device="cuda"), torch.ones(5, 8, device="cuda")
    for error, call in (
            (TypeError, lambda: ops.embedding(w, ids.float())), (TypeError, lambda: ops.embedding(w.half(), ids)),
            (TypeError, lambda: ops.embedding(w, ids, dtype=torch.float16)), (TypeError, lambda: ops.embedding(w, 3)),
            (ValueError, lambda: ops.embedding(w, ids.cpu())), (ValueError, lambda: ops.embedding(w.T, ids)),
            (ValueError, lambda: ops.embedding(ones, ids)), (TypeError, lambda: ops.embedding(w, ids, scale="a")),
            (MuonAdamWError, lambda: ops.embedding(w, ids, scale=float("nan"))),
            (ValueError, lambda: ops.embedding_backward(torch.zeros(2, 16, device="cuda"), ids, w)),
            (ValueError, lambda: ops.embedding_backward(torch.zeros(3, 8, device="cuda"), ids, w)),
            (TypeError, lambda: ops.qk_norm_rope(x, x.float(), ones, ones, table, table, ids)),
            (ValueError, lambda: ops.qk_norm_rope(x, x[:2], ones, ones, table, table, ids)),
            (ValueError, lambda: ops.qk_norm_rope(x, x, ones[:8], ones, table, table, ids)),
            (ValueError, lambda: ops.qk_norm_rope(x, x, ones, ones, table, table[:4], ids)),
            (ValueError, lambda: ops.qk_norm_rope(x, x, ones, ones, table, table, ids[:2])),
            (ValueError, lambda: ops.qk_norm_rope(x[0], x, ones, ones, table, table, ids)),
            (MuonAdamWError, lambda: ops.qk_norm_rope(x, x, ones, ones, torch.ones(5, 7, device="cuda"),
                                                      torch.ones(5, 7, device="cuda"), ids)),
            (ValueError, lambda: ops.qk_norm_rope_backward(x, x.float(), x, x, ones, ones, table, table, ids)),
            (TypeError, lambda: ops.window_attention(x.float(), x, x, window=1)),
            (ValueError, lambda: ops.window_attention(x, x, x[:2], window=1)),
            (ValueError, lambda: ops.window_attention(x, x, x, window=1, cu_seqlens=ids)),
            (MuonAdamWError, lambda: ops.window_attention(x, x, x, window=-1)),
            (MuonAdamWError, lambda: ops.window_attention(x, x, x, window=1, sinks=200)),
            (MuonAdamWError, lambda: ops.window_attention(x, x, x, window=1, scale=-1.0)),
            (ValueError, lambda: ops.window_attention_backward(x, x, x, x, x, w, window=1))):
        with pytest.raises(error):
            call()
    ops.check()


@pytest.mark.parametrize("n,h,g,d,window,sinks", [
    (3890, 16, 8, 64, None, 0), (3890, 16, 8, 64, 300, 5), (2600, 16, 8, 128, 900, 3), (5000, 12, 12, 64, None, 2),
    (1300, 40, 20, 64, None, 1)])
def test_window_attention_many_items(ops, n, h, g, d, window, sinks):
    """More items than CTAs, in whole and part rounds: each key head's results are those of a call of its own."""
    import torch

    rng = np.random.default_rng(n + h)
    q, k, v, do = (cuda(signal(rng, n, x, d), "bf16") for x in (h, g, g, h))
    how = {"window": window, "sinks": sinks}
    out, lse = ops.window_attention(q, k, v, **how)
    grads = ops.window_attention_backward(do, q, k, v, out, lse, **how)
    assert all(bool(x.isfinite().all()) for x in (out, lse, *grads))
    per = h // g
    for i in range(g):
        hs, ks = slice(per * i, per * (i + 1)), slice(i, i + 1)
        o1, l1 = ops.window_attention(q[:, hs], k[:, ks], v[:, ks], **how)
        assert torch.equal(o1, out[:, hs]) and torch.equal(l1, lse[hs])
        one = ops.window_attention_backward(do[:, hs], q[:, hs], k[:, ks], v[:, ks], o1, l1, **how)
        for a, b in zip(one, (grads[0][:, hs], grads[1][:, ks], grads[2][:, ks])):
            assert torch.equal(a, b)
    ops.check()


@pytest.mark.parametrize("dim", [64, 128])
def test_window_attention_many_calls(ops, dim):
    """A packed batch again and again: no bounded wait runs out, and every call gives the same bits."""
    import torch

    rng = np.random.default_rng(18)
    q, k, v, do, cu = attn_case(rng, [513, 250, 1021, 64, 7, 700], 0, 16, 16, dim)
    how = {"window": 256, "sinks": 8, "cu_seqlens": cu}
    first = ops.window_attention(q, k, v, **how)
    grads = ops.window_attention_backward(do, q, k, v, *first, **how)
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(500):
        out = ops.window_attention(q, k, v, **how)
        again = ops.window_attention_backward(do, q, k, v, *out, **how)
        for a, b in zip((*out, *again), (*first, *grads)):
            same &= (a == b).all()
    assert bool(same)
    ops.check()


def test_attention_block_example():
    """The operators and the optimizer together: the loss of one batch falls."""
    import importlib.util
    import os

    from conftest import ROOT

    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.run(30)
    assert all(np.isfinite(losses))
    assert losses[-1] < 0.9 * losses[0]
    assert example.run(3) == losses[:3]
