"""The operators' autograd forms and what autograd is told of them.

What needs no kernel runs on the CPU, with plain stand-ins for the calls into
the library; the rest runs on the GPU.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    from muon_adamw_hybrid_grad_gb300 import build

    build.build()
    from muon_adamw_hybrid_grad_gb300 import ops as m

    return m


def sample_of(bounds, n):
    return torch.searchsorted(bounds.long(), torch.arange(n), right=True)


@pytest.fixture
def plain_attention(ops, monkeypatch):
    """Attention of one query head in plain CPU operations, in place of the library's calls."""

    def weights(q, k, window, sinks, scale, cu_seqlens):
        n = q.shape[0]
        i, j = torch.arange(n)[:, None], torch.arange(n)[None]
        cu = torch.tensor([0, n]) if cu_seqlens is None else cu_seqlens
        s = sample_of(cu, n)
        first = cu.long()[s - 1]
        see = (s[:, None] == s[None]) & (j <= i) & ((i - j < window) | (j - first[None] < sinks))
        return torch.softmax((scale * q[:, 0] @ k[:, 0].T).masked_fill(~see, -np.inf), -1)

    def forward(q, k, v, *, window, sinks=0, scale=None, cu_seqlens=None):
        p = weights(q, k, window, sinks, scale, cu_seqlens)
        return (p @ v[:, 0])[:, None], torch.zeros(1, q.shape[0])

    def backward(dout, q, k, v, out, lse, *, window, sinks=0, scale=None, cu_seqlens=None):
        p = weights(q, k, window, sinks, scale, cu_seqlens)
        dp = dout[:, 0] @ v[:, 0].T
        ds = scale * p * (dp - (p * dp).sum(1, keepdim=True))
        return tuple(x[:, None] for x in (ds @ k[:, 0], ds.T @ q[:, 0], p.T @ dout[:, 0]))

    monkeypatch.setattr(ops, "window_attention", forward)
    monkeypatch.setattr(ops, "window_attention_backward", backward)
    return weights


def leaves(n, d, seed):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(n, 1, d, generator=gen, dtype=torch.float64).requires_grad_() for _ in range(3)]


# ---- the samples' bounds ----

def test_attention_gradient_of_bounds_written_again_raises(ops, plain_attention):
    """One buffer of bounds, filled anew for each batch: a backward pass behind that must not take the new ones."""
    q, k, v = leaves(12, 4, 0)
    bounds = torch.tensor([0, 5, 12], dtype=torch.int32)
    out = ops.window_attention_autograd(q, k, v, window=3, scale=0.5, cu_seqlens=bounds)
    bounds.copy_(torch.tensor([0, 9, 12], dtype=torch.int32))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


@pytest.mark.parametrize("cu", [None, [0, 5, 12]])
def test_attention_form_takes_the_bounds_to_its_gradient(ops, plain_attention, cu):
    q, k, v = leaves(12, 4, 1)
    bounds = None if cu is None else torch.tensor(cu, dtype=torch.int32)
    how = {"window": 3, "sinks": 1, "scale": 0.5, "cu_seqlens": bounds}
    d = torch.randn(12, 1, 4, generator=torch.Generator().manual_seed(2), dtype=torch.float64)
    got = torch.autograd.grad(ops.window_attention_autograd(q, k, v, **how), (q, k, v), d)
    want = torch.autograd.grad((plain_attention(q, k, *how.values()) @ v[:, 0])[:, None], (q, k, v), d)
    # sums of at most 12 terms of size 10 in fp64
    assert all((a - b).abs().max() < 1e-12 for a, b in zip(got, want))


def packed_case(lengths, h, g, d, seed=0):
    rng = np.random.default_rng(seed)
    n = sum(lengths)
    q, k, v, do = (torch.tensor(rng.normal(size=(n, x, d)), dtype=torch.bfloat16, device="cuda") for x in (h, g, g, h))
    return q, k, v, do, torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32, device="cuda")


@pytest.mark.gpu
def test_autograd_of_packed_attention(ops):
    """Two micro-batches in flight, each with its own bounds; then bounds that are written again."""
    lengths = ([70, 1, 129], [200])
    cases = [packed_case(x, 4, 2, 64, i) for i, x in enumerate(lengths)]
    forms = []
    for q, k, v, do, cu in cases:
        x = [t.clone().requires_grad_() for t in (q, k, v)]
        forms.append((x, ops.window_attention_autograd(*x, window=40, sinks=2, cu_seqlens=cu)))
    for (q, k, v, do, cu), (x, out) in zip(cases, forms):
        out.backward(do)
        o, lse = ops.window_attention(q, k, v, window=40, sinks=2, cu_seqlens=cu)
        want = ops.window_attention_backward(do, q, k, v, o, lse, window=40, sinks=2, cu_seqlens=cu)
        assert torch.equal(out, o) and all(torch.equal(a.grad, b) for a, b in zip(x, want))
    q, k, v, do, cu = cases[0]
    out = ops.window_attention_autograd(q.requires_grad_(), k, v, window=40, cu_seqlens=cu)
    cu[1] = 7
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward(do)


# ---- second derivatives ----

NO_SECOND = "no second derivative"


def test_attention_refuses_a_second_derivative(ops, plain_attention):
    """A penalty on the gradient would otherwise go missing from the loss without a word."""
    q, k, v = leaves(9, 4, 3)
    out = ops.window_attention_autograd(q, k, v, window=4, scale=0.5)
    (g,) = torch.autograd.grad(out.sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match=NO_SECOND):
        (out.sum() + g.square().sum()).backward()


def test_norm_refuses_a_second_derivative(ops, monkeypatch):
    monkeypatch.setattr(ops, "qk_norm_rope", lambda q, k, qw, kw, *rest, **how: (q * q * qw, k * k * kw))
    monkeypatch.setattr(ops, "qk_norm_rope_backward", lambda dq, dk, q, k, qw, kw, *rest, **how: (
        2 * dq * q * qw, 2 * dk * k * kw, (dq * q * q).sum((0, 1)), (dk * k * k).sum((0, 1))))
    q, k, w = (torch.ones(s, dtype=torch.float64).requires_grad_() for s in ((3, 2, 4), (3, 1, 4), (4,)))
    t, pos = torch.ones(3, 2), torch.zeros(3, dtype=torch.int64)
    qo, ko = ops.qk_norm_rope_autograd(q, k, w, w, t, t, pos)
    (g,) = torch.autograd.grad(qo.sum() + ko.sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match=NO_SECOND):
        (qo.sum() + g.square().sum()).backward()


def test_embedding_refuses_a_second_derivative(ops, monkeypatch):
    """Its gradient is linear in what comes in: only a gradient of that one goes on."""
    monkeypatch.setattr(ops, "embedding", lambda w, ids, *, scale, dtype: scale * w[ids])
    monkeypatch.setattr(ops, "embedding_backward",
                        lambda dout, ids, grad, *, scale: grad.zero_().index_add_(0, ids, scale * dout))
    w, ids = torch.ones(5, 4, dtype=torch.float64).requires_grad_(), torch.tensor([1, 3, 1])
    out = ops.embedding_autograd(w, ids, scale=2.0)
    (g,) = torch.autograd.grad(out.square().sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match=NO_SECOND):
        (out.sum() + g.square().sum()).backward()
    (g,) = torch.autograd.grad(ops.embedding_autograd(w, ids, scale=2.0).sum(), w, create_graph=True)
    assert not g.requires_grad


def test_a_graph_of_the_gradient_that_nothing_differentiates(ops, plain_attention):
    """create_graph alone is no error, and gives the same first derivatives."""
    q, k, v = leaves(9, 4, 4)
    out = ops.window_attention_autograd(q, k, v, window=4, scale=0.5)
    held = torch.autograd.grad(out.square().sum(), (q, k, v), create_graph=True)
    out = ops.window_attention_autograd(q, k, v, window=4, scale=0.5)
    plain = torch.autograd.grad(out.square().sum(), (q, k, v))
    assert all(torch.equal(a, b) for a, b in zip(held, plain))


# ---- gradients in layouts that autograd chose ----

@pytest.mark.gpu
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("d", [64, 72])
def test_attention_gradient_of_a_slice_off_16_bytes(ops, first, d):
    """The output joined with a column: its gradient comes back as a slice whose rows miss 16-byte boundaries."""
    h, g = 4, 2
    q, k, v, do, cu = packed_case([130, 57], h, g, d)
    how = {"window": 50, "sinks": 2, "cu_seqlens": cu}
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    out = ops.window_attention_autograd(*x, **how)
    gate = torch.ones(len(do), 1, dtype=torch.bfloat16, device="cuda")
    parts = [out.flatten(1), gate] if first else [gate, out.flatten(1)]
    wide = torch.full((len(do), h * d + 1), 3.0, dtype=torch.bfloat16, device="cuda")
    (wide[:, :-1] if first else wide[:, 1:]).copy_(do.flatten(1))
    torch.cat(parts, 1).backward(wide)
    o, lse = ops.window_attention(q, k, v, **how)
    want = ops.window_attention_backward(do, q, k, v, o, lse, **how)
    assert all(torch.equal(a.grad, b) for a, b in zip(x, want))


@pytest.mark.gpu
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_gradient_of_a_slice_off_16_bytes(ops, first, dtype):
    n, h, g, d = 37, 4, 2, 64
    rng = np.random.default_rng(1)
    t = lambda *s: torch.tensor(rng.normal(size=s), dtype=dtype, device="cuda")  # noqa: E731
    q, k, dq, dk = t(n, h, d), t(n, g, d), t(n, h, d), t(n, g, d)
    qw, kw = (1 + 0.1 * t(d).float() for _ in range(2))
    cos, sin = t(8, 16).float(), t(8, 16).float()
    pos = torch.arange(n, device="cuda") % 8
    x = [y.clone().requires_grad_() for y in (q, k, qw, kw)]
    outs = ops.qk_norm_rope_autograd(*x, cos, sin, pos)
    gate = torch.ones(n, 1, dtype=dtype, device="cuda")
    joined, wides = [], []
    for y, dy in zip(outs, (dq, dk)):
        joined.append(torch.cat([y.flatten(1), gate] if first else [gate, y.flatten(1)], 1))
        wides.append(torch.full_like(joined[-1], 3.0))
        (wides[-1][:, :-1] if first else wides[-1][:, 1:]).copy_(dy.flatten(1))
    torch.autograd.backward(joined, wides)
    want = ops.qk_norm_rope_backward(dq, dk, q, k, qw, kw, cos, sin, pos)
    assert all(torch.equal(a.grad, b) for a, b in zip(x, want))


# ---- the gradient buffer's version ----

@pytest.mark.gpu
@pytest.mark.parametrize("n", [40, 5000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_gradient_tells_autograd_of_its_write(ops, n, accumulate):
    """A graph that saved the buffer before the call must not go on with what the call has put there."""
    ids = torch.arange(n, device="cuda") % 30
    grad = torch.ones(30, 16, device="cuda")
    x = torch.ones(30, 16, device="cuda", requires_grad=True)
    y = (x * grad).sum()
    before = grad._version
    ops.embedding_backward(torch.ones(n, 16, device="cuda"), ids, grad, accumulate=accumulate)
    assert grad._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    before = grad._version
    with pytest.raises(ValueError):
        ops.embedding_backward(torch.ones(n, 8, device="cuda"), ids, grad)
    assert grad._version == before  # a refused call has written nothing
    with torch.inference_mode():
        held = torch.ones(30, 16, device="cuda")
    ops.embedding_backward(torch.ones(n, 16, device="cuda"), ids, held)  # an inference tensor has no version


# ---- numbers past 64 bits ----

@pytest.mark.gpu
def test_window_past_64_bits_is_every_earlier_token(ops):
    """And a count of sinks past them is refused like any other that is too large."""
    from muon_adamw_hybrid_grad_gb300 import MuonAdamWError

    q, k, v, do, cu = packed_case([90, 40], 2, 1, 64)
    want = ops.window_attention(q, k, v, window=None, cu_seqlens=cu)
    got = ops.window_attention(q, k, v, window=10 ** 30, cu_seqlens=cu)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for how in ({"window": -10 ** 30}, {"window": 1, "sinks": 10 ** 30}, {"window": 1, "sinks": -10 ** 30}):
        with pytest.raises(MuonAdamWError):
            ops.window_attention(q, k, v, **how)
