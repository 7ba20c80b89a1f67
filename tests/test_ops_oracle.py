"""The operators' fp64 definitions: gradients against differences, and hand-made cases."""
import numpy as np
import pytest

from oracle import operators as O


def numeric(f, x, h=1e-6):
    """Central differences of the scalar f at x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += h
        up = f(y)
        y[i] -= 2 * h
        g[i] = (up - f(y)) / (2 * h)
    return g


# central differences: truncation h^2 |f'''| / 6 ~ 1e-12, rounding 1e-16 |f| / h ~ 1e-9
DIFF = 1e-7


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(0)
    w, ids, d = rng.normal(size=(5, 3)), [4, 0, -1, 4, 7, 4], rng.normal(size=(6, 3))
    want = numeric(lambda x: (O.embedding(x, ids, 1.5) * d).sum(), w)
    grad, mag, count = O.embedding_backward(d, ids, 5, 1.5)
    assert np.abs(grad - want).max() < DIFF
    assert count[:, 0].tolist() == [1, 0, 0, 0, 3]
    assert (mag >= np.abs(grad) - 1e-15).all()


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_norm_rope_gradient_against_differences(neighbours, rot):
    rng = np.random.default_rng(1)
    x, w, dy = rng.normal(size=(2, 3, 8)), rng.normal(size=8), rng.normal(size=(2, 3, 8))
    ang = rng.normal(size=(2, rot // 2))
    cos, sin = np.cos(ang), np.sin(ang)
    f = lambda x, w: (O.norm_rope(x, w, cos, sin, 1e-3, neighbours)[0] * dy).sum()  # noqa: E731
    dx, dw = O.norm_rope_backward(dy, x, w, cos, sin, 1e-3, neighbours)[:2]
    assert np.abs(dx - numeric(lambda y: f(y, w), x)).max() < DIFF
    assert np.abs(dw - numeric(lambda y: f(x, y), w)).max() < DIFF


def test_rotation_keeps_pair_norms_and_adds_angles():
    rng = np.random.default_rng(2)
    x, w = rng.normal(size=(1, 1, 8)), np.ones(8)
    a, b = rng.normal(size=(1, 4)), rng.normal(size=(1, 4))
    once = O.norm_rope(x, w, np.cos(a + b), np.sin(a + b), 0.0, False)[0]
    first = O.norm_rope(x, w, np.cos(a), np.sin(a), 0.0, False)[0]  # mean square 1, so a second norm does nothing
    assert np.abs(O.norm_rope(first, w, np.cos(b), np.sin(b), 0.0, False)[0] - once).max() < 1e-12
    assert np.abs((once ** 2).sum() - 8) < 1e-12


@pytest.mark.parametrize("window,sinks", [(3, 1), (1, 0), (100, 0), (0, 2), (0, 0)])
def test_attention_gradient_against_differences(window, sinks):
    rng = np.random.default_rng(3)
    n, lengths = 9, [5, 3]  # the last token lies behind the samples
    q, k, v = rng.normal(size=(n, 4, 4)), rng.normal(size=(n, 2, 4)), rng.normal(size=(n, 2, 4))
    d, see = rng.normal(size=(n, 4, 4)), O.visible(n, lengths, window, sinks)
    f = lambda q, k, v: (O.window_attention(q, k, v, see, 0.5)[0] * d).sum()  # noqa: E731
    (dq, dk, dv), _ = O.window_attention_backward(d, q, k, v, see, 0.5)
    assert np.abs(dq - numeric(lambda x: f(x, k, v), q)).max() < DIFF
    assert np.abs(dk - numeric(lambda x: f(q, x, v), k)).max() < DIFF
    assert np.abs(dv - numeric(lambda x: f(q, k, x), v)).max() < DIFF


def test_what_a_query_sees():
    see = O.visible(8, [6, 1], 2, 1)
    assert [np.flatnonzero(r).tolist() for r in see] == [[0], [0, 1], [0, 1, 2], [0, 2, 3], [0, 3, 4], [0, 4, 5], [6], []]


def test_attention_of_one_key_is_its_value():
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(2, 1, 4)), rng.normal(size=(2, 1, 4)), rng.normal(size=(2, 1, 4))
    see = O.visible(2, [2], 1, 0)
    out, lse, _, _ = O.window_attention(q, k, v, see, 2.0)
    assert np.abs(out - v).max() < 1e-15
    assert np.abs(lse[0] - 2 * (q * k).sum((1, 2))).max() < 1e-12
    (dq, dk, _), _ = O.window_attention_backward(q, q, k, v, see, 2.0)
    assert np.abs(dq).max() < 1e-14 and np.abs(dk).max() < 1e-14
