"""Dropout, residual norm, expert products and log probabilities on the GPU against their fp64 definitions.

Tolerances come from the arithmetic alone (``oracle/operators.py``): fp32 sums,
a power of two good to 2^-22, and one rounding of each result to its type
(2^-8 relative for bf16, 2^-24 for fp32, 2^-4 for e4m3).
"""
import numpy as np
import pytest

from oracle import operators as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TINY = 1e-30  # absolute slack for results that are zero
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
UNIT = {torch.float32: O.U32, torch.bfloat16: O.UB}


@pytest.fixture(scope="module")
def ops():
    from muon_adamw_hybrid_grad_gb300 import build

    build.build()
    from muon_adamw_hybrid_grad_gb300 import ops as m

    yield m
    m.check()
    torch.cuda.empty_cache()


def host(x):
    return x.detach().double().cpu().numpy()


def cuda(x, dtype="fp32"):
    return torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda").to(DTYPES[dtype])


def within(got, want, bound):
    """|got - want| <= bound, plus one rounding of a value up to |want| + bound to the result's type."""
    unit, got = UNIT[got.dtype], host(got)
    assert got.shape == want.shape
    plain = np.isfinite(want)
    assert np.array_equal(got[~plain], want[~plain], equal_nan=True), (got[~plain][:5], want[~plain][:5])
    bound = np.broadcast_to(bound, want.shape)
    got, want, bound = got[plain], want[plain], bound[plain]
    assert np.isfinite(got).all()
    err, lim = np.abs(got - want), bound + unit * (np.abs(want) + bound) + TINY
    bad = err > lim
    assert not bad.any(), (int(bad.sum()), float((err / lim).max()), np.argwhere(bad)[:3].tolist())


def rng_of(seed, step):
    return torch.tensor([seed, step], device="cuda")


SEED, STEP = -0x1234567890ABCDEF, (5 << 32) + 77
U64 = (1 << 64) - 1


def factors(n, p, site, seed=SEED, step=STEP, first=0):
    return O.dropout_factors(n, p, seed & U64, step & U64, site, first)


# ---- dropout ----

@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (7, 13), (3, 2, 64), (8191,), (8197,), (40000,)])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(ops, shape, dt, p):
    rng = np.random.default_rng(sum(shape))
    x = cuda(rng.normal(size=shape), dt)
    f = factors(x.numel(), p, 3).reshape(shape)
    got = ops.dropout(x, p, rng_of(SEED, STEP), site=3)
    within(got, host(x) * f, 2 * O.U32 * np.abs(host(x) * f))
    assert torch.equal(got != 0, (cuda(f) != 0) & (x != 0))
    assert torch.equal(got, ops.dropout_backward(x, p, rng_of(SEED, STEP), site=3))
    # off 16-byte boundaries, and with strides
    wide = torch.zeros(x.numel() + 1, device="cuda", dtype=x.dtype)
    wide[1:] = x.flatten()
    assert torch.equal(ops.dropout(wide[1:], p, rng_of(SEED, STEP), site=3), got.flatten())
    if x.dim() == 2:
        assert torch.equal(ops.dropout(x.T.contiguous().T, p, rng_of(SEED, STEP), site=3), got)


def test_dropout_keeps_what_the_counter_says(ops):
    x = torch.ones(1000, device="cuda")
    base = ops.dropout(x, 0.5, rng_of(1, 2), site=0)
    for rng, site in ((rng_of(1, 2), 1), (rng_of(1, 3), 0), (rng_of(2, 2), 0), (rng_of(1, 2 + (1 << 32)), 0)):
        assert (ops.dropout(x, 0.5, rng, site=site) != base).any()
    assert torch.equal(ops.dropout(x, 0.5, rng_of(1, 2), site=0), base)
    assert ops.dropout(x[:0], 0.5, rng_of(1, 2)).shape == (0,)


def test_dropped_elements_are_zero_whatever_they_hold(ops):
    x = torch.full((4096,), float("nan"), device="cuda", dtype=torch.bfloat16)
    got = ops.dropout(x, 0.5, rng_of(3, 4))
    f = cuda(factors(4096, 0.5, 0, 3, 4))
    assert torch.equal(got.isnan(), f != 0) and not got[f == 0].any()
    x.fill_(float("inf"))
    assert torch.equal(ops.dropout(x, 0.5, rng_of(3, 4)).isinf(), f != 0)


def test_dropout_past_2_31_elements(ops):
    n = (1 << 31) + 8205
    x = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    got = ops.dropout(x, 0.5, rng_of(3, 4), site=1)
    for first in (0, (1 << 31) - 64, n // 8 * 8 - 8000):
        want = factors(min(8005, n - first), 0.5, 1, 3, 4, first)
        assert np.array_equal(host(got[first:first + len(want)]), want)


def test_dropout_in_a_graph_takes_the_step_of_each_replay(ops):
    x, rng = torch.ones(5000, device="cuda"), rng_of(9, 0)
    ops.dropout(x, 0.3, rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.dropout(x, 0.3, rng)
        rng[1].add_(1)
    for step in range(3):
        graph.replay()
        assert np.allclose(host(out), factors(5000, 0.3, 0, 9, step))


# ---- residual and norm ----

WIDTHS = [1, 7, 8, 24, 250, 256, 264, 512, 520, 1000, 1001, 1024, 1032, 2048, 2050, 2056, 4096, 4104, 8192, 8200, 9001,
          16384, 16392, 32760, 32768]
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]


def norm_case(width, n, dt, st, residual=True, p=0.0, strided=False, seed=0):
    rng = np.random.default_rng(width + n + seed)
    loud = 1 + 9 * (rng.random(width) < 0.05)

    def rows(scale, t):
        x = cuda(rng.normal(size=(n, width)) * scale, t)
        if not strided:
            return x
        wide = torch.full((n, width + 8), float("nan"), device="cuda", dtype=x.dtype)
        wide[:, :width] = x
        return wide[:, :width]

    x, res = rows(1.0, dt), rows(2 * loud, st) if residual else None
    return x, res, cuda(1 + 0.2 * rng.normal(size=width)), factors(n * width, p, 2).reshape(n, width)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dt,st", TYPES)
@pytest.mark.parametrize("p,residual", [(0.0, True), (0.2, True), (0.2, False), (0.0, False)])
def test_residual_norm(ops, width, dt, st, p, residual):
    if not residual and dt != st:
        pytest.skip("without a residual the stream has the branch's type")
    for n in (1, 11):
        for strided in (False, True):
            x, res, w, f = norm_case(width, n, dt, st, residual, p, strided)
            how = {"eps": 1e-5, "p": p, "rng": rng_of(SEED, STEP) if p else None, "site": 2}
            y, r = ops.residual_norm(x, res, w, **how)
            zeros = np.zeros((n, width))
            wy, wr, by, br = O.residual_norm(host(x), zeros if res is None else host(res), host(w), 1e-5, f)
            within(y, wy, by)
            within(r, wr, br)
            assert y.dtype == x.dtype and r.dtype == DTYPES[st]
            assert (r is x) == (not residual and p == 0)
            q, scales, r8 = ops.residual_norm(x, res, w, eight_bit=True, **how)
            assert q.dtype == torch.float8_e4m3fn and torch.equal(r8, r)
            top, btop = np.abs(wy).max(-1), by.max(-1)
            within(scales, top / 448, btop / 448 + 2 * O.U32 * top / 448)
            s = host(scales)[:, None]
            stands = host(q.float()) * s
            lim = by + 4 * O.U32 * np.abs(wy) + O.E4M3_UNIT * (np.abs(wy) + by) * (1 + 8 * O.U32) + s * O.E4M3_TINY
            assert (np.abs(stands - wy) <= lim + TINY).all()
            # the largest element takes the largest value
            assert (host(q.float().abs()).max(-1) == 448).all() or width == 1


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dt,st", TYPES)
@pytest.mark.parametrize("p,other", [(0.0, True), (0.2, True), (0.2, False), (0.0, False)])
def test_residual_norm_backward(ops, width, dt, st, p, other):
    for n, strided in ((1, False), (13, True), (13, False)):
        dy, dres, w, f = norm_case(width, n, dt, st, True, p, strided)
        _, r, _, _ = norm_case(width, n, dt, st, True, p, strided, seed=1)
        got = ops.residual_norm_backward(dy, dres if other else None, r, w, eps=1e-5, p=p,
                                         rng=rng_of(SEED, STEP) if p else None, site=2)
        want, bound = O.residual_norm_backward(host(dy), host(dres) if other else np.zeros((n, width)), host(r), host(w),
                                               1e-5, f)
        for x, y, b in zip(got, want, bound):
            within(x, y, b)
        assert (got[0] is got[1]) == (p == 0 and dt == st)


@pytest.mark.parametrize("n,width", [(20011, 72), (9000, 264), (5003, 1032), (3001, 2048), (1501, 4096), (777, 8192), (2500, 1001)])
@pytest.mark.parametrize("dt,st", TYPES)
def test_residual_norm_of_many_rows(ops, n, width, dt, st):
    """Several rows to a group of threads, and blocks' partial sums of the weight's gradient."""
    x, res, w, f = norm_case(width, n, dt, st, True, 0.1)
    how = {"eps": 1e-5, "p": 0.1, "rng": rng_of(SEED, STEP), "site": 2}
    y, r = ops.residual_norm(x, res, w, **how)
    wy, wr, by, br = O.residual_norm(host(x), host(res), host(w), 1e-5, f)
    within(y, wy, by)
    within(r, wr, br)
    got = ops.residual_norm_backward(x, res, r, w, **how)
    want, bound = O.residual_norm_backward(host(x), host(res), host(r), host(w), 1e-5, f)
    for a, b, c in zip(got, want, bound):
        within(a, b, c)
    again = ops.residual_norm_backward(x, res, r, w, **how)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("width", [64, 2048, 2056])
def test_residual_norm_rows_of_zeros_and_of_nan(ops, width):
    x, res, w, _ = norm_case(width, 6, "bf16", "bf16")
    want = ops.residual_norm(x, res, w, eight_bit=True)
    x[1], res[1], x[4, width // 2] = 0, 0, float("nan")
    q, s, r = ops.residual_norm(x, res, w, eight_bit=True)
    y, _ = ops.residual_norm(x, res, w)
    keep = torch.tensor([0, 2, 3, 5], device="cuda")
    assert all(torch.equal(a[keep].float(), b[keep].float()) for a, b in zip((q, s, r), want))
    assert not q[1].float().any() and s[1] == 0 and not y[1].any()
    assert y[4].isnan().all() and q[4].float().isnan().all()
    tiny = torch.full_like(x, 1e-38)
    from muon_adamw_hybrid_grad_gb300 import MuonAdamWError
    with pytest.raises(MuonAdamWError, match="eps"):
        ops.residual_norm(tiny, None, w, eps=0.0, eight_bit=True)
    q, s, _ = ops.residual_norm(tiny, None, w, eps=2e-38, eight_bit=True)
    assert q.float().isfinite().all() and s.isfinite().all()
    within(ops.residual_norm(tiny, None, w, eps=2e-38)[0], *[O.residual_norm(
        host(tiny), 0 * host(tiny), host(w), float(np.float32(2e-38)), np.ones(tiny.shape))[i] for i in (0, 2)])
    q, s, _ = ops.residual_norm(torch.full((2, width), 1.0, device="cuda"), None, torch.full_like(w, 1e-42), eight_bit=True)
    assert (q.float() == 448).all() and (s > 0).all()


def test_residual_norm_shapes(ops):
    x, res, w, _ = norm_case(40, 12, "bf16", "fp32")
    y, r = ops.residual_norm(x, res, w)
    y3, r3 = ops.residual_norm(x.view(2, 3, 2, 40), res.view(2, 3, 2, 40), w)
    assert y3.shape == r3.shape == (2, 3, 2, 40) and torch.equal(y3.flatten(0, 2), y) and torch.equal(r3.flatten(0, 2), r)
    yt, rt = ops.residual_norm(x.T.contiguous().T, res, w)
    assert torch.equal(yt, y) and torch.equal(rt, r)
    q, s, _ = ops.residual_norm(x.view(3, 4, 40), None, w, eight_bit=True)
    assert q.shape == (3, 4, 40) and s.shape == (3, 4)
    y0, r0 = ops.residual_norm(x[:0], res[:0], w)
    assert y0.shape == r0.shape == (0, 40)
    dx, dr, dw = ops.residual_norm_backward(x[:0], res[:0], res[:0], w)
    assert dx.shape == (0, 40) and not dw.any() and dw.shape == (40,)
    shared = x[:1].expand(12, 40)  # a broadcast gradient
    assert torch.equal(ops.residual_norm_backward(shared, None, r, w)[1],
                       ops.residual_norm_backward(shared.contiguous(), None, r, w)[1])


def test_residual_norm_past_2_31_elements(ops):
    n, width = 1_050_007, 2056
    x, res = (torch.empty(n, width, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(0)
    x.normal_(generator=gen)
    res.normal_(generator=gen)
    w, how = cuda(np.linspace(0.5, 1.5, width)), {"eps": 1e-5, "p": 0.5, "rng": rng_of(SEED, STEP), "site": 2}
    y, r = ops.residual_norm(x, res, w, **how)
    dx, dr, _ = ops.residual_norm_backward(x, res, r, w, **how)
    for rows in (slice(0, 2), slice(n - 3, n)):
        f = factors((rows.stop - rows.start) * width, 0.5, 2, first=rows.start * width).reshape(-1, width)
        wy, wr, by, br = O.residual_norm(host(x[rows]), host(res[rows]), host(w), 1e-5, f)
        within(y[rows], wy, by)
        within(r[rows], wr, br)
        (wx, wd, _), (bx, bd, _) = O.residual_norm_backward(host(x[rows]), host(res[rows]), host(r[rows]), host(w), 1e-5, f)
        within(dx[rows], wx, bx)
        within(dr[rows], wd, bd)


# ---- log probabilities ----

def logit_rows(rng, n, v):
    z = rng.normal(size=(n, v)) * 2
    z[np.arange(n)[:, None], rng.integers(0, v, (n, 3))] += 10
    return z


def check_logprobs(ops, z, ids, scale, top):
    want, bound = O.token_logprobs(host(z).reshape(-1, z.shape[-1]), host(ids).astype(np.int64).reshape(-1), scale, top)
    got = ops.token_logprobs(z, ids, scale=scale, top=top)
    for x, w, b in zip(got[:4], want[:4], bound):
        within(x.reshape(w.shape), w, b)
    assert np.array_equal(got[4].reshape(want[4].shape).cpu().numpy(), want[4])
    assert got[4].dtype == torch.int64 and got[3].shape == got[4].shape == (*ids.shape, top)
    return got


# one vector and less, both edges of rows off 16 bytes, one pass of a block and its borders, clusters of 2 to 8
VOCABS = [1, 2, 7, 8, 31, 100, 1000, 1001, 2048, 8191, 8192, 8200, 16384, 20001, 40003, 70000, 151936]


@pytest.mark.parametrize("v", VOCABS)
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 90])
def test_token_logprobs(ops, v, dt, n):
    if n == 90 and v > 41000:
        n = 40
    rng = np.random.default_rng(v + n)
    z, ids = cuda(logit_rows(rng, n, v), dt), torch.tensor(rng.integers(-1, v + 1, n), device="cuda")
    for top in sorted({0, 1, min(v, 5), min(v, 32)}):
        got = check_logprobs(ops, z, ids, 0.8, top)
    dlp, dh = cuda(rng.normal(size=n)), cuda(rng.normal(size=n))
    for l, h in ((dlp, dh), (dlp, None), (None, dh)):
        d = ops.token_logprobs_backward(l, h, z, ids, got[1], got[2], scale=0.8)
        zero = np.zeros(n)
        within(d, *O.token_logprobs_backward(zero if l is None else host(l), zero if h is None else host(h), host(z),
                                             ids.cpu().numpy(), host(got[1]), host(got[2]), 0.8))
        assert d.dtype == z.dtype
    i32 = ops.token_logprobs(z, ids.int(), scale=0.8, top=top)
    assert all(torch.equal(a, b) for a, b in zip(got, i32))


@pytest.mark.parametrize("n,v", [(700, 1003), (300, 33000), (170, 151935), (2, 1 << 20)])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_token_logprobs_of_many_rows(ops, n, v, dt):
    rng = np.random.default_rng(v)
    z = cuda(logit_rows(rng, min(n, 50), v), dt).repeat(-(-n // 50), 1)[:n]
    ids = torch.tensor(rng.integers(0, v, n), device="cuda")
    got = check_logprobs(ops, z, ids, 1.0, 20)
    again = ops.token_logprobs(z, ids, scale=1.0, top=20)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
def test_token_logprobs_layouts(ops, dt):
    rng = np.random.default_rng(4)
    wide = cuda(logit_rows(rng, 12, 1100), dt)
    ids = torch.tensor(rng.integers(0, 1000, 12), device="cuda")
    for z in (wide[:, :1000], wide[:, 3:1000], wide[::2, 5:1004], wide.T.contiguous().T):
        i = ids[:z.shape[0]] % z.shape[1]
        got = check_logprobs(ops, z, i, 1.0, 7)
        d = ops.token_logprobs_backward(got[0], got[1], z, i, got[1], got[2])
        c = ops.token_logprobs_backward(got[0], got[1], z.contiguous(), i, got[1], got[2])
        assert torch.equal(d, c) and d.is_contiguous()
    check_logprobs(ops, wide.view(3, 4, 1100), ids.view(3, 4), 1.0, 2)
    assert ops.token_logprobs(wide[:0], ids[:0], top=3)[3].shape == (0, 3)
    assert ops.token_logprobs_backward(ids[:0].float(), None, wide[:0], ids[:0], ids[:0].float(), ids[:0].float()).shape == (0, 1100)


@pytest.mark.parametrize("v", [50, 9000, 70001])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [2, 200])
def test_token_logprobs_masked_rows_and_ties(ops, v, dt, n):
    rng = np.random.default_rng(v)
    lowest = float(torch.finfo(DTYPES[dt]).min)
    z = np.full((9, v), -np.inf)
    z[1, [3, v - 1, v // 2]] = 1.0, 2.0, 2.0  # three allowed tokens, fewer than the alternatives
    z[2] = 0.5                                # all equal
    z[3] = lowest                             # masked by the type's lowest value
    z[4] = np.where(rng.random(v) < 0.5, -0.0, 0.0)
    z[5] = np.round(rng.normal(size=v))       # many ties
    z[6], z[6, v - 2] = lowest, 3.0
    z[7] = np.where(np.arange(v) % 2, -np.inf, rng.normal(size=v))
    z[8], z[8, 5:] = -np.inf, lowest
    z = cuda(np.tile(z, (-(-n // 9) if n > 9 else 1, 1)), dt)
    ids = torch.tensor(rng.integers(0, v, len(z)), device="cuda")
    ids[:9] = torch.tensor([1, 3, v - 1, 0, 2, 5, v - 2, 1, 0])
    got = check_logprobs(ops, z, ids, 1.0, 20)
    one = torch.ones(len(z), device="cuda")
    d = ops.token_logprobs_backward(one, one, z, ids, got[1], got[2])
    usual = torch.tensor([i for i in range(len(z)) if i % 9 not in (3, 8)], device="cuda")
    within(d[usual], *O.token_logprobs_backward(*(host(x[usual]) for x in (one, one, z)), ids[usual].cpu().numpy(),
                                                host(got[1][usual]), host(got[2][usual]), 1.0))
    assert not d[0].any() and d.isfinite().all()
    assert not ops.token_logprobs_backward(0 * one, 0 * one, z, ids, got[1], got[2]).any()


@pytest.mark.parametrize("v", [50, 9000, 70001])
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("scale", [0.7, 1.0, 3.0])
def test_token_logprobs_gradient_of_rows_of_large_values(ops, v, dt, scale):
    """Rows whose lse is too large to hold ln(sum), or is infinite: the gradient is the formula's, of z less its maximum."""
    rng = np.random.default_rng(v)
    lowest = float(torch.finfo(DTYPES[dt]).min)
    z = np.full((7, v), lowest)
    z[1, 5:] = -np.inf
    z[2] = 5000 + rng.normal(size=v)
    z[3] = np.where(rng.random(v) < 0.5, lowest, -4000 + 4 * rng.normal(size=v))
    z[4] = -lowest * np.where(rng.random(v) < 0.5, 1, 0.5)
    z[5] = -np.inf
    z[6] = rng.normal(size=v)
    z = cuda(z, dt)
    ids = torch.tensor([0, 3, 7, v - 1, 9, 1, 2], device="cuda")
    _, entropy, lse, _, _ = ops.token_logprobs(z, ids, scale=scale)
    one = torch.ones(7, device="cuda")
    for l, h in ((one, 0 * one), (0 * one, one), (-one, 0.5 * one)):
        d = ops.token_logprobs_backward(l, h, z, ids, entropy, lse, scale=scale)
        zr, at = host(z), ids.cpu().numpy()
        top = zr.max(-1, keepdims=True)
        zr = np.where(zr == -np.inf, -np.inf, zr - np.where(top == -np.inf, 0, top))
        (_, _, sums, _, _), _ = O.token_logprobs(zr, at, scale, 1)
        want, bound = O.token_logprobs_backward(host(l), host(h), zr, at, host(entropy), sums, scale)
        # ln s and its sum of v / 256 terms a thread; row 6 has its own lse, of magnitude below 2^4
        extra = (v / 256 + 16 + 2 ** 4) * O.U32 + 2 * O.EX2
        a = np.where(zr == -np.inf, 0, zr * scale - np.where(sums == -np.inf, 0, sums)[:, None])
        p = np.where(zr == -np.inf, 0, np.exp(a)) * (sums != -np.inf)[:, None]
        mag = scale * p * (1 + np.abs(a) + host(entropy)[:, None] + 1)
        within(d, want, bound + extra * mag)
    assert not ops.token_logprobs_backward(0 * one, 0 * one, z, ids, entropy, lse, scale=scale).any()
    assert ops.token_logprobs_backward(one, 1e12 * one, z, ids, entropy, lse, scale=scale).isfinite().all()


@pytest.mark.parametrize("n", [1, 200])
def test_token_logprobs_large_values_in_few_threads(ops, n):
    """More large logits in one thread's share than its list takes: columns 2048 apart, eight at a time."""
    v = 151936
    rng = np.random.default_rng(8)
    z = rng.normal(size=v)
    columns = np.arange(v)
    z[columns % 2048 < 24] = 100 + rng.normal(size=int((columns % 2048 < 24).sum()))
    z = cuda(np.tile(z, (n, 1)))
    check_logprobs(ops, z, torch.zeros(n, device="cuda", dtype=torch.int64), 0.5, 32)
    check_logprobs(ops, z.bfloat16(), torch.zeros(n, device="cuda", dtype=torch.int64), 0.5, 32)


@pytest.mark.parametrize("v", [100, 30000])
@pytest.mark.parametrize("n", [3, 300])
def test_token_logprobs_rows_of_nan_and_infinity(ops, v, n):
    rng = np.random.default_rng(v)
    z, ids = cuda(logit_rows(rng, n, v), "bf16"), torch.tensor(rng.integers(0, v, n), device="cuda")
    clean = ops.token_logprobs(z, ids, top=9)
    z[0, v // 3], z[1, 7], z[1, 8] = float("nan"), float("inf"), 0
    got = ops.token_logprobs(z, ids, top=9)
    assert all(torch.equal(a[2:], b[2:]) for a, b in zip(got, clean))
    assert all(x[:2].isnan().all() for x in got[:4])
    assert bool(((got[4] >= 0) & (got[4] < v)).all())
    z[0] = float("nan")
    got = ops.token_logprobs(z, ids, top=9)
    assert bool(((got[4] >= 0) & (got[4] < v)).all()) and got[0][0].isnan()


@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [1, 700])
def test_token_logprobs_of_nan_before_masked_tokens(ops, dt, n):
    """A NaN whose thread sees nothing but masked logits after it."""
    z = torch.full((n, 30000), -float("inf"), device="cuda", dtype=DTYPES[dt])
    ids = torch.zeros(n, device="cuda", dtype=torch.int64)
    z[:, 0] = 1.0
    for column in (8, 1000, 29999):
        z[0, column] = float("nan")
        assert all(x[0].isnan().all() for x in ops.token_logprobs(z, ids, top=3)[:4])
        assert all(x[0].isnan() for x in ops.token_logprobs(z, ids)[:3])
        z[0, column] = -float("inf")
    assert not any(x.any() for x in ops.token_logprobs(z, ids)[:2])


def test_token_logprobs_past_2_31_elements(ops):
    n, v = 14200, 151936
    z = torch.empty(n, v, device="cuda", dtype=torch.bfloat16)
    z.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    ids = torch.randint(0, v, (n,), device="cuda")
    got = ops.token_logprobs(z, ids, top=3)
    one = torch.ones(n, device="cuda")
    d = ops.token_logprobs_backward(one, one, z, ids, got[1], got[2])
    for rows in (slice(0, 2), slice(n - 3, n)):
        want, bound = O.token_logprobs(host(z[rows]), ids[rows].cpu().numpy(), 1.0, 3)
        for x, w, b in zip(got[:4], want[:4], bound):
            within(x[rows], w, b)
        assert np.array_equal(got[4][rows].cpu().numpy(), want[4])
        within(d[rows], *O.token_logprobs_backward(*(host(x[rows]) for x in (one, one, z)), ids[rows].cpu().numpy(),
                                                   host(got[1][rows]), host(got[2][rows]), 1.0))


# ---- products grouped by expert ----

def offsets_of(lengths):
    return torch.tensor(np.cumsum([0] + list(lengths)), device="cuda", dtype=torch.int32)


EXPERTS = [
    ((1,), 8, 8), ((3,), 64, 128), ((0,), 16, 16), ((300, 0, 5), 136, 520), ((31, 32, 33, 63, 64, 65), 72, 264),
    ((255, 256, 257), 128, 256), ((513, 1, 0, 0, 700), 192, 320), ((128,) * 3, 1000, 136), ((16, 17, 15), 8, 1032),
    ((2,) * 40, 256, 64), ((0, 0, 1, 0), 520, 8), ((1025,), 2048, 24), ((48, 80), 4096, 512), ((5,) * 500, 24, 40)]


@pytest.mark.parametrize("lengths,inner,outer", EXPERTS)
@pytest.mark.parametrize("behind", [0, 70])
def test_expert_matmul(ops, lengths, inner, outer, behind):
    rng = np.random.default_rng(inner + outer + behind)
    t = sum(lengths) + behind
    x, w = cuda(rng.normal(size=(t, inner)), "bf16"), cuda(rng.normal(size=(len(lengths), outer, inner)), "bf16")
    off = offsets_of(lengths)
    want, mag = O.expert_matmul(host(x), host(w), off.tolist())
    got = ops.expert_matmul(x, w, off)
    within(got, want, (inner + 16) * O.U32 * mag)
    assert not got[sum(lengths):].any()
    # rows of wider tensors, and matrices apart from one another
    wide_x = torch.full((t, inner + 16), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide_x[:, 8:8 + inner] = x
    wide_w = torch.full((len(lengths), outer + 3, inner + 8), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide_w[:, :outer, :inner] = w
    assert torch.equal(ops.expert_matmul(wide_x[:, 8:8 + inner], wide_w[:, :outer, :inner], off), got)


@pytest.mark.parametrize("lengths,inner,outer", EXPERTS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_expert_matmul_backward(ops, lengths, inner, outer, dt):
    rng = np.random.default_rng(inner * 3 + outer)
    t = sum(lengths) + 9
    x, w = cuda(rng.normal(size=(t, inner)), "bf16"), cuda(rng.normal(size=(len(lengths), outer, inner)), "bf16")
    dout, off = cuda(rng.normal(size=(t, outer)), "bf16"), offsets_of(lengths)
    (wx, ww), (mx, mw) = O.expert_matmul_backward(host(dout), host(x), host(w), off.tolist())
    grad = torch.full(w.shape, float("nan"), device="cuda", dtype=DTYPES[dt])
    dx, got = ops.expert_matmul_backward(dout, x, w, off, grad)
    assert got is grad
    within(dx, wx, (outer + 16) * O.U32 * mx)
    most = (max(lengths) + 16) * O.U32 * mw
    within(grad, ww, most)
    assert not dx[sum(lengths):].any()
    before = cuda(rng.normal(size=w.shape), dt)
    more = before.clone()
    none, _ = ops.expert_matmul_backward(dout, x, w, off, more, accumulate=True, input_grad=False)
    assert none is None
    within(more, ww + host(before), most + 2 * O.U32 * (np.abs(ww) + np.abs(host(before))))
    only, none = ops.expert_matmul_backward(dout, x, w, off, None)
    assert none is None and torch.equal(only, dx)
    # a gradient in a layout that the kernels cannot read
    odd = torch.zeros(t, outer + 1, device="cuda", dtype=torch.bfloat16)
    odd[:, 1:] = dout
    again = torch.empty_like(grad)
    assert torch.equal(ops.expert_matmul_backward(odd[:, 1:], x, w, off, again)[0], dx) and torch.equal(again, grad)


@pytest.mark.parametrize("lengths", [(70, 3, 130, 1, 64, 20)])
def test_expert_matmul_keeps_to_its_tokens(ops, lengths):
    """NaN and infinities of one expert's tokens, and behind all of them, reach no other expert."""
    rng = np.random.default_rng(3)
    off, t = offsets_of(lengths), sum(lengths) + 40
    x, w = cuda(rng.normal(size=(t, 200)), "bf16"), cuda(rng.normal(size=(len(lengths), 264, 200)), "bf16")
    dout = cuda(rng.normal(size=(t, 264)), "bf16")
    g = torch.empty(w.shape, device="cuda")
    out, (dx, _) = ops.expert_matmul(x, w, off), ops.expert_matmul_backward(dout, x, w, off, g)
    for bad in (float("nan"), float("inf")):
        for e in (1, 3, None):
            rows = slice(off[e], off[e + 1]) if e is not None else slice(sum(lengths), t)
            x2, w2, d2, g2 = x.clone(), w.clone(), dout.clone(), torch.empty_like(g)
            x2[rows], d2[rows] = bad, bad
            if e is not None:
                w2[e] = bad
            out2, (dx2, _) = ops.expert_matmul(x2, w2, off), ops.expert_matmul_backward(d2, x2, w2, off, g2)
            keep = torch.ones(t, dtype=torch.bool, device="cuda")
            if e is not None:
                keep[rows] = False
                assert not out2[rows].isfinite().any() and not g2[e].isfinite().any()
            others = [i for i in range(len(lengths)) if i != e]
            assert torch.equal(out2[keep], out[keep]) and torch.equal(dx2[keep], dx[keep])
            assert torch.equal(g2[others], g[others])


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [10, 20, 30, 40], [0, -5, 1000, 2000], [0, 100, 100, 99], [5, 4, 3, 2],
                                     [0, 2 ** 31 - 1, -2 ** 31, 60]])
def test_expert_matmul_offsets_out_of_order(ops, offsets):
    """Whatever they hold: the first counts as 0, another as at least the one before and at most all tokens."""
    rng = np.random.default_rng(5)
    x, w = cuda(rng.normal(size=(100, 64)), "bf16"), cuda(rng.normal(size=(3, 40, 64)), "bf16")
    dout = cuda(rng.normal(size=(100, 40)), "bf16")
    plain = [0]
    for o in offsets[1:]:
        plain.append(min(max(o, plain[-1]), 100))
    off, good = (torch.tensor(o, device="cuda", dtype=torch.int64).to(torch.int32) for o in (offsets, plain))
    g1, g2 = torch.empty(w.shape, device="cuda"), torch.empty(w.shape, device="cuda")
    assert torch.equal(ops.expert_matmul(x, w, off), ops.expert_matmul(x, w, good))
    assert torch.equal(ops.expert_matmul_backward(dout, x, w, off, g1)[0], ops.expert_matmul_backward(dout, x, w, good, g2)[0])
    assert torch.equal(g1, g2)


def test_expert_matmul_without_tokens(ops):
    x, w, off = (torch.zeros(*s, device="cuda", dtype=torch.bfloat16) for s in ((0, 64), (3, 40, 64), (4,)))
    off = off.int()
    assert ops.expert_matmul(x, w, off).shape == (0, 40)
    grad = torch.ones(3, 40, 64, device="cuda")
    dx, _ = ops.expert_matmul_backward(torch.zeros(0, 40, device="cuda", dtype=torch.bfloat16), x, w, off, grad, accumulate=True)
    assert dx.shape == (0, 64) and (grad == 1).all()
    ops.expert_matmul_backward(torch.zeros(0, 40, device="cuda", dtype=torch.bfloat16), x, w, off, grad)
    assert not grad.any()


def test_expert_matmul_of_512_experts(ops):
    rng = np.random.default_rng(6)
    lengths = rng.integers(0, 19, 512)
    x, w = cuda(rng.normal(size=(int(lengths.sum()), 64)), "bf16"), cuda(rng.normal(size=(512, 72, 64)), "bf16")
    off = offsets_of(lengths)
    want, mag = O.expert_matmul(host(x), host(w), off.tolist())
    out = ops.expert_matmul(x, w, off)
    within(out, want, 80 * O.U32 * mag)
    (wx, ww), (mx, mw) = O.expert_matmul_backward(host(out), host(x), host(w), off.tolist())
    dx, grad = ops.expert_matmul_backward(out, x, w, off, torch.empty_like(w))
    within(dx, wx, 88 * O.U32 * mx)
    within(grad, ww, 40 * O.U32 * mw)


@pytest.mark.parametrize("lengths,inner,outer", [((3000, 1, 2500, 4000, 130), 1024, 2048), ((20000,), 512, 776)])
def test_expert_matmul_of_many_units(ops, lengths, inner, outer):
    """Several units to a pair of CTAs, in both accumulators and past the ring's first lap."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    t = sum(lengths)
    x, dout = (torch.randn(t, d, generator=gen, device="cuda").bfloat16() for d in (inner, outer))
    w, off = torch.randn(len(lengths), outer, inner, generator=gen, device="cuda").bfloat16(), offsets_of(lengths)
    grad = torch.empty(w.shape, device="cuda")
    out, (dx, _) = ops.expert_matmul(x, w, off), ops.expert_matmul_backward(dout, x, w, off, grad)
    for e, n in enumerate(lengths):
        rows = slice(int(off[e]), int(off[e + 1]))
        for got, a, b, k in ((out[rows], x[rows], w[e].T, inner), (dx[rows], dout[rows], w[e], outer),
                             (grad[e], dout[rows].T, x[rows], n)):
            want, mag = a.double() @ b.double(), a.double().abs() @ b.double().abs()
            bound = (k + 16) * O.U32 * mag
            assert bool(((got.double() - want).abs() <= bound + UNIT[got.dtype] * (want.abs() + bound)).all())
    ops.check()


def test_expert_matmul_past_2_31_elements(ops):
    lengths, inner, outer = (1, 263001, 7), 16, 8200
    gen = torch.Generator(device="cuda").manual_seed(2)
    t, off = sum(lengths) + 5, offsets_of(lengths)
    x = torch.randn(t, inner, generator=gen, device="cuda").bfloat16()
    w = torch.randn(3, outer, inner, generator=gen, device="cuda").bfloat16()
    out = ops.expert_matmul(x, w, off)
    for rows in (slice(0, 40), slice(263001 // 2, 263001 // 2 + 40), slice(t - 40, t)):
        local = [min(max(int(o) - rows.start, 0), 40) for o in off]
        want, mag = O.expert_matmul(host(x[rows]), host(w), local)
        within(out[rows], want, (inner + 16) * O.U32 * mag)
    dx, _ = ops.expert_matmul_backward(out, x, w, off, None)
    rows = slice(t - 40, t)
    (want, _), (mag, _) = O.expert_matmul_backward(host(out[rows]), host(x[rows]), host(w),
                                                   [min(max(int(o) - rows.start, 0), 40) for o in off])
    within(dx[rows], want, (outer + 16) * O.U32 * mag)


# ---- refusals, streams, graphs, autograd ----

def test_refusals(ops):
    from muon_adamw_hybrid_grad_gb300 import MuonAdamWError

    x = torch.zeros(4, 16, device="cuda", dtype=torch.bfloat16)
    w, rng, ids = torch.ones(16, device="cuda"), rng_of(1, 2), torch.zeros(4, device="cuda", dtype=torch.int64)
    e, off = torch.zeros(2, 24, 16, device="cuda", dtype=torch.bfloat16), torch.tensor([0, 2, 4], device="cuda", dtype=torch.int32)
    bad = [
        (TypeError, lambda: ops.dropout(x.half(), 0.1, rng)), (MuonAdamWError, lambda: ops.dropout(x, 1.5, rng)),
        (ValueError, lambda: ops.dropout(x, 0.1, None)), (ValueError, lambda: ops.dropout(x, 0.1, rng.int())),
        (ValueError, lambda: ops.dropout(x, 0.1, rng.cpu())), (MuonAdamWError, lambda: ops.dropout(x, 0.1, rng, site=-1)),
        (MuonAdamWError, lambda: ops.dropout(x, 0.1, rng, site=2 ** 31)),
        (MuonAdamWError, lambda: ops.residual_norm(x, x, w, p=0.1, rng=rng, site=2 ** 32)),
        (ValueError, lambda: ops.residual_norm(x, x[:2], w)), (ValueError, lambda: ops.residual_norm(x, x, w[:8])),
        (ValueError, lambda: ops.residual_norm(x, x, w.bfloat16())), (MuonAdamWError, lambda: ops.residual_norm(x, x, w, p=0.1)),
        (MuonAdamWError, lambda: ops.residual_norm(x.float(), x, w)),
        (ValueError, lambda: ops.residual_norm_backward(x, x.float(), x, w)),
        (ValueError, lambda: ops.residual_norm_backward(x[:2], None, x, w)),
        (TypeError, lambda: ops.expert_matmul(x.float(), e, off)), (ValueError, lambda: ops.expert_matmul(x, e, off[:2])),
        (ValueError, lambda: ops.expert_matmul(x, e, off.long())), (ValueError, lambda: ops.expert_matmul(x[:, :8], e, off)),
        (ValueError, lambda: ops.expert_matmul(x, e.transpose(1, 2), off)),
        (MuonAdamWError, lambda: ops.expert_matmul(torch.zeros(4 * 16 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(4, 16), e, off)),
        (ValueError, lambda: ops.expert_matmul_backward(x, x, e, off, None)),
        (ValueError, lambda: ops.expert_matmul_backward(torch.zeros(4, 24, device="cuda", dtype=torch.bfloat16), x, e, off, e[:1])),
        (ValueError, lambda: ops.token_logprobs(x, ids[:2])), (TypeError, lambda: ops.token_logprobs(x, ids.float())),
        (MuonAdamWError, lambda: ops.token_logprobs(x, ids, top=17)), (MuonAdamWError, lambda: ops.token_logprobs(x, ids, top=33)),
        (MuonAdamWError, lambda: ops.token_logprobs(x, ids, scale=0.0)),
        (ValueError, lambda: ops.token_logprobs_backward(ids.float()[:2], None, x, ids, ids.float(), ids.float())),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    torch.cuda.synchronize()


def all_calls(ops, seed=0):
    """One call of each operator and its outputs, on the current stream."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, res = (torch.randn(300, 256, generator=gen, device="cuda").bfloat16() for _ in range(2))
    w, rng = torch.rand(256, generator=gen, device="cuda"), rng_of(5, seed)
    e, off = torch.randn(3, 136, 256, generator=gen, device="cuda").bfloat16(), offsets_of((100, 33, 160))
    z, ids = torch.randn(9, 5000, generator=gen, device="cuda"), torch.randint(0, 5000, (9,), generator=gen, device="cuda")
    grad, one = torch.empty(3, 136, 256, device="cuda"), torch.ones(9, device="cuda")

    def run():
        y, r = ops.residual_norm(x, res, w, p=0.2, rng=rng, site=1)
        q = ops.residual_norm(x, res, w, eight_bit=True)
        out = ops.expert_matmul(y, e, off)
        lp = ops.token_logprobs(z, ids, top=4)
        return [ops.dropout(x, 0.3, rng), y, r, q[0].float(), q[1], out, *lp,
                *ops.residual_norm_backward(y, x, r, w, p=0.2, rng=rng, site=1),
                ops.expert_matmul_backward(out, y, e, off, grad)[0], grad.clone(),
                ops.token_logprobs_backward(one, one, z, ids, lp[1], lp[2])]

    return run


def test_streams_and_graphs(ops):
    """On a side stream, captured, and two graphs replayed at once: what the plain calls give."""
    runs = [all_calls(ops, i) for i in range(2)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in runs]
    got = []
    for side, run in zip(sides, runs):
        with torch.cuda.stream(side):
            got.append(run())
    torch.cuda.synchronize()
    graphs, held = [], []
    for run in runs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(run())
    for _ in range(3):
        for side, graph in zip(sides, graphs):
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for a in (got, held):
        for x, y in zip(a, want):
            assert all(torch.equal(i, j) for i, j in zip(x, y))
    ops.check()


def test_autograd(ops):
    gen = torch.Generator(device="cuda").manual_seed(0)
    leaf = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16().requires_grad_()  # noqa: E731
    x, res, e = leaf(40, 64), leaf(40, 64), leaf(2, 72, 64)
    w = torch.rand(64, generator=gen, device="cuda").requires_grad_()
    rng, off = rng_of(1, 2), offsets_of((25, 11))
    ids = torch.randint(0, 72, (40,), generator=gen, device="cuda")
    y, r = ops.residual_norm_autograd(x, res, w, p=0.25, rng=rng, site=4)
    out = ops.expert_matmul_autograd(ops.dropout_autograd(y, 0.5, rng, site=5), e, off)
    lp, h, tl, ti = ops.token_logprobs_autograd(out, ids, scale=0.5, top=3)
    assert not tl.requires_grad and not ti.requires_grad
    loss = (lp - 0.1 * h).sum() + r.float().square().sum()
    got = torch.autograd.grad(loss, (x, res, w, e), retain_graph=True)
    # the same chain by the plain calls
    dlp = torch.ones(40, device="cuda")
    _, entropy, lse, _, _ = ops.token_logprobs(out.detach(), ids, scale=0.5)
    dout = ops.token_logprobs_backward(dlp, -0.1 * dlp, out.detach(), ids, entropy, lse, scale=0.5)
    grad = torch.empty_like(e)
    yd = ops.dropout(y.detach(), 0.5, rng, site=5)
    dy, _ = ops.expert_matmul_backward(dout, yd, e.detach(), off, grad)
    dr = (2 * r.detach().float()).bfloat16()
    dx, dres, dw = ops.residual_norm_backward(ops.dropout_backward(dy, 0.5, rng, site=5), dr, r.detach(), w.detach(),
                                              p=0.25, rng=rng, site=4)
    for a, b in zip(got, (dx, dres, dw, grad)):
        assert torch.equal(a, b)
    # parts of the outputs alone
    assert torch.equal(torch.autograd.grad(r.float().sum(), res, retain_graph=True)[0], torch.ones_like(res))
    (da,) = torch.autograd.grad(h.sum(), out, retain_graph=True)
    assert torch.equal(da, ops.token_logprobs_backward(None, dlp, out.detach(), ids, entropy, lse, scale=0.5))
    y1, same = ops.residual_norm_autograd(x, None, w)
    assert same is x and torch.equal(torch.autograd.grad(y1.sum(), x)[0],
                                     ops.residual_norm_backward(torch.ones_like(x), None, x.detach(), w.detach())[0])
    # a second derivative raises, and so does a gradient behind a new step
    for out1, at in ((ops.dropout_autograd(x, 0.5, rng), x), (ops.residual_norm_autograd(x, res, w)[0], x),
                     (ops.expert_matmul_autograd(x, e, off), e), (ops.token_logprobs_autograd(x, ids % 64)[0], x)):
        first, = torch.autograd.grad((out1.float() * x.float().mean()).sum(), at, create_graph=True)
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(first.float().square().sum(), x)
    d = ops.dropout_autograd(x, 0.5, rng)
    rng[1].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        d.sum().backward()


def test_expert_gradient_raises_its_version(ops):
    x, w = torch.ones(4, 8, device="cuda").bfloat16(), torch.ones(1, 8, 8, device="cuda").bfloat16()
    grad = torch.zeros(1, 8, 8, device="cuda")
    before = grad._version
    ops.expert_matmul_backward(x, x, w, offsets_of((4,)), grad)
    assert grad._version > before
