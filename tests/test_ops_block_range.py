"""Dropout, residual norm, expert products and log probabilities where their ranges end: long sums, large values,
calls that take longer than a wait may."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import operators as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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


def normal(*shape, seed=0, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, device="cuda", dtype=dtype).normal_(generator=gen)


# ---- residual and norm ----

@pytest.mark.parametrize("width", [64, 1001, 2048, 2050, 16384])
@pytest.mark.parametrize("size,eps,of_dy", [(1e17, 1e-6, 1e-6), (1e17, 1e-6, 1e-10), (1e15, 1e-6, 1e-12),
                                            (1e-19, 2e-38, 100.0), (3e-20, 1.2e-38, 1e15), (1e-17, 1e-34, 1e16)])
def test_residual_norm_gradient_of_large_and_small_rows(ops, width, size, eps, of_dy):
    """Rows far from 1 whose squares still have a sum in fp32, or are outweighed by eps: the formula's intermediate
    values stay in range, and the bounds are those of usual rows."""
    r = size * normal(13, width, dtype=torch.float32)
    dy = of_dy * normal(13, width, seed=1, dtype=torch.float32)
    w = 1 + 0.2 * normal(width, seed=2, dtype=torch.float32)
    dx, dr, dw = (host(x) for x in ops.residual_norm_backward(dy, None, r, w, eps=eps))
    one = np.ones((13, width))
    want, bound = O.residual_norm_backward(host(dy), 0 * one, host(r), host(w), float(np.float32(eps)), one)
    for x, y, b in zip((dx, dr, dw), want, bound):
        assert np.isfinite(x).all() and (np.abs(x - y) <= b + 2.0 ** -24 * (np.abs(y) + b)).all()


# ---- products grouped by expert ----

WAIT_LIMIT = "kWaitLimitNs = 2000000000ull"


@pytest.fixture(scope="module")
def short_waits(tmp_path_factory):
    """The expert products with waits of at most 5 ms in place of 2 s, as a library of their own."""
    from muon_adamw_hybrid_grad_gb300 import build as b

    at = tmp_path_factory.mktemp("short_waits")
    src = at / "csrc"
    shutil.copytree(b.CSRC, src)
    header = src / "tcgen05.cuh"
    text = header.read_text()
    assert text.count(WAIT_LIMIT) == 1
    header.write_text(text.replace(WAIT_LIMIT, "kWaitLimitNs = 5000000ull"))
    (src / "errors.cu").write_text('#include "internal.h"\nnamespace ma {\nvoid set_last_error(const char*) {}\n'
                                   "void clear_last_error() {}\n}\n")
    flags = [f if f != b.CSRC else str(src) for f in b.NVCC_FLAGS]
    lib = str(at / "libexpert.so")
    subprocess.run([b._nvcc(), *b.ARCH, *flags, "-shared", "-cudart", "static", "-o", lib,
                    *(str(src / f) for f in ("expert_matmul.cu", "operators.cu", "errors.cu")), "-ldl", "-lpthread", "-lrt"],
                   check=True)
    assert os.path.exists(lib)
    return ctypes.CDLL(lib)


def test_expert_gradients_longer_than_a_wait(ops, short_waits):
    """The input gradient's units, 22 ms of them (2 * 16385 * 32768^2 operations at 1.6 PFLOP/s), go by before the
    weights' first unit has rows to clear: no wait of 5 ms is to run out meanwhile."""
    import muon_adamw_hybrid_grad_gb300 as mx

    t, k = 16385, 32768
    x, dout, w = normal(t, k), normal(t, k, seed=1), normal(1, k, k, seed=2)
    offsets = torch.tensor([0, t], device="cuda", dtype=torch.int32)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    d = mx.ExpertMatmul(n_tokens=t, n_experts=1, inner=k, outer=k, offsets=offsets.data_ptr(), x=x.data_ptr(), x_stride=k,
                        weight=w.data_ptr(), weight_row_stride=k, weight_expert_stride=k * k)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    call = short_waits.muon_adamw_expert_matmul_backward
    assert call(ctypes.byref(d), ctypes.c_void_p(dout.data_ptr()), ctypes.c_int64(k), ctypes.c_void_p(dx.data_ptr()),
                ctypes.c_void_p(dw.data_ptr()), 1, 0, stream) == 0
    assert short_waits.muon_adamw_operators_check(stream) == 0
    grad = torch.empty_like(w)
    again, _ = ops.expert_matmul_backward(dout, x, w, offsets, grad)
    assert torch.equal(dx, again) and torch.equal(dw, grad)


# Of one step of 16 terms, relative to the sum so far: it and the terms are cut off toward zero where they are added,
# the sum by less than its last bit, each term by less than a quarter of that (two bits further): 1 + 16 / 4 bits of
# 2^-23 at the most. (Of positive terms a million times smaller than their sum 2.4 are lost on average.)
STEP = 5 * 2.0 ** -23


@pytest.mark.parametrize("tokens", [2048, 4096, 65536, 1 << 20, (1 << 20) + 77])
@pytest.mark.parametrize("sign", ["both", "one"])
def test_fp32_weight_gradients_of_many_tokens(ops, tokens, sign):
    """The error does not grow with the tokens: an accumulator takes runs of 2048, 128 steps. The sum so far is on
    average half of the whole for terms of one sign, and 2/3 for those of both (it grows as a square root). The runs'
    sums are added to nearest: 512 additions, each off by 2^-24 of at most the whole, in both directions."""
    x, dout = normal(tokens, 64), normal(tokens, 128, seed=1)
    if sign == "one":
        x.abs_(), dout.abs_()
    w, offsets = normal(1, 128, 64, seed=2), torch.tensor([0, tokens], device="cuda", dtype=torch.int32)
    want = dout.double().T @ x.double()
    bound = 128 * STEP * 2 / 3 + 512 ** 0.5 * 2.0 ** -24
    before = normal(1, 128, 64, seed=3, dtype=torch.float32)
    for held in (None, before):
        grad = torch.empty_like(before) if held is None else held.clone()
        ops.expert_matmul_backward(dout, x, w, offsets, grad, accumulate=held is not None, input_grad=False)
        total = want if held is None else want + held[0].double()
        assert float((grad[0].double() - total).norm()) <= bound * float(want.norm()) + 2.0 ** -24 * float(total.norm())


@pytest.mark.parametrize("length,tokens", [(8192, 40), (8200, 300), (65536, 40), (1 << 20, 8)])
def test_long_contractions_of_expert_products(ops, length, tokens):
    """out and dx of terms of one sign, whose sums an accumulator cuts off in one direction. Runs of 8192, 512 steps,
    keep that below 1.6e-4; the result's own rounding is half a step of bf16, up to 3.9e-3."""
    x, w = normal(tokens, length).abs_(), normal(1, 16, length, seed=1).abs_()
    offsets = torch.tensor([0, tokens], device="cuda", dtype=torch.int32)
    want = x.double() @ w[0].double().T
    bound = torch.exp2(torch.floor(torch.log2(want)) - 8) + 512 * STEP / 2 * want
    assert ((ops.expert_matmul(x, w, offsets).double() - want).abs() <= bound).all()
    dx, _ = ops.expert_matmul_backward(x, x[:, :16], w.transpose(1, 2).contiguous(), offsets, None)
    assert ((dx.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("lengths,inner,outer", [((2049, 0, 4096, 31, 8193), 72, 520), ((20000, 64, 3), 264, 136)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_expert_gradients_of_several_runs(ops, lengths, inner, outer, dtype):
    """Units of one run between units of several: each result is that of its expert alone, bit by bit."""
    t = sum(lengths)
    x, dout, w = normal(t, inner), normal(t, outer, seed=1), normal(len(lengths), outer, inner, seed=2)
    bounds = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    offsets = torch.tensor(bounds, device="cuda", dtype=torch.int32)
    grad = torch.empty(w.shape, device="cuda", dtype=dtype)
    dx, _ = ops.expert_matmul_backward(dout, x, w, offsets, grad)
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        one = torch.tensor([0, b - a], device="cuda", dtype=torch.int32)
        alone = torch.empty_like(grad[e:e + 1])
        dx_e, _ = ops.expert_matmul_backward(dout[a:b], x[a:b], w[e:e + 1], one, alone)
        assert torch.equal(grad[e], alone[0]) and torch.equal(dx[a:b], dx_e)
        exact = dout[a:b].double().T @ x[a:b].double()
        unit = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
        run = 128 if dtype is torch.float32 else 512
        size = dout[a:b].double().abs().T @ x[a:b].double().abs()
        assert ((grad[e].double() - exact).abs() <= unit * exact.abs() + (run * STEP + 2.0 ** -20) * size).all()
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_several_runs_in_several_units_of_a_pair(ops, dtype, accumulate):
    """270 units of the weights and some 350 of dx over 76 pairs, of one to five runs each in any order: the two
    accumulators change their parts between units. dx has 8200 terms, two runs."""
    lengths, inner, outer = (2049, 100, 4096, 0, 31, 8193, 640, 2048), 1032, 8200
    t = sum(lengths)
    x, w = normal(t, inner), 0.02 * normal(len(lengths), outer, inner, seed=2)
    dout = 0.1 * normal(t, outer, seed=1)
    bounds = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    offsets = torch.tensor(bounds, device="cuda", dtype=torch.int32)
    held = normal(*w.shape, seed=3).to(dtype)
    grad = held.clone() if accumulate else torch.empty(w.shape, device="cuda", dtype=dtype)
    dx, _ = ops.expert_matmul_backward(dout, x, w, offsets, grad, accumulate=accumulate)
    unit, run = (2.0 ** -8, 512) if dtype is torch.bfloat16 else (2.0 ** -24, 128)
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a == b:
            assert torch.equal(grad[e], held[e]) if accumulate else not grad[e].any()
            continue
        d, xe, we = dout[a:b].double(), x[a:b].double(), w[e].double()
        want = d.T @ xe + (held[e].double() if accumulate else 0)
        # (every step is off by STEP at most, of a sum so far that is no larger than its terms' magnitudes)
        size = d.abs().T @ xe.abs()
        assert ((grad[e].double() - want).abs() <= unit * want.abs() + (run * STEP + 2.0 ** -20) * size).all()
        want, size = d @ we, d.abs() @ we.abs()
        assert ((dx[a:b].double() - want).abs() <= 2.0 ** -8 * want.abs() + (512 * STEP + 2.0 ** -20) * size).all()


# ---- log probabilities ----

@pytest.mark.parametrize("v", [60, 1003, 40001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [0.0, 50.0, 500.0, 2000.0, -700.0])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_token_logprobs_gradient_of_the_logits_alone(ops, v, dtype, at, scale):
    """The gradient is that of the logits, wherever their maximum lies: a stored lse adds no more than half a step of
    fp32 below kLseMax, 2^-19 for fp32 logits and 2^-14 for bf16 ones. The rest is the arithmetic of z less its
    maximum, and ln s, whose sum has v / 512 terms a thread, its joins and its new maxima."""
    n = 40
    z = (at + 3 * normal(n, v, dtype=torch.float32)).to(dtype)
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(-1, v, (n,), generator=gen, device="cuda")
    l, h = normal(n, seed=5, dtype=torch.float32), normal(n, seed=6, dtype=torch.float32)
    _, entropy, lse, _, _ = ops.token_logprobs(z, ids, scale=scale)
    zr = host(z)
    zr = zr - zr.max(-1, keepdims=True)
    at_ = ids.cpu().numpy()
    (_, exact_h, exact_lse, _, _), (_, bound_h, _, _) = O.token_logprobs(zr, at_, scale, 1)
    logs = (v / 512 + 64) * O.U32 + (v / 8192 + 16) * 2 * O.EX2
    unit = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
    for dl, dh in ((l, None), (None, h), (l, h)):
        d = host(ops.token_logprobs_backward(dl, dh, z, ids, entropy, lse, scale=scale))
        dl, dh = (np.zeros(n) if x is None else host(x) for x in (dl, dh))
        want, bound = O.token_logprobs_backward(dl, dh, zr, at_, exact_h, exact_lse, scale)
        p = np.exp(zr * scale - exact_lse[:, None])
        a, hh = np.abs(zr * scale - exact_lse[:, None]), np.abs(dh)[:, None]
        # a relative error of p, and an absolute one of log p and of the entropy
        off = (2.0 ** -14 if dtype is torch.bfloat16 else 2.0 ** -19) + logs
        inside = np.where((at_ >= 0) & (at_ < v), np.abs(dl), 0)[:, None]
        bound = bound + scale * p * (off * (inside + hh * (a + exact_h[:, None] + 1)) + hh * bound_h[:, None])
        assert (np.abs(d - want) <= bound + unit * (np.abs(want) + bound) + 1e-30).all()


@pytest.mark.parametrize("v", [40001, 151936, 1 << 20])
def test_token_logprobs_of_many_unlikely_tokens(ops, v):
    """A few likely tokens and a long tail, whose terms lie below one of the running sum: the errors of many rows have
    no common direction but the power of two's (2^-22 of each term) and that of the rounded scale * log2(e), 2^-24 of
    each exponent. The others are roundings to nearest: a group's 16 additions, the sum's, one for each group, and the
    results' own, each uniform within 2^-24 of a value below 1 + |log p|."""
    n, scale = 600, 1.25
    z = 2 * normal(n, v)
    gen = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, v, (n,), generator=gen, device="cuda")
    z[torch.arange(n, device="cuda"), ids] = (12 + 2 * normal(n, seed=2)).to(z.dtype)
    logprobs, entropy, lse, _, _ = ops.token_logprobs(z, ids, scale=scale)
    error, width, exponent = [], [], []
    for rows in torch.arange(n, device="cuda").split(50):
        a = z[rows].double() * scale
        want = torch.log_softmax(a, -1)
        given = want[torch.arange(len(rows)), ids[rows]]
        error.append(logprobs[rows].double() - given)
        width.append((16 + v / 4096 + 16 + (1 + given.abs()) ** 2) ** 0.5 * 2.0 ** -24 / 3 ** 0.5)
        exponent.append((want.exp() * (a.amax(-1, keepdim=True) - a)).sum(-1))
    error, width, exponent = torch.cat(error), torch.cat(width), torch.cat(exponent)
    common = 2.0 ** -22 + 2.0 ** -24 * float(exponent.mean())
    assert abs(float(error.mean())) <= common + 4 * float(width.square().mean()) ** 0.5 / n ** 0.5


def test_token_logprobs_gradient_of_masked_rows_takes_no_longer(ops):
    """A quarter of the rows without any token, or without a gradient at values whose lse is not used, beside usual
    rows: the batch moves the same bytes, and takes less than twice as long (times of one GPU in one process)."""
    n, v = 1200, 151936
    z = normal(n, v)
    ids = torch.arange(n, device="cuda")
    one = torch.ones(n, device="cuda")

    def best(z, l):
        _, entropy, lse, _, _ = ops.token_logprobs(z, ids)
        times = []
        for _ in range(6):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            for _ in range(4):
                ops.token_logprobs_backward(l, 0 * l, z, ids, entropy, lse)
            end.record()
            torch.cuda.synchronize()
            times.append(begin.elapsed_time(end))
        return min(times)

    usual = best(z, one)
    masked = z.clone()
    masked[::4] = -float("inf")
    assert best(masked, one) < 2 * usual
    masked[::4] = 5000
    l = one.clone()
    l[::4] = 0
    assert best(masked, l) < 2 * usual


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first", [0, 1])
def test_token_logprobs_gradient_of_rows_past_the_lowest_value(ops, dtype, first):
    """lse is -infinity although some logits are finite, in one block of several: the others' masked logits have no
    gradient, and the given token has its own wherever it is."""
    v, lowest = 30001, float(torch.finfo(dtype).min)
    wide = torch.full((4, v + first), -float("inf"), device="cuda", dtype=dtype)
    z = wide[:, first:]
    z[:3, 20000:20004] = lowest
    ids = torch.tensor([5, 20001, -1, 5], device="cuda")
    one = torch.ones(4, device="cuda")
    _, entropy, lse, _, _ = ops.token_logprobs(z, ids, scale=2.0)
    assert bool((lse == -float("inf")).all())
    d = ops.token_logprobs_backward(one, None, z, ids, entropy, lse, scale=2.0)
    want = torch.zeros(4, v, device="cuda")
    want[:2, 20000:20004] = -2 / 4
    want[0, 5], want[1, 20001] = 2, 2 - 2 / 4
    assert torch.allclose(d.float(), want, rtol=2.0 ** -20, atol=0)
