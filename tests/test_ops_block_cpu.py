"""Dropout, residual norm, expert products and log probabilities without a GPU: the oracle's pins and the refusals."""
import ctypes
import math

import numpy as np
import pytest

from oracle import operators as O

# ---- pins of the definitions ----


@pytest.mark.parametrize("counter,key,want", [
    # the generator's published known answers
    ([0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0], "d16cfe09 94fdcceb 5001e420 24126ea1")])
def test_philox_known_answers(counter, key, want):
    got = O.philox(np.array([counter], dtype=np.uint64), key)[0]
    assert " ".join("%08x" % int(x) for x in got) == want


def test_dropout_factors():
    f = O.dropout_factors(100000, 0.25, 7, 1 << 40, 2)
    kept = (f > 0).mean()
    assert set(np.unique(f)) == {0.0, 1 / 0.75}
    assert abs(kept - 0.75) < 5 * math.sqrt(0.25 * 0.75 / 100000)
    assert np.array_equal(O.dropout_factors(40, 0.25, 7, 1 << 40, 2, first=64), f[64:104])
    for other in ((8, 1 << 40, 2), (7, 1, 2), (7, 1 << 40, 3)):
        assert (O.dropout_factors(1000, 0.25, *other) != f[:1000]).any()
    assert not O.dropout_factors(9, 1.0, 1, 2, 3).any()
    assert (O.dropout_factors(9, 0.0, 1, 2, 3) == 1).all()


def differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        at = flat[i]
        flat[i] = at + h
        up = f()
        flat[i] = at - h
        out[i] = (up - f()) / (2 * h)
        flat[i] = at
    return g


def test_residual_norm_backward_is_the_forward_derivative():
    rng = np.random.default_rng(0)
    x, res, w = rng.normal(size=(3, 10)), rng.normal(size=(3, 10)), 1 + 0.3 * rng.normal(size=10)
    dy, dres = rng.normal(size=(3, 10)), rng.normal(size=(3, 10))
    f = O.dropout_factors(30, 0.3, 1, 2, 3).reshape(3, 10)

    def loss():
        y, r, _, _ = O.residual_norm(x, res, w, 1e-3, f)
        return (y * dy).sum() + (r * dres).sum()

    (dx, dr, dw), _ = O.residual_norm_backward(dy, dres, O.residual_norm(x, res, w, 1e-3, f)[1], w, 1e-3, f)
    for got, at in ((dx, x), (dr, res), (dw, w)):
        assert np.abs(got - differences(loss, at)).max() < 1e-7


def test_token_logprobs_backward_is_the_forward_derivative():
    rng = np.random.default_rng(1)
    z, ids = rng.normal(size=(4, 9)), np.array([0, 8, -1, 4])
    z[1, 3] = z[3, 0] = -np.inf
    dlp, dh = rng.normal(size=4), rng.normal(size=4)

    def loss():
        (lp, h, _, _, _), _ = O.token_logprobs(z, ids, 1.3, 0)
        return (lp * dlp).sum() + (h * dh).sum()

    (lp, h, lse, tl, order), _ = O.token_logprobs(z, ids, 1.3, 3)
    got, _ = O.token_logprobs_backward(dlp, dh, z, ids, h, lse, 1.3)
    finite = np.isfinite(z)
    want = differences(loss, z)
    assert np.abs(got - want)[finite].max() < 1e-8 and not got[~finite].any()
    p = np.exp(1.3 * z) / np.exp(1.3 * z).sum(-1, keepdims=True)
    assert np.allclose(lp, [np.log(p[0, 0]), np.log(p[1, 8]), 0, np.log(p[3, 4])])
    assert np.allclose(h, -(p * np.log(np.maximum(p, 1e-300))).sum(-1))
    assert np.allclose(tl, np.sort(np.log(np.maximum(p, 1e-300)), -1)[:, :-4:-1])
    assert (O.token_logprobs(np.full((2, 5), -np.inf), np.array([1, -1]), 1.0, 2)[0][0] == [-np.inf, 0]).all()


def test_expert_matmul_backward_is_the_forward_derivative():
    rng = np.random.default_rng(2)
    x, w, dout, off = rng.normal(size=(7, 3)), rng.normal(size=(3, 4, 3)), rng.normal(size=(7, 4)), [0, 2, 2, 6]

    def loss():
        return (O.expert_matmul(x, w, off)[0] * dout).sum()

    (dx, dw), _ = O.expert_matmul_backward(dout, x, w, off)
    assert np.abs(dx - differences(loss, x)).max() < 1e-7 and np.abs(dw - differences(loss, w)).max() < 1e-7
    assert not dx[6:].any() and not dw[1].any()


# ---- refusals: arguments refused before any CUDA call; the pointers are host memory that nothing reads ----

BUF = ctypes.create_string_buffer(4096 + 256)
AT = (ctypes.addressof(BUF) + 255) // 256 * 256


@pytest.fixture(scope="module")
def mx():
    from muon_adamw_hybrid_grad_gb300 import build

    build.build()
    import muon_adamw_hybrid_grad_gb300 as m

    m.load_library()
    return m


def refused(mx, name, status, *args):
    lib = mx.load_library()
    got = getattr(lib, name)(*args)
    assert got == getattr(mx, "MA_ERR_" + status), (got, lib.muon_adamw_last_error())
    assert lib.muon_adamw_last_error()


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, "DTYPE"), ({"n": -1}, "SHAPE"), ({"n": 2 ** 35 + 1}, "SHAPE"), ({"p": -0.1}, "ARG"),
    ({"p": 1.1}, "ARG"), ({"p": math.nan}, "ARG"), ({"site": -1}, "ARG"), ({"x": None}, "ARG"), ({"out": None}, "ARG"),
    ({"rng": None}, "ARG"), ({"x": AT + 1}, "ALIGN"), ({"out": AT + 1}, "ALIGN"), ({"rng": AT + 4}, "ALIGN")])
def test_dropout_refuses(mx, kw, status):
    a = dict(x=AT, dtype=1, n=4, p=0.1, rng=AT, site=0, out=AT)
    a.update(kw)
    refused(mx, "muon_adamw_dropout", status, a["x"], a["dtype"], a["n"], a["p"], a["rng"], a["site"], a["out"], None)


def norm(mx, **kw):
    a = dict(n_tokens=4, width=16, dtype=1, stream_dtype=1, eps=1e-6, p=0.1, rng=AT, site=0)
    a.update(kw)
    return ctypes.byref(mx.ResidualNorm(**a))


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, "DTYPE"), ({"stream_dtype": -1}, "DTYPE"), ({"dtype": 0, "stream_dtype": 1}, "DTYPE"),
    ({"n_tokens": -1}, "SHAPE"), ({"n_tokens": 2 ** 30 + 1}, "SHAPE"), ({"width": 0}, "SHAPE"),
    ({"width": 32769}, "SHAPE"), ({"eps": -1.0}, "ARG"), ({"eps": math.inf}, "ARG"), ({"eps": 0.0}, "ARG"),
    ({"eps": 1e-39}, "ARG"), ({"p": 2.0}, "ARG"),
    ({"rng": None}, "ARG"), ({"rng": AT + 4}, "ALIGN"), ({"site": -1}, "ARG"),
    ({"n_tokens": 2 ** 30, "width": 64}, "SHAPE")])
def test_residual_norm_refuses(mx, kw, status):
    stride = kw.get("width", 16)
    refused(mx, "muon_adamw_residual_norm", status, norm(mx, **kw), AT, stride, AT, stride, AT, AT, None, AT, None)
    refused(mx, "muon_adamw_residual_norm_backward", status, norm(mx, **kw), AT, stride, AT, stride, AT, stride, AT, AT,
            AT, AT, AT, 1 << 40, None)


def test_residual_norm_refuses_tensors(mx):
    name, ok = "muon_adamw_residual_norm", [norm(mx), AT, 16, AT, 16, AT, AT, AT, AT, None]
    for i, x, status in ((0, None, "ARG"), (1, None, "ARG"), (1, AT + 1, "ALIGN"), (2, 15, "SHAPE"), (3, AT + 1, "ALIGN"),
                         (4, 8, "SHAPE"), (5, None, "ARG"), (5, AT + 2, "ALIGN"), (6, None, "ARG"), (7, AT + 2, "ALIGN"),
                         (8, AT + 1, "ALIGN")):
        bad = list(ok)
        bad[i] = x
        refused(mx, name, status, *bad)
    name = "muon_adamw_residual_norm_backward"
    ok = [norm(mx), AT, 16, AT, 16, AT, 16, AT, AT, AT, AT, AT, 1 << 30, None]
    for i, x, status in ((1, None, "ARG"), (2, 8, "SHAPE"), (3, AT + 1, "ALIGN"), (5, None, "ARG"), (6, 4, "SHAPE"),
                         (7, None, "ARG"), (8, None, "ARG"), (9, None, "ARG"), (10, None, "ARG"), (10, AT + 2, "ALIGN"),
                         (11, None, "ARG"), (11, AT + 16, "ALIGN"), (12, 8, "ARG")):
        bad = list(ok)
        bad[i] = x
        refused(mx, name, status, *bad)
    lib, n = mx.load_library(), ctypes.c_int64()
    assert lib.muon_adamw_residual_norm_backward_workspace(norm(mx), ctypes.byref(n)) == 0 and n.value >= 4 * 16 * 4
    refused(mx, name + "_workspace", "ARG", norm(mx), None)
    refused(mx, name + "_workspace", "SHAPE", norm(mx, width=0), ctypes.byref(n))


def expert(mx, **kw):
    a = dict(n_tokens=4, n_experts=2, inner=16, outer=24, offsets=AT, x=AT, x_stride=16, weight=AT,
             weight_row_stride=16, weight_expert_stride=16 * 24)
    a.update(kw)
    return ctypes.byref(mx.ExpertMatmul(**a))


@pytest.mark.parametrize("kw,status", [
    ({"n_experts": 0}, "SHAPE"), ({"n_experts": 513}, "SHAPE"), ({"inner": 12}, "SHAPE"), ({"inner": 0}, "SHAPE"),
    ({"outer": 20}, "SHAPE"), ({"outer": 2 ** 21}, "SHAPE"), ({"n_tokens": -1}, "SHAPE"),
    ({"n_tokens": 2 ** 28 + 1}, "SHAPE"), ({"offsets": None}, "ARG"), ({"offsets": AT + 2}, "ALIGN"),
    ({"weight": None}, "ARG"), ({"weight": AT + 8}, "ALIGN"), ({"weight_row_stride": 8}, "SHAPE"),
    ({"weight_row_stride": 20, "weight_expert_stride": 480}, "ALIGN"), ({"weight_expert_stride": 100}, "SHAPE"),
    ({"weight_expert_stride": 388}, "ALIGN"), ({"x": None}, "ARG"), ({"x": AT + 2}, "ALIGN"), ({"x_stride": 8}, "SHAPE"),
    ({"x_stride": 20}, "ALIGN"), ({"n_tokens": 2 ** 28, "outer": 2 ** 20, "weight_expert_stride": 2 ** 25}, "SHAPE")])
def test_expert_matmul_refuses(mx, kw, status):
    refused(mx, "muon_adamw_expert_matmul", status, expert(mx, **kw), AT, None)
    refused(mx, "muon_adamw_expert_matmul_backward", status, expert(mx, **kw), AT, kw.get("outer", 24), AT, AT, 0, 0, None)


def test_expert_matmul_refuses_tensors(mx):
    refused(mx, "muon_adamw_expert_matmul", "ARG", None, AT, None)
    refused(mx, "muon_adamw_expert_matmul", "ARG", expert(mx), None, None)
    refused(mx, "muon_adamw_expert_matmul", "ALIGN", expert(mx), AT + 8, None)
    name, ok = "muon_adamw_expert_matmul_backward", [expert(mx), AT, 24, AT, AT, 0, 0, None]
    for i, x, status in ((1, None, "ARG"), (1, AT + 2, "ALIGN"), (2, 16, "SHAPE"), (2, 28, "ALIGN"), (3, AT + 8, "ALIGN"),
                         (4, AT + 8, "ALIGN"), (5, 2, "DTYPE"), (6, 2, "ARG")):
        bad = list(ok)
        bad[i] = x
        refused(mx, name, status, *bad)


def logits(mx, **kw):
    a = dict(n_tokens=4, vocab=30, stride=32, dtype=1, id_bytes=8, scale=1.0, logits=AT, ids=AT)
    a.update(kw)
    return ctypes.byref(mx.TokenLogprobs(**a))


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, "DTYPE"), ({"id_bytes": 2}, "ARG"), ({"n_tokens": -1}, "SHAPE"), ({"vocab": 0}, "SHAPE"),
    ({"vocab": 2 ** 20 + 1, "stride": 2 ** 21}, "SHAPE"), ({"n_tokens": 2 ** 30, "vocab": 2 ** 20, "stride": 2 ** 20}, "SHAPE"),
    ({"stride": 29}, "SHAPE"), ({"scale": 0.0}, "ARG"), ({"scale": -1.0}, "ARG"), ({"scale": math.nan}, "ARG"),
    ({"scale": 1e39}, "ARG"), ({"scale": 1e-60}, "ARG"), ({"scale": 1e-31}, "ARG"), ({"scale": 1e31}, "ARG"), ({"logits": None}, "ARG"), ({"ids": None}, "ARG"),
    ({"logits": AT + 1}, "ALIGN"), ({"ids": AT + 4}, "ALIGN")])
def test_token_logprobs_refuses(mx, kw, status):
    refused(mx, "muon_adamw_token_logprobs", status, logits(mx, **kw), 2, AT, AT, AT, AT, AT, None)
    refused(mx, "muon_adamw_token_logprobs_backward", status, logits(mx, **kw), AT, AT, AT, AT, AT, 2 ** 21, None)


def test_token_logprobs_refuses_tensors(mx):
    name, ok = "muon_adamw_token_logprobs", [logits(mx), 2, AT, AT, AT, AT, AT, None]
    for i, x, status in ((0, None, "ARG"), (1, -1, "ARG"), (1, 33, "ARG"), (1, 31, "ARG"), (2, None, "ARG"),
                         (3, None, "ARG"), (4, None, "ARG"), (4, AT + 2, "ALIGN"), (5, None, "ARG"), (6, None, "ARG"),
                         (6, AT + 4, "ALIGN")):
        bad = list(ok)
        bad[i] = x
        refused(mx, name, status, *bad)
    name, ok = "muon_adamw_token_logprobs_backward", [logits(mx), AT, AT, AT, AT, AT, 32, None]
    for i, x, status in ((1, AT + 2, "ALIGN"), (2, AT + 2, "ALIGN"), (3, None, "ARG"), (4, None, "ARG"), (5, None, "ARG"),
                         (5, AT + 1, "ALIGN"), (6, 29, "SHAPE")):
        bad = list(ok)
        bad[i] = x
        refused(mx, name, status, *bad)


def test_wrappers_refuse_cpu_tensors(mx):
    torch = pytest.importorskip("torch")
    from muon_adamw_hybrid_grad_gb300 import ops

    x, w, rng = torch.zeros(3, 16), torch.ones(16), torch.zeros(2, dtype=torch.int64)
    ids, off, e = torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32), torch.zeros(1, 8, 16)
    for call in (lambda: ops.dropout(x, 0.1, rng), lambda: ops.residual_norm(x, x, w),
                 lambda: ops.residual_norm_backward(x, x, x, w), lambda: ops.expert_matmul(x, e, off),
                 lambda: ops.expert_matmul_backward(x, x, e, off, None), lambda: ops.token_logprobs(x, ids),
                 lambda: ops.token_logprobs_backward(x, x, x, ids, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="tensor"):
        ops.dropout(3, 0.1, rng)
