"""Dropout, residual norm, expert products and log probabilities where their ranges end: long sums, large values,
calls that take longer than a wait may."""
import ctypes
import os
import shutil
import subprocess

import pytest

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


def normal(*shape, seed=0, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, device="cuda", dtype=dtype).normal_(generator=gen)


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
