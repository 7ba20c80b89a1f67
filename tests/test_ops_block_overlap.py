"""Which calls of the log probabilities' gradient may write over what they read."""
import ctypes

import pytest

from test_ops_block_cpu import AT, logits, mx, refused  # noqa: F401


@pytest.mark.parametrize("vocab", [8193, 151936])
@pytest.mark.parametrize("dtype", [0, 1])
def test_gradient_over_the_logits_of_several_blocks_is_refused(mx, vocab, dtype):  # noqa: F811
    refused(mx, "muon_adamw_token_logprobs_backward", "ARG", logits(mx, vocab=vocab, stride=vocab, dtype=dtype), AT, AT,
            AT, AT, AT, vocab, None)


@pytest.mark.gpu
@pytest.mark.parametrize("v", [7, 1000, 8191, 8192])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("first", [0, 1])
def test_gradient_over_the_logits_of_one_block(mx, v, dtype, first):  # noqa: F811
    torch = pytest.importorskip("torch")
    from muon_adamw_hybrid_grad_gb300 import build

    build.build()
    from muon_adamw_hybrid_grad_gb300 import ops

    n, stride = 60, v + 5
    gen = torch.Generator(device="cuda").manual_seed(v)
    wide = 3 * torch.randn(n, stride, generator=gen, device="cuda")
    wide[::3] += 5000  # whose sums are formed again
    wide[1::6] = -float("inf")
    wide = wide.to(getattr(torch, dtype))
    z = wide[:, first:first + v]
    ids = torch.randint(0, v, (n,), generator=gen, device="cuda")
    l, h = (torch.randn(n, generator=gen, device="cuda") for _ in range(2))
    _, entropy, lse, _, _ = ops.token_logprobs(z, ids)
    want = ops.token_logprobs_backward(l, h, z, ids, entropy, lse)
    before = wide.clone()
    d = mx.TokenLogprobs(n_tokens=n, vocab=v, stride=stride, dtype=1 if dtype == "bfloat16" else 0, id_bytes=8, scale=1.0,
                         logits=z.data_ptr(), ids=ids.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    assert mx.load_library().muon_adamw_token_logprobs_backward(
        ctypes.byref(d), l.data_ptr(), h.data_ptr(), entropy.data_ptr(), lse.data_ptr(), z.data_ptr(), stride, stream) == 0
    assert torch.equal(z, want)
    assert torch.equal(wide[:, :first], before[:, :first]) and torch.equal(wide[:, first + v:], before[:, first + v:])
