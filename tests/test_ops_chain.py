"""The operators of a transformer layer with experts, run together: examples/expert_block.py."""
import importlib.util
import math
import os

import pytest
from conftest import ROOT

from oracle import operators as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from muon_adamw_hybrid_grad_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("expert_block", os.path.join(ROOT, "examples", "expert_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def loss_in_64_bits(ex, layer, batch, rng):
    """The example's loss from plain operations, and its parameters as leaves."""
    p = {k: v.detach().double().requires_grad_() for k, v in layer.leaf.items()}
    n, seed, step = len(batch["ids"]), *rng.tolist()

    def drop(x, site):
        return x * torch.tensor(O.dropout_factors(x.numel(), ex.DROP, seed, step, site), device="cuda").view(x.shape)

    ids = batch["ids"]
    res = p["embed_tokens"][ids.clamp(min=0)] * (ids >= 0)[:, None] * ex.WIDTH ** 0.5
    qkv = (norm(res, p["input_norm"]) @ p["attn.qkv"].T).view(n, -1, ex.DIM)
    cos, sin = (t.double()[batch["positions"]][:, None] for t in (layer.cos, layer.sin))
    q = rotate(norm(qkv[:, :ex.HEADS], p["attn.q_norm"]), cos, sin)
    k = rotate(norm(qkv[:, ex.HEADS:ex.HEADS + ex.KV_HEADS], p["attn.k_norm"]), cos, sin)
    v = qkv[:, ex.HEADS + ex.KV_HEADS:]
    per = ex.HEADS // ex.KV_HEADS
    k, v = k.repeat_interleave(per, 1), v.repeat_interleave(per, 1)
    at = torch.arange(n, device="cuda")
    sample = torch.searchsorted(batch["cu_seqlens"].long(), at, right=True)
    back, pos = at[:, None] - at, batch["positions"]
    see = (sample[:, None] == sample) & (back >= 0) & ((back < ex.WINDOW) | (pos < ex.SINKS))
    s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(ex.DIM)
    out = torch.einsum("hij,jhd->ihd", torch.softmax(s.masked_fill(~see, -math.inf), -1), v)
    res = res + drop(out.flatten(1) @ p["attn.o"].T, 0)
    h, off = norm(res, p["post_attention_norm"])[batch["order"]], batch["offsets"].tolist()
    up = torch.cat([h[off[e]:off[e + 1]] @ p["experts.up"][e].T for e in range(ex.EXPERTS)])
    act = drop(up.relu().square(), 1)
    down = torch.cat([act[off[e]:off[e + 1]] @ p["experts.down"][e].T for e in range(ex.EXPERTS)])
    res = res + drop(torch.zeros_like(down).index_copy(0, batch["order"], down), 2)
    logp = torch.log_softmax(norm(res, p["norm"]) @ p["lm_head"].T, -1)
    t = batch["targets"]
    given = logp.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0)
    return -(given - ex.BONUS * (logp.exp() * logp).sum(-1)).mean(), p


def test_gradients_of_the_whole_layer(example):
    """Some two dozen tensors on the way there and back are rounded to bf16, by at most 2^-8 of their size each: the
    gradients' 2-norms may be off by the sum of these."""
    layer, batch, rng = example.Layer(3), example.make_batch(4), torch.tensor([11, 1 << 33], device="cuda")
    loss = layer.loss(batch, rng)
    loss.backward()
    want, p = loss_in_64_bits(example, layer, batch, rng)
    want.backward()
    assert abs(loss.item() - want.item()) <= 24 * O.UB * abs(want.item())
    for name, leaf in layer.leaf.items():
        off = float((leaf.grad.double() - p[name].grad).norm() / p[name].grad.norm())
        assert off <= 24 * O.UB, (name, off)
        assert leaf.grad.isfinite().all()
    layer.opt.close()


def test_example_runs(example):
    losses = example.run(6)
    assert len(losses) == 6 and all(math.isfinite(x) for x in losses)
    assert example.run(3) == losses[:3]


def test_step_in_a_graph(example):
    """Forward and backward captured once, replayed with a step that the graph counts up: each replay's gradients are the
    plain call's."""
    layer, batch = example.Layer(5), example.make_batch(6)
    rng = torch.tensor([7, 0], device="cuda")

    def grads():
        for leaf in layer.leaf.values():
            leaf.grad.zero_()
        layer.loss(batch, rng).backward()

    want = []
    for i in range(2):
        rng.copy_(torch.tensor([7, i], device="cuda"))
        grads()
        want.append([leaf.grad.clone() for leaf in layer.leaf.values()])
    rng.zero_()
    rng[0] = 7
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads()
        rng[1].add_(1)
    for i in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert int(rng[1]) == i + 1
        for a, b in zip((leaf.grad for leaf in layer.leaf.values()), want[i]):
            assert torch.equal(a, b)
    layer.opt.close()
