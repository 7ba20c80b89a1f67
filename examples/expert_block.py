"""A transformer layer with experts, trained with the operators' autograd forms and the optimizer.

A batch of packed samples goes through the embedding, attention, a layer of
experts and the output projection; dropout acts on both branches and inside
the experts, whose tokens are sorted by expert first. The loss is the mean
negative log probability of the next tokens with a bonus for entropy. Autograd
adds its gradients to the buffers that the optimizer has registered (each
expert's matrix is a parameter of its own), and MuonAdamW steps on them.

    python examples/expert_block.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import muon_adamw_hybrid_grad_gb300 as mx  # noqa: E402
from muon_adamw_hybrid_grad_gb300 import ops  # noqa: E402

VOCAB, WIDTH, HEADS, KV_HEADS, DIM = 1000, 256, 4, 2, 64
EXPERTS, HIDDEN = 5, 384
LENGTHS = (200, 1, 77, 130)
WINDOW, SINKS, DROP, BONUS = 64, 4, 0.1, 0.01


class Layer:
    """Parameters (fp32 masters, bf16 copies, gradients) and the optimizer that holds them."""

    def __init__(self, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shapes = {
            "embed_tokens.weight": (VOCAB, WIDTH),
            "layers.0.attn.qkv.weight": ((HEADS + 2 * KV_HEADS) * DIM, WIDTH),
            "layers.0.attn.o.weight": (WIDTH, HEADS * DIM),
            "layers.0.experts.up.weight": (EXPERTS, HIDDEN, WIDTH),
            "layers.0.experts.down.weight": (EXPERTS, WIDTH, HIDDEN),
            "lm_head.weight": (VOCAB, WIDTH),
            "layers.0.attn.q_norm.weight": (DIM,),
            "layers.0.attn.k_norm.weight": (DIM,),
            "layers.0.input_norm.weight": (WIDTH,),
            "layers.0.post_attention_norm.weight": (WIDTH,),
            "norm.weight": (WIDTH,),
        }
        self.leaf, entries = {}, []
        for name, shape in shapes.items():
            if len(shape) == 1:  # norms stay in fp32
                master = leaf = torch.ones(shape, device="cuda")
            else:
                master = torch.randn(shape, generator=gen, device="cuda") * 0.05
                leaf = master.bfloat16()
            grad = torch.zeros_like(leaf)
            shadow = None if leaf is master else leaf
            full = "model.action_expert." + name
            if len(shape) == 3:
                entries += [(f"{full}.{e}", master[e], grad[e], shadow[e]) for e in range(EXPERTS)]
            else:
                entries.append((full, master, grad, shadow))
            leaf.requires_grad_()
            leaf.grad = grad  # where autograd adds
            self.leaf[name.removeprefix("layers.0.").removesuffix(".weight")] = leaf
        self.opt = mx.MuonAdamW(entries)
        angle = torch.arange(max(LENGTHS), device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, DIM, 2, device="cuda") / DIM)
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()

    def loss(self, batch, rng) -> torch.Tensor:
        p, n = self.leaf, len(batch["ids"])
        drop = {"p": DROP, "rng": rng}
        x = ops.embedding_autograd(p["embed_tokens"], batch["ids"], scale=WIDTH ** 0.5)
        h, res = ops.residual_norm_autograd(x, None, p["input_norm"])
        qkv = (h @ p["attn.qkv"].T).view(n, HEADS + 2 * KV_HEADS, DIM)
        q, k = ops.qk_norm_rope_autograd(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], p["attn.q_norm"],
                                         p["attn.k_norm"], self.cos, self.sin, batch["positions"])
        out = ops.window_attention_autograd(q, k, qkv[:, HEADS + KV_HEADS:], window=WINDOW, sinks=SINKS,
                                            cu_seqlens=batch["cu_seqlens"])
        h, res = ops.residual_norm_autograd(out.flatten(1) @ p["attn.o"].T, res, p["post_attention_norm"], site=0, **drop)
        order, offsets = batch["order"], batch["offsets"]
        up = ops.expert_matmul_autograd(h[order], p["experts.up"], offsets)
        act = ops.dropout_autograd(up.relu().square(), DROP, rng, site=1)
        down = ops.expert_matmul_autograd(act, p["experts.down"], offsets)
        branch = torch.zeros_like(down).index_copy(0, order, down)
        h, _ = ops.residual_norm_autograd(branch, res, p["norm"], site=2, **drop)
        logprobs, entropy, _, _ = ops.token_logprobs_autograd(h @ p["lm_head"].T, batch["targets"], top=4)
        return -(logprobs + BONUS * entropy).mean()

    def step(self, batch, rng, lr: float) -> torch.Tensor:
        for leaf in self.leaf.values():
            leaf.grad.zero_()
        loss = self.loss(batch, rng)
        loss.backward()
        self.opt.step(lr)
        return loss.detach()


def make_batch(seed: int = 1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(LENGTHS)
    ids = torch.randint(0, VOCAB, (n,), generator=gen, device="cuda")
    ids[::17] = -1  # positions that hold no token
    targets = ids.roll(-1)
    bounds = torch.tensor([sum(LENGTHS[:i]) for i in range(len(LENGTHS) + 1)], device="cuda", dtype=torch.int32)
    targets[bounds[1:].long() - 1] = -1  # a sample's last token has no next one
    expert = ids.clamp(min=0) % EXPERTS  # the router of this example; expert 0 takes the empty positions too
    counts = torch.zeros(EXPERTS + 1, device="cuda", dtype=torch.int64).scatter_add_(0, expert + 1, torch.ones_like(expert))
    return {"ids": ids, "targets": targets, "cu_seqlens": bounds, "order": expert.argsort(stable=True),
            "offsets": counts.cumsum(0).to(torch.int32),
            "positions": torch.cat([torch.arange(m, device="cuda") for m in LENGTHS])}


def run(steps: int = 20, lr: float = 3e-3, seed: int = 0):
    """The losses of `steps` steps on one batch."""
    layer, batch = Layer(seed), make_batch(seed + 1)
    losses = [layer.step(batch, torch.tensor([seed, i], device="cuda"), lr) for i in range(steps)]
    ops.check()
    layer.opt.close()
    return [float(x) for x in losses]


if __name__ == "__main__":
    for i, loss in enumerate(run(int(sys.argv[1]) if len(sys.argv) > 1 else 20)):
        print(f"step {i}: loss {loss:.4f}")
