"""One attention block trained with the operators and the optimizer.

A batch of packed samples goes through the embedding, a fused query/key/value
projection, the norm and rotation of queries and keys, and sliding-window
attention with sinks; the mean squared error against random targets comes back
through the operators' gradients into the buffers that the optimizer has
registered, and MuonAdamW steps on them. The projections are plain matrix
products of torch.

    python examples/attention_block.py [steps]
"""
from __future__ import annotations

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import muon_adamw_hybrid_grad_gb300 as mx  # noqa: E402
from muon_adamw_hybrid_grad_gb300 import ops  # noqa: E402

VOCAB, WIDTH, HEADS, KV_HEADS, DIM = 1000, 256, 4, 2, 64
LENGTHS = (200, 1, 77, 130)
WINDOW, SINKS = 64, 4


class Block:
    """Parameters (fp32 masters, bf16 copies, gradients) and the optimizer that holds them."""

    def __init__(self, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shapes = {
            "model.action_expert.embed_tokens.weight": (VOCAB, WIDTH),
            "model.action_expert.layers.0.attn.qkv.weight": ((HEADS + 2 * KV_HEADS) * DIM, WIDTH),
            "model.action_expert.layers.0.attn.o.weight": (WIDTH, HEADS * DIM),
            "model.action_expert.layers.0.attn.q_norm.weight": (DIM,),
            "model.action_expert.layers.0.attn.k_norm.weight": (DIM,),
        }
        self.master, self.copy, self.grad = [], [], []
        for shape in shapes.values():
            p = (torch.ones(shape, device="cuda") if len(shape) == 1
                 else torch.randn(shape, generator=gen, device="cuda") * 0.05)
            self.master.append(p)
            self.copy.append(p.bfloat16())
            # the norms' gradients come in fp32, the others in bf16
            self.grad.append(torch.zeros(shape, device="cuda", dtype=torch.float32 if len(shape) == 1 else torch.bfloat16))
        self.opt = mx.MuonAdamW(list(zip(shapes, self.master, self.grad, self.copy)))
        angle = torch.arange(max(LENGTHS), device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(0, DIM, 2, device="cuda") / DIM)
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()

    def step(self, ids, positions, cu_seqlens, target, lr: float) -> torch.Tensor:
        embed, qkv_w, o_w, _, _ = self.copy
        q_norm, k_norm = self.master[3], self.master[4]
        how = {"window": WINDOW, "sinks": SINKS, "cu_seqlens": cu_seqlens}
        scale = math.sqrt(WIDTH)
        # forward
        x = ops.embedding(embed, ids, scale=scale)
        qkv = (x @ qkv_w.T).view(len(ids), HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        qr, kr = ops.qk_norm_rope(q, k, q_norm, k_norm, self.cos, self.sin, positions)
        out, lse = ops.window_attention(qr, kr, v, **how)
        flat = out.view(len(ids), -1)
        error = (flat @ o_w.T).float() - target
        # backward, into the registered gradients
        dy = (error * (2.0 / error.numel())).bfloat16()
        torch.matmul(dy.T, flat, out=self.grad[2])
        dqr, dkr, dv = ops.window_attention_backward((dy @ o_w).view_as(out), qr, kr, v, out, lse, **how)
        dq, dk, dqn, dkn = ops.qk_norm_rope_backward(dqr, dkr, q, k, q_norm, k_norm, self.cos, self.sin, positions)
        self.grad[3].copy_(dqn)
        self.grad[4].copy_(dkn)
        dqkv = torch.cat((dq, dk, dv), 1).flatten(1)
        torch.matmul(dqkv.T, x, out=self.grad[1])
        ops.embedding_backward(dqkv @ qkv_w, ids, self.grad[0], scale=scale)
        self.opt.step(lr)
        return error.square().mean()


def run(steps: int = 30, lr: float = 3e-3, seed: int = 0):
    """The losses of `steps` steps on one batch."""
    block = Block(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    n = sum(LENGTHS)
    ids = torch.randint(0, VOCAB, (n,), generator=gen, device="cuda")
    ids[::17] = -1  # positions that hold no token
    positions = torch.cat([torch.arange(m, device="cuda") for m in LENGTHS])
    cu_seqlens = torch.tensor([sum(LENGTHS[:i]) for i in range(len(LENGTHS) + 1)], device="cuda", dtype=torch.int32)
    target = torch.randn(n, WIDTH, generator=gen, device="cuda")
    losses = [block.step(ids, positions, cu_seqlens, target, lr) for _ in range(steps)]
    ops.check()
    block.opt.close()
    return [float(x) for x in losses]


if __name__ == "__main__":
    for i, loss in enumerate(run(int(sys.argv[1]) if len(sys.argv) > 1 else 30)):
        print(f"step {i}: loss {loss:.4f}")
