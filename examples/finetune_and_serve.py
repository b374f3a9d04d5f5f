"""Fine-tuning two adapters of one frozen int8 block, and serving both at once.

    python examples/finetune_and_serve.py [--steps 60]

The block is y = x + down(SiLU(up(norm(x)))), its projections frozen in int8 with
two low-rank adapters each. Every training batch holds sequences of two tenants,
whose targets differ; one AdamW step with 8-bit states updates the norm and both
tenants' adapters. Afterwards single tokens of both tenants (and of one without an
adapter) go through the block in one batch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int8_quantized_linear_rowwise_amd as I8  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, width: int, hidden: int, adapters: int, rank: int, seed: int, device="cuda:0"):
        super().__init__()
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return torch.randn((n, k), generator=g, device=device) * k ** -0.5

        kw = dict(adapters=adapters, rank=rank, alpha=2.0 * rank, dtype=torch.bfloat16)
        self.norm = I8.LayerNorm(width, device=device)
        self.up = I8.Int8LoraLinear(weight(hidden, width), **kw)
        self.down = I8.Int8LoraLinear(weight(width, hidden), **kw)

    def forward(self, x, seg_offsets=None, seg_adapter=None):
        h = self.up(self.norm(x), seg_offsets, seg_adapter)
        return x + self.down(torch.nn.functional.silu(h), seg_offsets, seg_adapter)


def main(steps: int = 60, width: int = 256, hidden: int = 704, tokens: int = 192, rank: int = 16):
    dev = "cuda:0"
    torch.manual_seed(0)
    block = Block(width, hidden, adapters=2, rank=rank, seed=1)
    teachers = [Block(width, hidden, adapters=1, rank=rank, seed=1) for _ in range(2)]
    with torch.no_grad():
        for t in teachers:                     # a tenant's target: the same block with weights of its own
            for p in (t.up.lora_B, t.down.lora_B):
                p.normal_(0, 0.1)
    # two sequences of either tenant, of different lengths
    off = torch.tensor([0, tokens // 4, tokens // 2, tokens - 24, tokens], dtype=torch.int32, device=dev)
    ids = torch.tensor([0, 1, 0, 1], dtype=torch.int32, device=dev)
    bounds = off.tolist()
    opt = I8.AdamW(block.parameters(), lr=4e-3, weight_decay=0.0, state_bits=8, master=True)
    losses = []
    for _ in range(steps):
        x = torch.randn((tokens, width), device=dev).to(torch.bfloat16)
        with torch.no_grad():
            want = torch.cat([teachers[a](x[lo:hi]) for lo, hi, a in zip(bounds, bounds[1:], ids.tolist())])
        loss = (block(x, off, ids) - want).float().square().mean()
        opt.zero_grad(set_to_none=False)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    losses = torch.stack(losses).tolist()

    # serving: one token of each of five requests, tenants in any order, one request without an adapter
    block.requires_grad_(False)
    x = torch.randn((5, width), device=dev).to(torch.bfloat16)
    one = torch.arange(6, dtype=torch.int32, device=dev)
    who = torch.tensor([1, 0, -1, 1, 0], dtype=torch.int32, device=dev)
    served = block(x, one, who)
    alone = torch.cat([block(x[i:i + 1], one[:2], who[i:i + 1]) for i in range(5)])
    return losses, served, alone


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    losses, served, alone = main(ap.parse_args().steps)
    print("loss:", " ".join(f"{x:.4f}" for x in losses[:: max(1, len(losses) // 10)] + losses[-1:]))
    print("served in one batch and alone, largest difference:", float((served - alone).abs().max()))
