"""A small next-token model trained with the operators beside the sharded step.

    tokens -> embedding (bf16 table, scaled) -> 8-bit linear + ReLU -> 8-bit linear
    (logits) -> cross entropy

The forward pass reads bf16 copies of the fp32 masters; gradients go into fp32
main gradients (the second half of a batch added to the first's); AdamW updates
masters, states and copies of every tensor in one launch, its gradients scaled by
a clip coefficient that never leaves the device.

    python examples/low_precision_training.py [--steps N] [--state-bits 8|32]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fsdp_sharded_mixed_pass_gb300 as fsp  # noqa: E402


class Model:
    """Masters, copies and main gradients of an embedding and two linear layers."""

    def __init__(self, vocab: int, dim: int, hidden: int, state_bits: int, lr: float, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        shapes = {"embedding": (vocab, dim), "up": (hidden, dim), "head": (vocab, hidden)}
        self.masters = {k: torch.randn(s, generator=gen, device="cuda") * s[1] ** -0.5 for k, s in shapes.items()}
        self.copies = {k: m.bfloat16() for k, m in self.masters.items()}
        self.grads = {k: torch.zeros_like(m) for k, m in self.masters.items()}
        self.scale = dim ** 0.5
        self.up = fsp.Fp8Linear(self.copies["up"], train=True)
        self.head = fsp.Fp8Linear(self.copies["head"], train=True)
        self.opt = fsp.TensorAdamW(self.masters.values(), self.grads.values(), self.copies.values(), lr=lr,
                                   betas=(0.9, 0.95), weight_decay=0.01, state_bits=state_bits)

    def micro_batch(self, tokens, targets, weight: float, first: bool):
        """Forward and backward; adds ``weight`` times the mean loss's gradient to the
        main gradients (``first``: replaces them) and returns the loss."""
        x = fsp.embedding(self.copies["embedding"], tokens, scale=self.scale)
        pre = self.up.forward(x)
        act = torch.relu(pre)
        logits = self.head.forward(act, out_dtype=torch.float32)
        log_p = logits - logits.logsumexp(-1, keepdim=True)
        rows = torch.arange(tokens.numel(), device="cuda")
        loss = -log_p[rows, targets].mean()
        d_logits = log_p.exp_()
        d_logits[rows, targets] -= 1
        d_logits *= weight / tokens.numel()
        d_act = self.head.backward(act, d_logits.bfloat16(), self.grads["head"], accumulate=not first)
        d_x = self.up.backward(x, torch.where(pre > 0, d_act, torch.zeros_like(d_act)), self.grads["up"],
                               accumulate=not first)
        fsp.embedding_backward(tokens, d_x, self.grads["embedding"], scale=self.scale, accumulate=not first)
        return loss

    def step(self, max_norm: float):
        norm = torch.stack([g.square().sum() for g in self.grads.values()]).sum().sqrt()
        self.opt.step(grad_scale=(max_norm / (norm + 1e-6)).clamp(max=1.0))
        self.up.update(self.copies["up"])
        self.head.update(self.copies["head"])


def train(steps: int = 60, state_bits: int = 8, vocab: int = 1000, dim: int = 128, hidden: int = 256, batch: int = 2048,
          lr: float = 3e-3, seed: int = 0) -> list:
    """Losses of ``steps`` updates on a fixed successor table (each token's next one)."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    successor = torch.randperm(vocab, generator=gen, device="cuda")
    model = Model(vocab, dim, hidden, state_bits, lr, seed)
    losses = []
    for _ in range(steps):
        tokens = torch.randint(0, vocab, (batch,), generator=gen, device="cuda")
        halves = tokens.chunk(2)
        parts = [model.micro_batch(t, successor[t], 0.5, first=i == 0) for i, t in enumerate(halves)]
        model.step(max_norm=1.0)
        losses.append(torch.stack(parts).mean())
    return torch.stack(losses).tolist()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps, a.state_bits)):
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i:4d}  loss {loss:.4f}")
    if bits := fsp.device_error():
        sys.exit(f"device error word {bits}")


if __name__ == "__main__":
    main()
