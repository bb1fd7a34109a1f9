"""A small next-token model of pre-norm blocks, trained with the operators beside the sharded step.

    tokens -> embedding -> blocks -> norm -> 8-bit linear (logits) -> cross entropy
    block: h += dropout(attention(norm(h))), h += dropout(mlp(norm(h)))

Queries and keys leave one projection's rows rotated by their positions; causal attention is
plain torch; each dropout adds onto the residual stream, and each norm's gradient joins it.
Products run on 8-bit operands, gradients go into fp32 main gradients, and AdamW updates
masters, states and bf16 copies of every tensor in one launch.  The update's number, which also
numbers the dropout masks, lives on the device, so that a step can be captured in a CUDA graph.

    python examples/block_training.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import fsdp_sharded_mixed_pass_gb300 as fsp  # noqa: E402


class PlainLinear:
    """``fsp.Fp8Linear``'s calls with fp32 products in torch."""

    def __init__(self, weight, train=True):
        self.weight = weight

    def update(self, weight):
        self.weight = weight

    def forward(self, x, out_dtype=None):
        return x.float() @ self.weight.float().t()

    def backward(self, x, grad_out, grad_weight, accumulate=True):
        grad_weight.addmm_(grad_out.flatten(0, -2).float().t(), x.flatten(0, -2).float(), beta=1 if accumulate else 0)
        return grad_out.float() @ self.weight.float()


class Block:
    """``params`` and ``grads``: dicts of this block's tensors (norms fp32, products' weights)."""

    def __init__(self, params, grads, heads: int, p: float, seed: int, linear=fsp.Fp8Linear):
        self.params, self.grads, self.heads, self.p, self.seed = params, grads, heads, p, seed
        self.head_dim = params["proj"].shape[0] // heads
        self.rope = fsp.Rotary(self.head_dim)
        self.linear = {k: linear(params[k], train=True) for k in ("qkv", "proj", "up", "down")}

    def forward(self, h, positions, call):
        """The block's output and what ``backward`` needs; h: (batch, tokens, width)."""
        b, t, _ = h.shape
        n1, s1 = fsp.layer_norm(h, self.params["norm1"], self.params["bias1"], stats=True)
        qkv = self.linear["qkv"].forward(n1).view(b, t, 3 * self.heads, self.head_dim)
        q, k, v = qkv.split(self.heads, 2)
        q, k = self.rope.forward((q, k), positions)
        q, k, v = (x.float().transpose(1, 2) for x in (q, k, v))   # (batch, heads, tokens, head_dim)
        later = torch.ones(t, t, dtype=torch.bool, device=h.device).triu(1)
        probs = (q @ k.transpose(2, 3) * self.head_dim ** -0.5).masked_fill(later, float("-inf")).softmax(-1)
        o = (probs @ v).transpose(1, 2).reshape(h.shape)
        h2 = fsp.dropout(self.linear["proj"].forward(o), self.p, self.seed, call, residual=h)
        n2, s2 = fsp.layer_norm(h2, self.params["norm2"], center=False, stats=True)
        a = self.linear["up"].forward(n2)
        r = torch.relu(a)
        out = fsp.dropout(self.linear["down"].forward(r), self.p, self.seed + 1, call, residual=h2)
        return out, (h, s1, n1, q, k, v, probs, o, h2, s2, n2, r, positions, call)

    def backward(self, grad, saved, accumulate: bool):
        """The gradient of h; adds to (or, without ``accumulate``, replaces) the main gradients."""
        h, s1, n1, q, k, v, probs, o, h2, s2, n2, r, positions, call = saved
        g, kind = self.grads, dict(accumulate=accumulate)
        dz = fsp.dropout_backward(grad, self.p, self.seed + 1, call)
        da = self.linear["down"].backward(r, dz, g["down"], **kind) * (r > 0)
        dn2 = self.linear["up"].backward(n2, da, g["up"], **kind)
        dh2 = fsp.layer_norm_backward(h2, s2, dn2, self.params["norm2"], center=False, grad_weight=g["norm2"], add=grad, **kind)
        do = self.linear["proj"].backward(o, fsp.dropout_backward(dh2, self.p, self.seed, call), g["proj"], **kind)
        do = do.float().view(*h.shape[:2], self.heads, self.head_dim).transpose(1, 2)
        dv, dp = probs.transpose(2, 3) @ do, do @ v.transpose(2, 3)
        ds = probs * (dp - (probs * dp).sum(-1, keepdim=True)) * self.head_dim ** -0.5
        dqkv = torch.empty(*h.shape[:2], 3, self.heads, self.head_dim, device=h.device)
        dq, dk = ((x @ y).transpose(1, 2) for x, y in ((ds, k), (ds.transpose(2, 3), q)))
        self.rope.backward((dq, dk), positions, out=(dqkv[:, :, 0], dqkv[:, :, 1]))
        dqkv[:, :, 2] = dv.transpose(1, 2)
        dn1 = self.linear["qkv"].backward(n1, dqkv.flatten(2), g["qkv"], **kind)
        return fsp.layer_norm_backward(h, s1, dn1, self.params["norm1"], grad_weight=g["norm1"], grad_bias=g["bias1"], add=dh2, **kind)


class Model:
    def __init__(self, vocab=1000, width=128, heads=4, blocks=2, p=0.1, lr=3e-3, seed=0, linear=fsp.Fp8Linear):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        matrix = lambda *s: torch.randn(s, generator=gen, device="cuda") * s[1] ** -0.5  # noqa: E731
        ones = lambda: torch.ones(width, device="cuda")  # noqa: E731
        self.masters = {"embedding": matrix(vocab, width), "norm": ones(), "head": matrix(vocab, width)}
        for i in range(blocks):
            self.masters |= {f"{i}.norm1": ones(), f"{i}.bias1": torch.zeros(width, device="cuda"), f"{i}.qkv": matrix(3 * width, width),
                             f"{i}.proj": matrix(width, width), f"{i}.norm2": ones(), f"{i}.up": matrix(4 * width, width),
                             f"{i}.down": matrix(width, 4 * width)}
        self.copies = {k: m.bfloat16() if m.dim() == 2 else None for k, m in self.masters.items()}
        self.grads = {k: torch.zeros_like(m) for k, m in self.masters.items()}
        read = {k: m if self.copies[k] is None else self.copies[k] for k, m in self.masters.items()}
        of = lambda d, i: {k.split(".")[1]: v for k, v in d.items() if k.startswith(f"{i}.")}  # noqa: E731
        self.blocks = [Block(of(read, i), of(self.grads, i), heads, p, 1000 * seed + 2 * i, linear) for i in range(blocks)]
        self.read, self.head = read, linear(read["head"], train=True)
        self.opt = fsp.TensorAdamW(self.masters.values(), self.grads.values(), self.copies.values(), lr=lr, capturable=True)
        self.call = torch.zeros(1, dtype=torch.int64, device="cuda")   # numbers the dropout masks

    def gradients(self, tokens, targets, accumulate=False):
        """The mean loss; its gradients go to the main gradients."""
        positions = torch.arange(tokens.shape[1], device="cuda")
        h = fsp.embedding(self.read["embedding"], tokens, out_dtype=torch.float32)
        saved = []
        for block in self.blocks:
            h, s = block.forward(h, positions, self.call)
            saved.append(s)
        n, stats = fsp.layer_norm(h, self.read["norm"], center=False, stats=True)
        log_p = self.head.forward(n, out_dtype=torch.float32).log_softmax(-1)
        loss = -log_p.gather(-1, targets[..., None]).mean()
        d = log_p.exp_().scatter_add_(-1, targets[..., None], torch.full_like(log_p[..., :1], -1.0)).mul_(1 / tokens.numel())
        dn = self.head.backward(n, d, self.grads["head"], accumulate=accumulate)
        grad = fsp.layer_norm_backward(h, stats, dn, self.read["norm"], center=False, grad_weight=self.grads["norm"], accumulate=accumulate)
        for block, s in zip(reversed(self.blocks), reversed(saved)):
            grad = block.backward(grad, s, accumulate)
        fsp.embedding_backward(tokens, grad, self.grads["embedding"], accumulate=accumulate)
        return loss

    def step(self, tokens, targets):
        loss = self.gradients(tokens, targets)
        self.opt.step()
        self.call += 1
        for block in self.blocks:
            for k, layer in block.linear.items():
                layer.update(block.params[k])
        self.head.update(self.read["head"])
        return loss


def train(steps: int = 60, batch: int = 32, length: int = 64, vocab: int = 1000) -> list:
    """Losses of ``steps`` updates on a fixed successor table (each token's next one)."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    successor = torch.randperm(vocab, generator=gen, device="cuda")
    model, losses = Model(vocab), []
    for _ in range(steps):
        tokens = torch.randint(0, vocab, (batch, length), generator=gen, device="cuda")
        losses.append(model.step(tokens, successor[tokens]))
    return torch.stack(losses).tolist()


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    for i, loss in enumerate(train(ap.parse_args().steps)):
        if i % 10 == 0:
            print(f"step {i:4d}  loss {loss:.4f}")
    if bits := fsp.device_error():
        sys.exit(f"device error word {bits}")


if __name__ == "__main__":
    main()
