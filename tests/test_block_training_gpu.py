"""The example of pre-norm blocks: its gradients, its capture in a CUDA graph, its run."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp

import block_reference as R
from gpu_cases import ensure_built

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _loss(model, params, tokens, targets):
    """The model in 64 bits for autograd, its masks from the generator's statement."""
    h = params["embedding"][tokens]
    b, t, width = h.shape

    def dropout(x, seed, p):
        lost = int(p * 65536 + 0.5)
        keep = torch.from_numpy(R.random16(x.numel(), seed, int(model.call)) >= lost).cuda().view(x.shape)
        return x * keep * (65536 / (65536 - lost))

    def norm(x, w, bias=0.0, center=False):
        x = x - x.mean(-1, keepdim=True) if center else x
        return x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + bias

    def rotate(x, block):
        angle = torch.arange(t, device="cuda", dtype=torch.float64)[:, None, None] * torch.tensor(block.rope.frequencies, device="cuda", dtype=torch.float64)
        u, v = x.chunk(2, -1)
        return torch.cat([u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()], -1)

    for i, block in enumerate(model.blocks):
        p = {k: params[f"{i}.{k}"] for k in block.params}
        q, k, v = (norm(h, p["norm1"], p["bias1"], True) @ p["qkv"].t()).view(b, t, 3 * block.heads, -1).split(block.heads, 2)
        q, k, v = (x.transpose(1, 2) for x in (rotate(q, block), rotate(k, block), v))
        mask = torch.full((t, t), -math.inf, device="cuda", dtype=torch.float64).triu(1)
        o = ((q @ k.transpose(2, 3) * block.head_dim ** -0.5 + mask).softmax(-1) @ v).transpose(1, 2).reshape(h.shape)
        h = h + dropout(o @ p["proj"].t(), block.seed, block.p)
        h = h + dropout(torch.relu(norm(h, p["norm2"]) @ p["up"].t()) @ p["down"].t(), block.seed + 1, block.p)
    logits = norm(h, params["norm"]) @ params["head"].t()
    return torch.nn.functional.cross_entropy(logits.flatten(0, 1), targets.flatten())


@pytest.mark.parametrize("width,heads,length", [(64, 2, 33), (96, 3, 16)])
def test_gradients(width, heads, length):
    from block_training import Model, PlainLinear
    model = Model(vocab=211, width=width, heads=heads, blocks=2, p=0.2, linear=PlainLinear, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(0)
    for name, m in model.masters.items():   # norms away from ones and zeros
        if m.dim() == 1:
            m.add_(torch.randn(width, generator=gen, device="cuda") * 0.2)
    tokens, targets = torch.randint(0, 211, (2, 3, length), generator=gen, device="cuda")
    model.call.fill_(41)
    params = {k: v.double().requires_grad_() for k, v in model.read.items()}
    want = _loss(model, params, tokens, targets)
    want.backward()
    loss = model.gradients(tokens, targets)
    # some 20 stages, each within 64 roundings (2^-24) of its operands' size, none of which the next enlarges more than
    # tenfold: 20 * 64 * 2^-24 * 10, below 2^-10 of a gradient's norm
    assert abs(float(loss) - float(want.detach())) <= 2.0 ** -10 * float(want.detach())
    for k, p in params.items():
        assert float((model.grads[k] - p.grad).norm()) <= 2.0 ** -10 * float(p.grad.norm()), k
    first = {k: g.clone() for k, g in model.grads.items()}
    model.gradients(tokens, targets, accumulate=True)   # a second micro-batch's adds to them
    for k, g in model.grads.items():
        assert float((g - 2 * first[k]).norm()) <= 2.0 ** -20 * float(first[k].norm()), k
    assert fsp.device_error() == 0


def test_a_captured_step_replays():
    """A step in a CUDA graph: the update's and the masks' numbers advance on the device, as eager steps' do."""
    from block_training import Model
    gen = torch.Generator(device="cuda").manual_seed(5)
    batches = torch.randint(0, 1000, (4, 4, 32), generator=gen, device="cuda")
    eager, captured = Model(seed=7), Model(seed=7)
    for x in batches:
        eager.step(x, (x + 1) % 1000)
    x = batches[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        captured.step(x, (x + 1) % 1000)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step(x, (x + 1) % 1000)
    for b in batches[1:]:
        x.copy_(b)
        graph.replay()
    assert int(captured.call) == int(eager.call) == 4 and captured.opt.t == eager.opt.t == 4
    # the products' and sums' own order aside, which torch's library may choose anew: a few steps of bf16 copies
    for k, m in eager.masters.items():
        assert float((captured.masters[k] - m).abs().max()) <= 4 * 3e-3 * 2, k   # (no element moves further than lr a step)
        assert float((captured.masters[k] - m).norm()) <= 2.0 ** -6 * float(m.norm()), k
    assert fsp.device_error() == 0


@pytest.mark.parametrize("width,heads,dtype", [(512, 8, torch.float32), (513, 9, torch.bfloat16), (1001, 7, torch.bfloat16), (1002, 6, torch.bfloat16),
                                               (777, 7, torch.float32)])
def test_calls_that_follow_one_another_at_once(width, heads, dtype):
    """Each call starts while the one before it ends: a chain of calls in place gives what waiting after each gives.
    (Odd rows share pieces of memory with the rows beside them, which other CTAs write.)"""
    gen = torch.Generator(device="cuda").manual_seed(9)
    rope = fsp.Rotary(width // heads // 2 * 2)

    def chain(wait):
        done = torch.cuda.synchronize if wait else lambda: None
        h = torch.randn(3000, width, generator=gen.manual_seed(1), device="cuda").to(dtype)
        w, dw = torch.rand(width, generator=gen, device="cuda") + 0.5, torch.zeros(width, device="cuda")
        pos = torch.arange(3000, device="cuda")
        grad = torch.randn(3000, width, generator=gen, device="cuda").to(dtype)
        for k in range(6):
            n, stats = fsp.layer_norm(h, w, stats=True)
            done()
            rope.forward(n.view(3000, heads, -1), pos, out=n.view(3000, heads, -1))
            done()
            fsp.dropout(n, 0.3, 5, k, residual=h, out=h)
            done()
            fsp.layer_norm_backward(n, stats, grad, w, grad_weight=dw, accumulate=True, add=h, out=grad)
            done()
            fsp.layer_norm(grad, out=grad)
            done()
        return h, grad, dw

    want = chain(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
    # the same on two streams side by side
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            got.append(chain(False))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    assert fsp.device_error() == 0


def test_it_runs():
    from block_training import train
    losses = train(steps=4, batch=4, length=16, vocab=100)
    assert len(losses) == 4 and all(np.isfinite(losses)) and fsp.device_error() == 0
