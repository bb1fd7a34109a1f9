"""The operators together: the small next-token model of examples/."""
import os
import sys

import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp
from oracle import step as OS

from gpu_cases import ensure_built
from ops_reference import embedding_gradient, fp8

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def test_the_example_learns_its_table_with_either_state():
    from low_precision_training import train
    runs = {bits: train(steps=60, state_bits=bits) for bits in (8, 32)}
    for losses in runs.values():
        # uniform guessing over 1000 tokens costs ln 1000 = 6.9; a learnt table nothing
        assert losses[0] > 6 and losses[-1] < 1
    # the same data and start: 8-bit states follow 32-bit ones
    assert abs(runs[8][10] - runs[32][10]) < 0.1 * runs[32][10]
    assert fsp.device_error() == 0


def test_the_example_repeats_bit_for_bit():
    from low_precision_training import train
    assert train(steps=5) == train(steps=5)


def test_gradients_against_the_same_model_in_64_bits():
    """One micro-batch's gradients against the example's formulas in 64 bits, with the
    same roundings (bf16 between the products, 8-bit operands).  What differs is the
    sums' last bits: 2^-20 of a value, which moves a bf16 rounding (2^-8 apart) of one
    element in 2000, and with it one 8-bit code (2^-3.5 apart) in 25 of those: 4e-4 rms
    per product.  Four products in a row, and a margin of four: 2^-7."""
    from low_precision_training import Model
    bf = lambda x: OS.bf16_bits_to_f32(OS.bf16_rne(x.astype(np.float32))).astype(np.float64)  # noqa: E731
    model = Model(300, 64, 96, 8, 1e-3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    tokens = torch.randint(0, 300, (500,), generator=gen, device="cuda")
    targets = torch.randint(0, 300, (500,), generator=gen, device="cuda")
    loss = model.micro_batch(tokens, targets, 1.0, first=True)
    w = {k: c.float().cpu().numpy().astype(np.float64) for k, c in model.copies.items()}
    t, y = tokens.cpu().numpy(), targets.cpu().numpy()
    x = bf(w["embedding"][t] * model.scale)
    pre = bf(fp8(x) @ fp8(w["up"]).T)
    act = np.maximum(pre, 0)
    logits = fp8(act) @ fp8(w["head"]).T
    log_p = logits - np.log(np.exp(logits).sum(1, keepdims=True))
    want_loss = -log_p[np.arange(500), y].mean()
    d = np.exp(log_p)
    d[np.arange(500), y] -= 1
    d = bf(d / 500)
    d_act = bf(fp8(d) @ fp8(w["head"].T).T)
    d_pre = np.where(pre > 0, d_act, 0)
    d_x = bf(fp8(d_pre) @ fp8(w["up"].T).T)
    want = {"head": fp8(d.T) @ fp8(act.T).T, "up": fp8(d_pre.T) @ fp8(x.T).T,
            "embedding": embedding_gradient(t, d_x, 300, model.scale)[0]}
    assert abs(float(loss) - want_loss) < 2.0 ** -7 * want_loss
    for k, g in model.grads.items():
        got = g.cpu().numpy().astype(np.float64)
        assert np.linalg.norm(got - want[k]) < 2.0 ** -7 * np.linalg.norm(want[k]), k


@pytest.mark.parametrize("mode", ["fsdp2", "distopt"])
def test_the_operators_between_sharded_steps(mode):
    """Two ranks' training steps on the buffers of the sharded update: the embedding and
    the 8-bit layers read what the step gathered, their gradients (two micro-batches, the
    second accumulated) go into the ranks' main-grad buffers, and the step averages those.
    Beside it AdamW over the list of the same tensors, given the averaged gradients."""
    vocab, dim, hidden, ranks = 257, 64, 96, 2
    shapes = [(vocab, dim), (hidden, dim), (vocab, hidden)]
    gen = torch.Generator(device="cuda").manual_seed(3)
    opt = fsp.ShardedAdamW(shapes, ranks, mode=mode, lr=3e-3, betas=(0.9, 0.95), weight_decay=0.01)
    cut = lambda buf: [buf[o:o + r * c].view(r, c) for o, (r, c) in zip(opt.plan.param_offsets, shapes)]  # noqa: E731
    zeros = lambda dt: torch.zeros(opt.plan.full_len_padded, dtype=dt, device="cuda")  # noqa: E731
    params, grads, full = [zeros(torch.bfloat16) for _ in range(ranks)], [zeros(torch.float32) for _ in range(ranks)], zeros(torch.float32)
    for w in cut(full):
        w.copy_(torch.randn(w.shape, generator=gen, device="cuda") * w.shape[1] ** -0.5)
    opt.load_full(full)
    opt.unshard(params)
    mean = [torch.zeros(s, device="cuda") for s in shapes]
    copies = [w.clone() for w in cut(params[0])]
    listed = fsp.TensorAdamW([w.clone() for w in cut(full)], mean, copies, lr=3e-3, betas=(0.9, 0.95), weight_decay=0.01)
    layers = [(fsp.Fp8Linear(cut(p)[1], train=True), fsp.Fp8Linear(cut(p)[2], train=True)) for p in params]
    successor = torch.randperm(vocab, generator=gen, device="cuda")
    losses = []
    for _ in range(60):
        total = 0.0
        for q in range(ranks):
            (table, w_up, w_head), (g_table, g_up, g_head), (up, head) = cut(params[q]), cut(grads[q]), layers[q]
            up.update(w_up)
            head.update(w_head)
            for micro in range(2):
                tokens = torch.randint(0, vocab, (300,), generator=gen, device="cuda")
                x = fsp.embedding(table, tokens, scale=dim ** 0.5)
                pre = up.forward(x)
                act = torch.relu(pre)
                logits = head.forward(act, out_dtype=torch.float32)
                log_p = logits - logits.logsumexp(-1, keepdim=True)
                rows = torch.arange(300, device="cuda")
                total = total - log_p[rows, successor[tokens]].mean() / (2 * ranks)
                d = log_p.exp_()
                d[rows, successor[tokens]] -= 1
                d_act = head.backward(act, (d / 600).bfloat16(), g_head, accumulate=micro > 0)
                d_x = up.backward(x, torch.where(pre > 0, d_act, torch.zeros_like(d_act)), g_up, accumulate=micro > 0)
                fsp.embedding_backward(tokens, d_x, g_table, scale=dim ** 0.5, accumulate=micro > 0)
        losses.append(total)
        for m, a, b in zip(mean, cut(grads[0]), cut(grads[1])):
            torch.add(a, b, out=m).mul_(0.5)
        opt.step(grads, params)
        listed.step()
        for q in range(ranks):   # every rank's gathered copy: the list's, bit for bit
            for w, c in zip(cut(params[q]), copies):
                assert torch.equal(w, c)
    # uniform guessing over 257 tokens costs ln 257 = 5.5; a learnt table nothing
    assert losses[0] > 5 and losses[-1] < 1
    assert fsp.device_error() == 0
