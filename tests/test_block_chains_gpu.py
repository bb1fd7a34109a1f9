"""Calls of the block's operators that run into one another on the GPU, and what they write beside their results."""
import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp

from block_cases import DT, matrix
from gpu_cases import ensure_built
from test_layer_norm_gpu import EPS, MANY, SIZES, TYPES, _inputs, _vector

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


class Chain:
    """A chain of calls on buffers of its own, each of which reads what the one before it wrote, most of them in place.
    ``run`` makes them; with ``wait`` each ends before the next begins."""

    def __init__(self, rows, width, heads, dtype, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.rows, self.heads, self.rope = rows, heads, fsp.Rotary(width // heads // 2 * 2)
        self.h0, self.grad0 = rand(rows, width).to(dtype), rand(rows, width).to(dtype)
        self.h, self.grad, self.n = (torch.empty_like(self.h0) for _ in range(3))
        self.w, self.b, self.dw, self.db = rand(width) * 0.2 + 1, rand(width), torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
        self.stats, self.pos = torch.empty(rows, 2, device="cuda"), torch.arange(rows, device="cuda")
        self.call = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.work = torch.empty(fsp.layer_norm_backward_workspace_bytes(rows, width), dtype=torch.uint8, device="cuda")

    def run(self, wait=False):
        done = torch.cuda.synchronize if wait else lambda: None
        heads = self.n.view(self.rows, self.heads, -1)
        self.h.copy_(self.h0)
        self.grad.copy_(self.grad0)
        self.dw.zero_()
        self.db.zero_()
        self.call.zero_()
        done()
        for k in range(5):
            fsp.layer_norm(self.h, self.w, self.b, out=self.n, stats=self.stats)
            done()
            self.rope.forward(heads, self.pos, out=heads)
            done()
            fsp.dropout(self.n, 0.3, 5, self.call, residual=self.h, out=self.h)
            done()
            fsp.layer_norm_backward(self.n, self.stats, self.grad, self.w, grad_weight=self.dw, grad_bias=self.db, accumulate=True, add=self.h,
                                    out=self.grad, workspace=self.work)
            done()
            self.rope.backward(self.grad.view_as(heads), self.pos, out=self.grad.view_as(heads))
            done()
            fsp.layer_norm(self.grad, self.w, center=False, out=self.grad)
            done()
            fsp.dropout_backward(self.grad, 0.1, 6, k, out=self.grad)
            done()
            self.call.add_(1)
            done()

    def results(self):
        return [t.clone() for t in (self.h, self.grad, self.n, self.dw, self.db, self.stats, self.call)]


# rows at multiples of 16 bytes, even and odd ones; groups of 8 threads to 512; few rows and many
CHAINS = [(3000, 512, 8, "f32"), (3000, 513, 9, "bf16"), (3000, 1001, 7, "bf16"), (3000, 1002, 6, "bf16"), (2500, 777, 7, "f32"), (9000, 64, 1, "bf16"),
          (9001, 33, 1, "bf16"), (9001, 66, 1, "bf16"), (5000, 129, 1, "f32"), (100, 512, 4, "bf16"), (30, 1001, 7, "f32"), (400, 8192, 64, "bf16"),
          (300, 9999, 99, "bf16"), (40, 20000, 100, "bf16")]


@pytest.mark.parametrize("rows,width,heads,dtype", CHAINS)
def test_replays_of_a_chain(rows, width, heads, dtype):
    """Replayed from a graph, a launch follows the one before it on the GPU at once (eager calls of a few microseconds leave
    gaps of the host's time): bit for bit what waiting after each call gives."""
    chain = Chain(rows, width, heads, DT[dtype], 1)
    chain.run(wait=True)
    want = chain.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain.run()
    for _ in range(6):
        for t in (chain.n, chain.stats, chain.h, chain.grad):   # (nothing of an earlier replay helps)
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(chain.results(), want))
    graph.replay()
    graph.replay()   # back to back
    assert all(torch.equal(a, b) for a, b in zip(chain.results(), want)) and fsp.device_error() == 0


@pytest.mark.parametrize("rows,width,heads,dtype", [CHAINS[i] for i in (1, 2, 5, 7, 9, 12)])
def test_chains_side_by_side(rows, width, heads, dtype):
    """Two chains, each captured with a workspace of its own, replayed on two streams at the same time, many times over."""
    chains, graphs, want = [Chain(rows, width, heads, DT[dtype], seed) for seed in (2, 3)], [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for chain in chains:
        chain.run(wait=True)
        want.append(chain.results())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain.run()
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for chain, w in zip(chains, want):
        assert all(torch.equal(a, b) for a, b in zip(chain.results(), w))
    assert fsp.device_error() == 0


@pytest.mark.parametrize("x_t,out_t,par_t", TYPES)
@pytest.mark.parametrize("rows,dim,pad,shift", SIZES[::2] + MANY[1::3])
def test_results_do_not_depend_on_one_another(rows, dim, pad, shift, x_t, out_t, par_t):
    """Without statistics, without the parameters' gradients: the same bits, and nothing beside them is written."""
    rng = np.random.default_rng(rows * 19 + dim)
    x, x_ok = matrix(rows, dim, x_t, pad, shift, _inputs(rows, dim, rng))
    dy, dy_ok = matrix(rows, dim, out_t, pad, shift, rng.normal(0, 1, (rows, dim)))
    w, b = _vector(rng, dim, 1, 0.3, par_t), _vector(rng, dim, 0, 0.3, par_t)
    for center, bias, add in ((True, b, x), (False, None, None)):
        y, y_ok = matrix(rows, dim, out_t, pad, shift)
        again, again_ok = matrix(rows, dim, out_t, pad, shift)
        stats = fsp.layer_norm(x, w, bias, eps=EPS, center=center, out=y, stats=True)[1]
        fsp.layer_norm(x, w, bias, eps=EPS, center=center, out=again)
        assert torch.equal(y, again) and y_ok() and again_ok()
        dx, dx_ok = matrix(rows, dim, x_t, pad, shift)
        only, only_ok = matrix(rows, dim, x_t, pad, shift)
        dw, db = torch.empty(2, dim, device="cuda")
        fsp.layer_norm_backward(x, stats, dy, w, center=center, grad_weight=dw, grad_bias=db, add=add, out=dx)
        fsp.layer_norm_backward(x, stats, dy, w, center=center, add=add, out=only)
        assert torch.equal(dx, only) and dx_ok() and only_ok() and x_ok() and dy_ok()
        one = torch.empty_like(dw)
        fsp.layer_norm_backward(x, stats, dy, w, center=center, grad_weight=one, add=add, out=only)
        assert torch.equal(one, dw) and torch.equal(dx, only)
        fsp.layer_norm_backward(x, stats, dy, w, center=center, grad_bias=one, need_grad_x=False)
        assert torch.equal(one, db)
    assert fsp.device_error() == 0
