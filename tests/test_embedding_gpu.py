"""Embedding lookup with scaling and its gradient by sorted tokens."""
import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp
from oracle import step as OS

from gpu_cases import Guarded, ensure_built
from ops_reference import embedding_gradient, rounds_to

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
IX = {32: torch.int32, 64: torch.int64}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _values(x):
    return x.float().cpu().numpy()


def _matrix(rows, cols, dtype, pad=0, shift=0, values=None):
    """rows x cols with `pad` elements between rows, `shift` elements off
    alignment, in a guarded buffer; returns (tensor, guard, gaps-untouched check)."""
    n = rows * (cols + pad) + shift
    g = Guarded(n, DT[dtype], 0)
    t = g.t[shift:].view(rows, cols + pad)[:, :cols]
    if values is not None:
        t.copy_(torch.from_numpy(values.astype(np.float32)))
    return t, g


@pytest.mark.parametrize("weight,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("tokens,vocab,dim,pad,shift,index", [
    (1, 1, 1, 0, 0, 64), (1, 1000, 1024, 0, 0, 32), (7, 33, 8, 0, 0, 64), (9, 5, 517, 0, 0, 32), (300, 100, 64, 8, 0, 64),
    (65, 50, 256, 3, 0, 32), (33, 40, 24, 0, 1, 64), (2, 9, 2056, 0, 8, 32)])
def test_lookup_is_the_rounded_product(tokens, vocab, dim, pad, shift, index, weight, out):
    rng = np.random.default_rng(tokens + dim)
    w, _ = _matrix(vocab, dim, weight, pad, shift, rng.normal(0, 0.02, (vocab, dim)))
    ids = rng.integers(0, vocab, tokens)
    y, guard = _matrix(tokens, dim, out, pad, shift)
    scale = 22.627417
    got = fsp.embedding(w, torch.from_numpy(ids).to("cuda", IX[index]), scale=scale, out=y)
    assert got is y
    want = _values(w)[ids] * np.float32(scale)
    if out == "bf16":
        want = OS.bf16_bits_to_f32(OS.bf16_rne(want))
    assert np.array_equal(_values(y), want)
    if pad:
        assert float(guard.t[shift:].view(tokens, dim + pad)[:, dim:].abs().sum()) == 0
    assert guard.guards_intact() and fsp.device_error() == 0


def test_lookup_shapes_defaults_and_empties():
    w = torch.randn(10, 16, device="cuda")
    ids = torch.randint(0, 10, (3, 4), device="cuda")
    y = fsp.embedding(w, ids)
    assert y.shape == (3, 4, 16) and torch.equal(y, w[ids])
    assert fsp.embedding(w, ids, out_dtype=torch.bfloat16).dtype == torch.bfloat16
    assert fsp.embedding(w, ids[:0]).shape == (0, 4, 16)
    assert fsp.embedding(w[:, :0], ids).shape == (3, 4, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = fsp.embedding(w, ids, scale=2.0, stream=s)
    s.synchronize()
    assert torch.equal(z, 2 * w[ids])


def test_tokens_outside_the_table_are_reported():
    w = torch.randn(10, 16, device="cuda")
    ids = torch.tensor([1, -1, 10, 2, 2 ** 40], device="cuda")
    y = fsp.embedding(w, ids)
    assert torch.equal(y[[0, 3]], w[[1, 2]]) and float(y[[1, 2, 4]].abs().sum()) == 0
    assert fsp.device_error() == 16 and fsp.device_error() == 0
    dw = torch.full((10, 16), 7.0, device="cuda")
    fsp.embedding_backward(ids, torch.ones(5, 16, device="cuda"), dw)
    assert fsp.device_error() == 16
    want = torch.zeros(10, 16, device="cuda")
    want[[1, 2]] = 1
    assert torch.equal(dw, want)


def test_offsets_past_32_bits():
    rows = 2 ** 22 + 3   # x 1024 bf16 elements: 2^32 elements and more
    w = torch.zeros(rows, 1024, dtype=torch.bfloat16, device="cuda")
    w[-1] = 3
    ids = torch.tensor([rows - 1, 0], device="cuda")
    assert torch.equal(fsp.embedding(w, ids)[0], w[-1])
    dy = torch.ones(2, 1024, dtype=torch.bfloat16, device="cuda")
    fsp.embedding_backward(ids, dy, w, scale=0.5, accumulate=True)
    assert float(w[-1].float().mean()) == 3.5 and float(w[0].float().mean()) == 0.5 and float(w[1:-1].abs().amax()) == 0
    fsp.embedding_backward(ids, dy, w, scale=0.5)
    assert float(w[-1].float().mean()) == 0.5 and float(w[0].float().mean()) == 0.5 and float(w[1:-1].abs().amax()) == 0


# tokens, vocab, dim, pad, shift: one token to many; one row; chunk edges (32 pairs); odd and wide rows
GRAD = [(1, 1, 1, 0, 0), (1, 9, 64, 0, 0), (31, 7, 8, 0, 0), (32, 3, 12, 0, 0), (33, 1, 517, 0, 0), (64, 2, 40, 8, 0),
        (97, 1000, 33, 0, 0), (500, 30, 1024, 0, 0), (1000, 511, 96, 4, 4), (1000, 512, 96, 1, 1), (4096, 513, 16, 0, 0),
        (4097, 5003, 24, 0, 0), (5000, 1, 8, 0, 0), (9001, 262143, 4, 0, 0), (9001, 262144, 4, 0, 0), (300, 20, 3000, 0, 0), (3000, 70000, 1000, 0, 0)]


@pytest.mark.parametrize("grad,weight", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("tokens,vocab,dim,pad,shift", GRAD)
def test_gradient(tokens, vocab, dim, pad, shift, grad, weight):
    rng = np.random.default_rng(tokens * 7 + dim)
    for k, accumulate in enumerate((False, True)):
        # log-uniform: a few tokens hold much of the batch
        ids = np.minimum((np.exp(rng.uniform(0, np.log(vocab + 1), tokens)) - 1).astype(np.int64), vocab - 1)
        dy, _ = _matrix(tokens, dim, grad, pad, shift, rng.normal(0, 1, (tokens, dim)))
        dw, guard = _matrix(vocab, dim, weight, pad, shift, rng.normal(0, 1, (vocab, dim)))
        old = _values(dw)
        ids_d = torch.from_numpy(ids).to("cuda", IX[32 if k else 64])
        padding = int(ids[0]) if tokens > 2 and vocab > 1 and k else None
        fsp.embedding_backward(ids_d, dy, dw, scale=1.75, accumulate=accumulate, padding_idx=padding)
        got = _values(dw).astype(np.float64)
        want, mag, n = embedding_gradient(ids, _values(dy), vocab, 1.75, old if accumulate else None, padding)
        # n additions and the scaling, each at most 2^-24 of the magnitudes that enter it; the old value's addition
        tol = (n[:, None] + 2) * 2.0 ** -24 * mag + (2.0 ** -24 * np.abs(want) if accumulate else 0)
        if weight == "bf16":
            assert rounds_to(got, want, tol).all()
        else:
            assert (np.abs(got - want) <= tol).all()
        assert (got[n == 0] == (old[n == 0] if accumulate else 0)).all()
        if pad:
            assert float(guard.t[shift:].view(vocab, dim + pad)[:, dim:].abs().sum()) == 0
        assert guard.guards_intact() and fsp.device_error() == 0


def test_gradient_depends_on_the_inputs_alone():
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = (torch.rand(20000, generator=g, device="cuda") ** 4 * 3000).long()
    dy = torch.randn(20000, 72, generator=g, device="cuda")
    a, b = (torch.empty(3000, 72, device="cuda") for _ in range(2))
    fsp.embedding_backward(ids, dy, a)
    junk = torch.full((fsp.embedding_backward_workspace_bytes(3000, 72, 20000) + 100,), 0xFF, dtype=torch.uint8, device="cuda")
    fsp.embedding_backward(ids, dy, b, workspace=junk)
    assert torch.equal(a, b)


def test_gradient_against_differences():
    """<dW, D> is the difference quotient of L(W) = sum(dy * y(W)), which is linear in W."""
    rng = np.random.default_rng(0)
    w, d = rng.integers(-8, 9, (2, 50, 12)).astype(np.float64)
    ids = rng.integers(0, 50, 200)
    dy = rng.integers(-4, 5, (200, 12)).astype(np.float64)
    dw = torch.empty(50, 12, device="cuda")
    fsp.embedding_backward(torch.from_numpy(ids).cuda(), torch.from_numpy(dy).float().cuda(), dw, scale=0.5)
    loss = lambda x: (dy * _values(fsp.embedding(torch.from_numpy(x).float().cuda(), torch.from_numpy(ids).cuda(), scale=0.5))).sum()  # noqa: E731
    assert (loss(w + 0.25 * d) - loss(w)) / 0.25 == (_values(dw) * d).sum()


def test_empty_batches():
    dw = torch.ones(6, 5, device="cuda")
    ids, dy = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, 5, device="cuda")
    fsp.embedding_backward(ids, dy, dw, accumulate=True)
    assert float(dw.sum()) == 30
    fsp.embedding_backward(ids, dy, dw)
    assert float(dw.abs().sum()) == 0
    every = torch.full((70,), 2, device="cuda")
    fsp.embedding_backward(every, torch.ones(70, 5, device="cuda"), dw, padding_idx=2)   # nothing but padding
    assert float(dw.abs().sum()) == 0 and fsp.device_error() == 0


def test_gradient_into_a_slice_of_a_grad_buffer_and_on_another_stream():
    plan = fsp.plan_layout([(40, 16), (7,)], 2, "fsdp2")
    buf = torch.zeros(plan.full_len_padded, device="cuda")
    off = plan.param_offsets[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids = torch.arange(80, device="cuda") % 40
    dy = torch.ones(80, 16, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    fsp.embedding_backward(ids, dy, buf[off:off + 640].view(40, 16), accumulate=True, stream=s)
    s.synchronize()
    assert float(buf.sum()) == 80 * 16 and float(buf[off + 640:].abs().sum()) == 0


def test_refusals():
    w = torch.zeros(10, 16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    dy = torch.zeros(4, 16, device="cuda")
    for bad in (lambda: fsp.embedding(w, ids.short()), lambda: fsp.embedding(w.half(), ids),
                lambda: fsp.embedding_backward(ids.float(), dy, w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fsp.embedding(w, ids.cpu()), lambda: fsp.embedding(w.t(), ids), lambda: fsp.embedding(w[0], ids),
                lambda: fsp.embedding(w, ids, out=dy[:3]), lambda: fsp.embedding(w, torch.zeros(8, dtype=torch.int64, device="cuda")[::2]),
                lambda: fsp.embedding_backward(ids, dy[:3], w), lambda: fsp.embedding_backward(ids, dy, w, padding_idx=10)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fsp.FspError, match="overlaps"):
        fsp.embedding(w, ids, out=w[2:6])
    with pytest.raises(fsp.FspError, match="overlaps"):
        fsp.embedding_backward(ids, w[2:6], w)
    with pytest.raises(fsp.FspError, match="workspace"):
        fsp.embedding_backward(ids, dy, w, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fsp.FspError, match="empty table"):
        fsp.embedding(w[:0], ids)


@pytest.mark.parametrize("tokens,vocab,dim,pad,weight", [(2016, 60001, 517, 0, "f32"), (2017, 60001, 517, 0, "f32"),
                                                         (5000, 70000, 380, 4, "f32"), (40000, 52000, 1032, 0, "bf16")])
def test_gradient_of_large_tables(tokens, vocab, dim, pad, weight):
    """Tables of 100 MB and more, on both sides of 64 runs of 32 tokens: every row is written."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    ids = (torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64) ** 6 * vocab).long().clamp_(max=vocab - 1)
    dy = torch.randn(tokens, dim, generator=g, device="cuda").bfloat16()
    buf = torch.full((vocab, dim + pad), float("nan"), device="cuda", dtype=DT[weight])
    fsp.embedding_backward(ids, dy, buf[:, :dim], scale=0.5)
    add = lambda x: torch.zeros(vocab, dim, device="cuda", dtype=torch.float64).index_add_(0, ids, x * 0.5)  # noqa: E731
    want, mag = add(dy.double()), add(dy.double().abs())
    n = torch.bincount(ids, minlength=vocab)
    # n additions and the scaling, each at most 2^-24 of the magnitudes that enter it; then bf16's rounding
    tol = (n[:, None] + 2) * 2.0 ** -24 * mag
    got = buf[:, :dim].double()
    if weight == "bf16":
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert bool(((got - want).abs() <= tol).all())
    assert bool((got[n == 0] == 0).all()) and int((n == 0).sum()) > 0
    assert bool(buf[:, dim:].isnan().all())
    assert fsp.device_error() == 0


def test_a_refused_gradient_launches_nothing():
    dim = 65535 * 32 + 1   # one more column than the join's grid holds
    dw = torch.full((1, dim), 2.0, device="cuda")
    outside = torch.tensor([5], device="cuda")   # what the first launch would report
    with pytest.raises(fsp.FspError, match="columns"):
        fsp.embedding_backward(outside, torch.ones(1, dim, device="cuda"), dw)
    assert fsp.device_error() == 0 and float((dw - 2).abs().max()) == 0


# on both sides of what the sort keeps in registers (131072 tokens), in one, two and three passes
@pytest.mark.parametrize("tokens,vocab,dim,index", [(131072, 70000, 4, 64), (131073, 70000, 4, 32), (131073, 500, 8, 64),
                                                    (300001, 300000, 4, 32), (300001, 131071, 5, 64), (600000, 3, 1, 32)])
def test_gradient_of_long_batches(tokens, vocab, dim, index):
    g = torch.Generator(device="cuda").manual_seed(tokens + vocab)
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    ids = ((vocab + 1.0) ** u - 1).long().clamp_(max=vocab - 1)   # log-uniform: a few tokens hold much of the batch
    dy = torch.randn(tokens, dim, generator=g, device="cuda")
    old = torch.randn(vocab, dim, generator=g, device="cuda")
    add = lambda x: torch.zeros(vocab, dim, device="cuda", dtype=torch.float64).index_add_(0, ids, x * 0.5)  # noqa: E731
    want, mag = add(dy.double()), add(dy.double().abs())
    n = torch.bincount(ids, minlength=vocab)
    # n additions and the scaling, each at most 2^-24 of the magnitudes that enter it; the old value's addition
    tol = (n[:, None] + 2) * 2.0 ** -24 * mag
    for accumulate in (False, True):
        dw = old.clone()
        fsp.embedding_backward(ids.to(IX[index]), dy, dw, scale=0.5, accumulate=accumulate)
        right = want + old if accumulate else want
        assert bool(((dw - right).abs() <= tol + (2.0 ** -24 * right.abs() if accumulate else 0)).all())
        assert torch.equal(dw[n == 0], old[n == 0] if accumulate else torch.zeros_like(old)[n == 0])
    # the sums' order: stable, so that a token's rows are added first to last in runs of 32
    again = torch.empty_like(old)
    fsp.embedding_backward(ids, dy, again, scale=0.5)
    first = torch.empty_like(old)
    fsp.embedding_backward(ids.int(), dy, first, scale=0.5)
    assert torch.equal(again, first) and fsp.device_error() == 0
