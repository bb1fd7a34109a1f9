"""Dropout from the counter-based generator, onto a residual stream, and its gradient."""
import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp

import block_reference as R
from block_cases import DT, matrix, off_by, values
from gpu_cases import ensure_built

pytestmark = pytest.mark.gpu
SEED, CALL = 0xFEDCBA9876543210, -0x123456789ABCDEF


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


# rows, dim, pad, shift
SIZES = [(1, 1, 0, 0), (1, 7, 0, 0), (1, 8, 0, 0), (3, 3, 0, 0), (5, 7, 1, 0), (2, 8, 8, 0), (9, 24, 8, 8), (4, 24, 3, 0), (33, 64, 0, 1),
         (17, 129, 0, 0), (300, 517, 0, 0), (64, 512, 0, 0), (5, 2048, 16, 0), (3, 2050, 6, 0), (1, 100003, 0, 0)]


@pytest.mark.parametrize("x_t,res_t,out_t", [("f32", "", "f32"), ("bf16", "", "bf16"), ("bf16", "f32", "f32"), ("f32", "bf16", "bf16"),
                                             ("bf16", "bf16", "bf16"), ("f32", "", "bf16"), ("bf16", "", "f32"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("rows,dim,pad,shift", SIZES)
def test_dropout(rows, dim, pad, shift, x_t, res_t, out_t):
    rng = np.random.default_rng(rows * 11 + dim)
    x, _ = matrix(rows, dim, x_t, pad, shift, rng.normal(0, 1, (rows, dim)))
    h = matrix(rows, dim, res_t, pad, shift, rng.normal(0, 3, (rows, dim)))[0] if res_t else None
    for k, p in enumerate((0.1, 0.5)):
        y, intact = matrix(rows, dim, out_t, pad, shift)
        call = torch.full((1,), CALL, device="cuda") if k else CALL
        assert fsp.dropout(x, p, SEED, call, residual=h, out=y) is y
        res = values(h) if res_t else 0.0
        want, keep = R.dropout(values(x), p, SEED, CALL, res)
        # the scale's rounding, the product's (or the fused sum's)
        assert off_by(y, want, 2 * R.U * np.abs(want - res) + R.U * np.abs(want), out_t) == 0
        if not res_t:
            assert np.array_equal(values(y)[~keep], np.zeros((~keep).sum()))
        dy, _ = matrix(rows, dim, out_t, pad, shift, rng.normal(0, 1, (rows, dim)))
        dx, ok = matrix(rows, dim, x_t, pad, shift)
        assert fsp.dropout_backward(dy, p, SEED, call, out=dx) is dx
        grad = R.dropout(values(dy), p, SEED, CALL)[0]
        assert off_by(dx, grad, 2 * R.U * np.abs(grad), x_t) == 0
        assert intact() and ok() and fsp.device_error() == 0


@pytest.mark.parametrize("rows,dim,pad,shift,res_t,out_t", [(8193, 1024, 0, 0, "bf16", "bf16"), (8200, 1032, 8, 8, "f32", "f32"), (9001, 1001, 0, 0, "bf16", "f32"),
                                                            (8400, 1001, 3, 1, "f32", "bf16"), (4100, 2056, 16, 0, "", "bf16")])
def test_many_elements(rows, dim, pad, shift, res_t, out_t):
    """From 2^23 elements on a thread takes several blocks of the generator: the same results as call by call on parts."""
    n = rows * (dim + pad) + shift
    g = torch.Generator(device="cuda").manual_seed(rows)
    new = lambda t: torch.randn(n, generator=g, device="cuda").to(DT[t])[shift:].view(rows, dim + pad)[:, :dim]  # noqa: E731
    x, h, y = new("bf16"), new(res_t) if res_t else None, new(out_t)
    fsp.dropout(x, 0.1, SEED, CALL, residual=h, out=y)
    keep = torch.from_numpy(R.random16(rows * dim, SEED, CALL) >= 6554).cuda().view(rows, dim)
    want = torch.where(keep, x.double() * (65536 / (65536 - 6554)), 0.0) + (0 if h is None else h.double())
    tol = 2 * R.U * (x.double() * 1.2).abs() + R.U * want.abs()
    assert bool(((y - want).abs() <= tol + (2.0 ** -8 * (want.abs() + tol) if out_t == "bf16" else 0)).all())
    assert fsp.device_error() == 0


def test_the_mask_is_a_function_of_seed_call_and_index():
    ones = torch.ones(7, 1000, device="cuda")
    mask = lambda x, *a: fsp.dropout(x, 0.5, *a) != 0  # noqa: E731
    first = mask(ones, 1, 2)
    want = R.random16(7000, 1, 2) >= 32768
    assert np.array_equal(first.cpu().numpy().ravel(), want)
    assert torch.equal(first.view(-1), mask(ones.view(-1), 1, 2)) and torch.equal(first.view(-1), mask(ones.view(7, 10, 100), 1, 2).view(-1))
    assert torch.equal(first, mask(ones.bfloat16(), 1, 2)) and torch.equal(first[:2], mask(ones[:2], 1, 2))
    gaps = torch.ones(7, 1003, device="cuda")[:, :1000]
    assert torch.equal(first, mask(gaps, 1, 2))
    others = [mask(ones, *a) for a in ((2, 2), (1, 3), (1 + 2 ** 32, 2), (1, 2 + 2 ** 32), (1, 2 ** 33))]
    for m in others:   # 7000 fair coins against 7000 others: half of them, within six deviations
        assert abs(float((m == first).float().mean()) - 0.5) < 6 * 0.5 / 7000 ** 0.5
    assert torch.equal(first, mask(ones, 1 + 2 ** 64, 2))   # 64 bits of the seed


def test_how_often_and_how_much():
    n = 1 << 24
    x = torch.ones(n, device="cuda")
    for p in (0.1, 0.25, 0.9):
        y = fsp.dropout(x, p, 99, 7)
        lost = float((y == 0).double().mean())
        q = int(p * 65536 + 0.5) / 65536
        assert abs(lost - q) < 6 * (q * (1 - q) / n) ** 0.5
        assert set(y.unique().tolist()) == {0.0, float(np.float32(1 / (1 - q)))}
    assert torch.equal(fsp.dropout(x, 0.0, 5), x) and float(fsp.dropout(x, 1.0, 5).abs().max()) == 0
    assert torch.equal(fsp.dropout(x, 1.0, 5, residual=x), x) and torch.equal(fsp.dropout(x, 2.0 ** -18, 5), x)


def test_what_is_dropped_does_not_enter():
    x = torch.full((5000,), float("nan"), device="cuda")
    x[::2] = float("inf")
    h = torch.randn(5000, device="cuda")
    keep = torch.from_numpy(R.random16(5000, 3, 4) >= int(0.3 * 65536 + 0.5)).cuda()
    y = fsp.dropout(x, 0.3, 3, 4, residual=h)
    assert torch.equal(y[~keep], h[~keep]) and not bool(y[keep].isfinite().any())
    z = fsp.dropout(x.bfloat16(), 0.3, 3, 4)
    assert float(z[~keep].abs().max()) == 0 and not bool(z[keep].isfinite().any())


def test_in_place_other_streams_and_empties():
    for dim in (1024, 333):
        x, h = torch.randn(2, 50, dim, device="cuda")
        want = fsp.dropout(x, 0.2, 8, 9, residual=h)
        for k in range(2):
            t = [x.clone(), h.clone()]
            assert fsp.dropout(t[0], 0.2, 8, 9, residual=t[1], out=t[k]) is t[k] and torch.equal(t[k], want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = fsp.dropout(x, 0.2, 8, 9, residual=h, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    assert fsp.dropout(x[:0], 0.2, 8).shape == (0, 333) and fsp.dropout(x[:, :0].contiguous(), 0.2, 8).shape == (50, 0)
    one = torch.ones((), device="cuda")
    assert fsp.dropout(one, 0.0, 1).shape == () and float(fsp.dropout(one, 0.0, 1, residual=one)) == 2
    assert fsp.dropout(x.bfloat16(), 0.1, 1, residual=h).dtype == torch.float32


def test_numbers_past_32_bits():
    """More than 2^32 elements: the counter's second word and the offsets."""
    n = 2 ** 32 + 4096 + 5
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    fsp.dropout(x, 0.5, 21, 22, out=x)
    tail = x[2 ** 32 - 8:].float().cpu().numpy()
    i = np.arange(2 ** 29 - 1, 2 ** 29 + 513, dtype=np.uint64)
    one = np.ones_like(i)
    w = np.stack(R.philox([i, one * 0, one * np.uint64(22), one * 0], [21, 0]), 1)
    want = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)[:len(tail)] >= 32768
    assert np.array_equal(tail != 0, want)


def test_a_captured_call_reads_its_number():
    x, y = torch.randn(4000, device="cuda"), torch.empty(4000, device="cuda")
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    fsp.dropout(x, 0.5, 77, step, out=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fsp.dropout(x, 0.5, 77, step, out=y)
        step.add_(1)
    for k in range(1, 4):
        graph.replay()
        assert torch.equal(y, fsp.dropout(x, 0.5, 77, k))
    assert int(step) == 4


def test_refusals():
    x = torch.zeros(4, 16, device="cuda")
    for bad in (lambda: fsp.dropout(x.half(), 0.1, 1), lambda: fsp.dropout(x, 0.1, 1, residual=x.double()), lambda: fsp.dropout(x, 0.1, 1, out_dtype=torch.int32)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fsp.dropout(x.cpu(), 0.1, 1), lambda: fsp.dropout(x.t(), 0.1, 1), lambda: fsp.dropout(x, 0.1, 1, residual=x[:2]),
                lambda: fsp.dropout(x, 0.1, 1, out=x[:2]), lambda: fsp.dropout(x, 0.1, 1, out=x, out_dtype=torch.bfloat16),
                lambda: fsp.dropout(x, 0.1, 1, torch.zeros(2, dtype=torch.int64, device="cuda")),
                lambda: fsp.dropout(x, 0.1, 1, torch.zeros(1, device="cuda")), lambda: fsp.dropout(x, 0.1, 1, torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            bad()
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(fsp.FspError, match="p must"):
            fsp.dropout(x, p, 1)
    flat = torch.zeros(100, device="cuda")
    with pytest.raises(fsp.FspError, match="overlaps"):
        fsp.dropout(flat[:64], 0.1, 1, out=flat[8:72])
