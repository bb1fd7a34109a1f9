"""What the norm's arithmetic has to get right beyond the rounding of ordinary values: rows of one value."""
import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp

import block_reference as R
from block_cases import DT, matrix, off_by, values
from gpu_cases import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


# rows, dim, pad: few rows and many, lengths that have no exact reciprocal, even, odd, with gaps
ONE_VALUE = [(3, 6, 0), (300, 1000, 0), (4096, 1000, 0), (4096, 1001, 0), (1200, 700, 4), (40000, 30, 2), (30011, 33, 0), (100, 9999, 0), (100, 10000, 0),
             (60, 16381, 1), (3, 20000, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,pad", ONE_VALUE)
def test_rows_of_one_value(rows, dim, pad, dtype):
    """Values of eight significant bits: every partial sum of up to 2^16 of them is a float, and so is the mean:
    nothing is left of the row."""
    for value in (99840.0, -40960.0, 0.30078125, 3.5):
        x, _ = matrix(rows, dim, dtype, pad, fill=np.full((rows, dim), value))
        y, stats = fsp.layer_norm(x, stats=True)
        assert float(y.abs().max()) == 0 and bool((stats[:, 0] == value).all())
        dy, _ = matrix(rows, dim, dtype, pad, fill=np.random.default_rng(rows).normal(0, 1, (rows, dim)))
        dw = torch.empty(dim, device="cuda")
        dx = fsp.layer_norm_backward(x, stats, dy, grad_weight=dw)
        st = values(stats)
        want, tol = R.norm_gradients(values(x), st[:, 0], st[:, 1], values(dy), 1.0, 0.0, True)
        assert off_by(dx, want[0], tol[0], dtype) == 0 and float(dw.abs().max()) == 0
        dy.fill_(value)   # and nothing of a gradient of one value
        assert float(fsp.layer_norm_backward(x, stats, dy).abs().max()) == 0
    assert fsp.device_error() == 0


@pytest.mark.parametrize("rows,dim", [(5, 100), (9000, 100), (4096, 1001), (60, 16000), (3, 20000)])
def test_infinite_sums(rows, dim):
    """An infinity among a row's gradients, at h = 1: both means are infinite, and so is the gradient of every other element;
    a row whose sum of finite values leaves fp32's range has infinite statistics.  The rows beside them are as they were."""
    x, dy = torch.randn(2, rows, dim, device="cuda")
    _, stats = fsp.layer_norm(x, stats=True)
    clean = fsp.layer_norm_backward(x, stats, dy)
    dy[1, 7], x[1], stats[1] = float("inf"), 1, torch.tensor([0.0, 1.0], device="cuda")
    got = fsp.layer_norm_backward(x, stats, dy)
    assert bool(got[1, 7].isnan()) and bool((got[1, 8:] == -float("inf")).all()) and bool((got[1, :7] == -float("inf")).all())
    assert torch.equal(got[2:], clean[2:]) and torch.equal(got[0], clean[0])
    x[2] = 3e38
    y, stats = fsp.layer_norm(x, stats=True)
    assert bool(y[2].isnan().all()) and stats[2].tolist() == [float("inf"), 0.0] and bool(y[3:].isfinite().all())


@pytest.mark.parametrize("rows,dim", [(300, 64), (40000, 64), (20000, 128), (20000, 1024)])
def test_inverse_deviations(rows, dim):
    """Rows of +-a, a of seven bits: the squares, their sums (at most 2^24) and the division by 2^k are exact, so the
    variance is, and eps's sum is rounded once.  Then r's own roundings: 1.5 * 2^-24 of a step of Newton's method after
    the terms of its square (2^-46), or half of 2^-24 of a root and a division's."""
    rng = np.random.default_rng(dim)
    a = np.ldexp(rng.integers(64, 128, rows), rng.integers(-9, 3, rows)).astype(np.float32)
    x = torch.from_numpy((a[:, None] * np.where(rng.random((rows, dim)) < 0.5, -1, 1)).astype(np.float32)).cuda()
    for eps in (0.0, 1e-5, 2.0 ** -12, 0.3, 3e-3, 0.011):
        _, stats = fsp.layer_norm(x, eps=eps, center=False, stats=True)
        r = 1 / np.sqrt((a * a + np.float32(eps)).astype(np.float64))
        assert (np.abs(values(stats[:, 1]) - r) <= 1.51 * R.U * r).all() and float(stats[:, 0].abs().max()) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,pad,shift", [(4, 6, 0, 0), (5, 8, 0, 0), (7, 33, 0, 1), (130, 40, 0, 0), (300, 200, 0, 0), (300, 201, 3, 0), (9, 1000, 0, 0), (5, 2049, 0, 0),
                                                (3, 9000, 0, 0), (3, 9002, 2, 2), (3, 9001, 0, 1), (4, 128, 0, 0), (2, 20000, 0, 0)])
def test_means_far_from_the_rows_spread(rows, dim, pad, shift, dtype):
    """Rows of 2^112 whose inverse deviation is 2^20: m r is out of fp32's range, x - m is not.  (Sums of 2^112 up to
    2^15 times are floats.)"""
    x, _ = matrix(rows, dim, dtype, pad, shift, np.full((rows, dim), 2.0 ** 112))
    dy, _ = matrix(rows, dim, dtype, pad, shift, np.random.default_rng(dim).normal(0, 1, (rows, dim)))
    for center in (True, False):
        y, stats = fsp.layer_norm(x, eps=2.0 ** -40, center=center, stats=True)
        if not center:   # its variance is out of range: statistics as if there were none
            stats = torch.tensor([2.0 ** 112, 2.0 ** 20], device="cuda").repeat(rows, 1)
        assert bool((stats == torch.tensor([2.0 ** 112, 2.0 ** 20], device="cuda")).all())
        dw, db = torch.empty(2, dim, device="cuda")
        dx = fsp.layer_norm_backward(x, stats, dy, center=center, grad_weight=dw, grad_bias=db)
        want, tol = R.norm_gradients(values(x), values(stats[:, 0]), values(stats[:, 1]), values(dy), 1.0, 0.0, center)
        assert off_by(dx, want[0], tol[0], dtype) == 0 and float(dw.abs().max()) == 0 and off_by(db, want[2], tol[2], "f32") == 0
    assert fsp.device_error() == 0
