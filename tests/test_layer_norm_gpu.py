"""Layer norm, centred and by the root mean square, and its gradients."""
import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp

import block_reference as R
from block_cases import DT, matrix, off_by, values
from gpu_cases import ensure_built

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


# rows, dim, pad, shift: one element, odd and even sizes around each width that the kernels tell apart, rows with
# gaps, off alignment
SIZES = [(1, 1, 0, 0), (3, 2, 0, 0), (5, 7, 1, 0), (9, 8, 0, 0), (4, 31, 0, 1), (33, 64, 0, 0), (70, 128, 0, 0), (35, 128, 8, 8),
         (3, 136, 0, 0), (17, 129, 0, 0), (6, 256, 0, 0), (21, 264, 0, 0), (305, 512, 0, 0), (7, 517, 3, 0), (2, 520, 0, 0), (1, 1024, 0, 0),
         (700, 1024, 0, 0), (12, 1001, 0, 0), (5, 1024, 0, 1), (4, 1032, 0, 0), (2, 2040, 8, 0), (331, 2048, 0, 0), (3, 2049, 0, 0),
         (3, 2056, 0, 0), (5, 4096, 0, 0), (3, 4104, 0, 0), (2, 4099, 0, 0), (5, 8192, 0, 0), (2, 8200, 0, 0), (2, 8191, 1, 0),
         (3, 16384, 0, 0), (2, 16392, 0, 0), (2, 16383, 0, 0), (2, 40000, 0, 0), (1, 100003, 0, 0)]
TYPES = [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "bf16", "bf16")]


def _inputs(rows, dim, rng):
    return rng.normal(0, 1, (rows, dim)) * np.exp(rng.normal(0, 0.5, dim)) + rng.normal(0, 0.5, dim)


def _vector(rng, dim, mean, std, dtype):
    return torch.from_numpy(rng.normal(mean, std, dim).astype(np.float32)).to("cuda", DT[dtype])


@pytest.mark.parametrize("x_t,out_t,par_t", TYPES)
@pytest.mark.parametrize("rows,dim,pad,shift", SIZES)
def test_forward(rows, dim, pad, shift, x_t, out_t, par_t):
    rng = np.random.default_rng(rows * 13 + dim)
    x, _ = matrix(rows, dim, x_t, pad, shift, _inputs(rows, dim, rng))
    w, b = _vector(rng, dim, 1, 0.3, par_t), _vector(rng, dim, 0, 0.3, par_t)
    for center, weight, bias in ((True, w, b), (False, w, None), (True, None, b), (False, None, None)):
        y, intact = matrix(rows, dim, out_t, pad, shift)
        got, stats = fsp.layer_norm(x, weight, bias, eps=EPS, center=center, out=y, stats=True)
        assert got is y and stats.shape == (rows, 2)
        want, tol = R.norm(values(x), 1.0 if weight is None else values(weight), 0.0 if bias is None else values(bias), EPS, center)
        assert off_by(y, want[0], tol[0], out_t) == 0
        st = values(stats)
        assert off_by(st[:, 0], want[1], tol[1], "f32") == 0 and off_by(st[:, 1], want[2], tol[2], "f32") == 0
        assert intact() and fsp.device_error() == 0
        again, check = matrix(rows, dim, out_t, pad, shift)
        assert torch.equal(fsp.layer_norm(x, weight, bias, eps=EPS, center=center, out=again), y)   # without statistics


@pytest.mark.parametrize("x_t,dy_t,par_t", TYPES)
@pytest.mark.parametrize("rows,dim,pad,shift", SIZES)
def test_backward(rows, dim, pad, shift, x_t, dy_t, par_t):
    rng = np.random.default_rng(rows * 17 + dim)
    x, _ = matrix(rows, dim, x_t, pad, shift, _inputs(rows, dim, rng))
    dy, _ = matrix(rows, dim, dy_t, pad, shift, rng.normal(0, 1, (rows, dim)))
    add, _ = matrix(rows, dim, x_t, pad, shift, rng.normal(0, 1, (rows, dim)))
    w = _vector(rng, dim, 1, 0.3, par_t)
    for center, weight, plus, accumulate in ((True, w, None, False), (False, w, add, True), (True, None, add, False), (False, None, None, True)):
        _, stats = fsp.layer_norm(x, eps=EPS, center=center, stats=True)
        st = values(stats)
        dx, intact = matrix(rows, dim, x_t, pad, shift)
        dw, db = _vector(rng, dim, 0, 1, par_t), _vector(rng, dim, 0, 1, par_t)
        old = [values(t) if accumulate else 0.0 for t in (dw, db)]
        got = fsp.layer_norm_backward(x, stats, dy, weight, center=center, grad_weight=dw, grad_bias=db, accumulate=accumulate,
                                      add=plus, out=dx)
        assert got is dx
        want, tol = R.norm_gradients(values(x), st[:, 0], st[:, 1], values(dy), 1.0 if weight is None else values(weight),
                                     0.0 if plus is None else values(plus), center)
        assert off_by(dx, want[0], tol[0], x_t) == 0
        for g, o, v, t in zip((dw, db), old, want[1:], tol[1:]):
            assert off_by(g, v + o, t + R.U * (np.abs(v + o) + np.abs(v)), par_t) == 0
        assert intact() and fsp.device_error() == 0
        # each result alone: the same bits
        only, _ = matrix(rows, dim, x_t, pad, shift)
        fsp.layer_norm_backward(x, stats, dy, weight, center=center, add=plus, out=only)
        if not accumulate:
            one = torch.empty_like(dw)
            assert fsp.layer_norm_backward(x, stats, dy, weight, center=center, grad_weight=one, need_grad_x=False) is None
            assert torch.equal(one, dw)
            fsp.layer_norm_backward(x, stats, dy, weight, center=center, grad_bias=one, need_grad_x=False)
            assert torch.equal(one, db)
        assert off_by(only, want[0], tol[0], x_t) == 0


# enough elements for the kernel that streams rows: every width it tells apart, rows with gaps, off alignment, of a few
# elements, and counts of rows that leave groups of threads without one
MANY = [(300001, 3, 0, 0), (100003, 8, 0, 0), (120001, 7, 1, 1), (47001, 17, 0, 0), (20011, 40, 8, 8), (6301, 128, 0, 0), (6200, 129, 0, 1), (3301, 256, 16, 0),
        (2999, 263, 0, 0), (1601, 520, 8, 0), (1555, 517, 3, 1), (801, 1001, 0, 1), (790, 1024, 0, 2), (401, 2040, 0, 0), (391, 2047, 2, 0), (200, 4099, 0, 0),
        (193, 4096, 8, 8), (101, 8191, 1, 0), (97, 8192, 0, 0), (53, 16383, 0, 1), (49, 16384, 0, 0),
        (51, 16382, 2, 2), (90, 10000, 2, 4), (1500, 1002, 0, 0), (2000, 700, 4, 2), (50003, 30, 2, 0), (9001, 182, 0, 2), (13001, 64, 0, 0),
        (12500, 65, 0, 0), (30001, 32, 0, 0)]


@pytest.mark.parametrize("x_t,out_t,par_t", TYPES)
@pytest.mark.parametrize("rows,dim,pad,shift", MANY)
def test_many_rows(rows, dim, pad, shift, x_t, out_t, par_t):
    rng = np.random.default_rng(rows + dim)
    x, _ = matrix(rows, dim, x_t, pad, shift, _inputs(rows, dim, rng))
    w, b = _vector(rng, dim, 1, 0.3, par_t), _vector(rng, dim, 0, 0.3, par_t)
    for center, bias in ((True, b), (False, None)):
        y, intact = matrix(rows, dim, out_t, pad, shift)
        _, stats = fsp.layer_norm(x, w, bias, eps=EPS, center=center, out=y, stats=True)
        want, tol = R.norm(values(x), values(w), 0.0 if bias is None else values(bias), EPS, center)
        assert off_by(y, want[0], tol[0], out_t) == 0
        st = values(stats)
        assert off_by(st[:, 0], want[1], tol[1], "f32") == 0 and off_by(st[:, 1], want[2], tol[2], "f32") == 0
        assert intact()
    # in place, and the gradients (of the last statistics) into the place of grad_out
    if x_t == out_t:
        z, intact = matrix(rows, dim, x_t, pad, shift)
        z.copy_(x)
        assert torch.equal(fsp.layer_norm(z, w, eps=EPS, center=False, out=z), y) and intact()
    dy, intact = matrix(rows, dim, x_t, pad, shift, rng.normal(0, 1, (rows, dim)))
    want, tol = R.norm_gradients(values(x), st[:, 0], st[:, 1], values(dy), values(w), 0.0, False)
    dw, db = (torch.empty(dim, device="cuda") for _ in range(2))
    fsp.layer_norm_backward(x, stats, dy, w, center=False, grad_weight=dw, grad_bias=db, out=dy)
    assert off_by(dy, want[0], tol[0], x_t) == 0 and off_by(dw, want[1], tol[1], "f32") == 0 and off_by(db, want[2], tol[2], "f32") == 0
    assert intact() and fsp.device_error() == 0


@pytest.mark.parametrize("rows,dim,x_t", [(4099, 1024, "bf16"), (2500, 1001, "f32"), (40000, 128, "bf16"), (1999, 2048, "bf16"),
                                          (70001, 40, "f32"), (650, 8192, "bf16"), (20000, 17, "bf16"), (310, 16384, "f32")])
def test_long_batches(rows, dim, x_t):
    """Many rows, against 64 bits on the device; the parameters' gradients are the same whenever they are computed."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy, add = (torch.randn(rows, dim, generator=g, device="cuda").to(DT[x_t]) for _ in range(3))
    w, b = torch.rand(dim, generator=g, device="cuda") + 0.5, torch.randn(dim, generator=g, device="cuda")
    y, stats = fsp.layer_norm(x, w, b, eps=EPS, stats=True)
    dw, db = torch.empty(2, dim, device="cuda")
    dx = fsp.layer_norm_backward(x, stats, dy, w, grad_weight=dw, grad_bias=db, add=add)
    x64, w64, b64 = (t.double().requires_grad_() for t in (x, w, b))
    m = x64.mean(1, keepdim=True)
    y64 = (x64 - m) / ((x64 - m).square().mean(1, keepdim=True) + EPS).sqrt() * w64 + b64
    y64.backward(dy.double())
    # values of a few units: |h| < 8, |w| < 1.5, |dy| < 8; a row's result collects no more than (depth + 16) roundings of
    # such values, a column's at most `rows` of its terms' sizes
    half = 2.0 ** -8 if x_t == "bf16" else 0.0
    row_tol = (R.depth(dim) + 16) * R.U * 64
    assert bool(((y - y64).abs() <= row_tol + half * (y64.abs() + row_tol)).all())
    want = x64.grad + add
    assert bool(((dx - want).abs() <= row_tol + half * (want.abs() + row_tol)).all())
    h = ((x64 - m) * stats[:, 1:].double()).detach()
    for got, exact, mag in ((dw, w64.grad, (h * dy).abs().sum(0)), (db, b64.grad, dy.double().abs().sum(0))):
        assert bool(((got - exact).abs() <= (rows + 2 * R.depth(dim) + 16) * R.U * mag).all())
    for _ in range(2):
        dw2, db2 = torch.empty(2, dim, device="cuda")
        junk = torch.full((fsp.layer_norm_backward_workspace_bytes(rows, dim),), 0xFF, dtype=torch.uint8, device="cuda")   # (sums' places are written first)
        dx2 = fsp.layer_norm_backward(x, stats, dy, w, grad_weight=dw2, grad_bias=db2, add=add, workspace=junk)
        assert torch.equal(dw, dw2) and torch.equal(db, db2) and torch.equal(dx, dx2)
    assert fsp.device_error() == 0


def test_gradients_against_differences():
    """Central differences of sum(dy * y) along x, w and b together."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy, ddx = (torch.randn(6, 40, generator=g, device="cuda") for _ in range(3))
    w, b, ddw, ddb = (torch.randn(40, generator=g, device="cuda") for _ in range(4))
    for center in (True, False):
        t = 2.0 ** -6
        f = lambda s: float((fsp.layer_norm(x + s * t * ddx, w + s * t * ddw, b + s * t * ddb, center=center).double() * dy).sum())  # noqa: E731
        slope = (8 * (f(0.5) - f(-0.5)) - (f(1) - f(-1))) / (6 * t)   # fourth order in t
        _, stats = fsp.layer_norm(x, w, b, center=center, stats=True)
        dw, db = torch.empty(2, 40, device="cuda")
        dx = fsp.layer_norm_backward(x, stats, dy, w, center=center, grad_weight=dw, grad_bias=db)
        want = float((dx * ddx).double().sum() + (dw * ddw).double().sum() + (db * ddb).double().sum())
        # 240 results of size 1, each within some 2^-20, over t; the differences' own error of order t^4
        assert abs(slope - want) <= 240 * 2.0 ** -20 / t * 3 + 240 * 30 * t ** 4


def test_rows_keep_to_themselves():
    """Rows of constants, of huge and tiny values, with an infinity or a NaN: the others are as without them."""
    g = torch.Generator(device="cuda").manual_seed(5)
    for dim in (64, 129, 1024, 3000):
        x = torch.randn(9, dim, generator=g, device="cuda")
        plain = fsp.layer_norm(x, eps=EPS)
        _, plain_stats = fsp.layer_norm(x, eps=EPS, stats=True)
        y = x.clone()
        y[1], y[3] = 2.5, 0.0
        y[5, 1], y[6, dim // 2], y[7] = float("inf"), float("nan"), y[7] * 1e-30
        got, stats = fsp.layer_norm(y, eps=EPS, stats=True)
        for r in (0, 2, 4, 8):
            assert torch.equal(got[r], plain[r]) and torch.equal(stats[r], plain_stats[r])
        assert float(got[1].abs().max()) <= (R.depth(dim) + 2) * R.U * 2.5 / EPS ** 0.5   # only the mean's rounding is left
        assert float(got[3].abs().max()) == 0 and bool(got[5].isnan().any()) and bool(got[6].isnan().all())
        assert float(got[7].abs().max()) < 1e-25
        assert bool(fsp.layer_norm(y[3:4], eps=0.0, center=False).isnan().all())   # 0 / 0
        dy = torch.randn(9, dim, generator=g, device="cuda")
        clean, dirty = (fsp.layer_norm_backward(t, s, dy) for t, s in ((x, plain_stats), (y, stats)))
        for r in (0, 2, 4, 8):
            assert torch.equal(clean[r], dirty[r])
        dw = torch.empty(dim, device="cuda")
        fsp.layer_norm_backward(y, stats, dy, grad_weight=dw, need_grad_x=False)
        assert bool(dw.isnan().all())   # a NaN's row reaches every column


def test_in_place_and_shapes():
    g = torch.Generator(device="cuda").manual_seed(7)
    for dim in (96, 101, 1024, 20000):
        x, dy, add = (torch.randn(37, dim, generator=g, device="cuda") for _ in range(3))
        w = torch.rand(dim, generator=g, device="cuda")
        y, stats = fsp.layer_norm(x, w, stats=True)
        z = x.clone()
        assert fsp.layer_norm(z, w, out=z) is z and torch.equal(z, y)
        dw, dw2 = torch.empty(2, dim, device="cuda")
        dx = fsp.layer_norm_backward(x, stats, dy, w, grad_weight=dw, add=add)
        for k in range(3):   # into the place of x, of grad_out, of add
            t = [x.clone(), dy.clone(), add.clone()]
            assert fsp.layer_norm_backward(t[0], stats, t[1], w, grad_weight=dw2, add=t[2], out=t[k]) is t[k]
            assert torch.equal(t[k], dx) and torch.equal(dw, dw2)
    x = torch.randn(2, 3, 5, 32, device="cuda")
    y, stats = fsp.layer_norm(x, stats=True)
    assert y.shape == x.shape and stats.shape == (2, 3, 5, 2) and y.dtype == x.dtype
    fill = torch.empty(2, 3, 5, 2, device="cuda")
    assert fsp.layer_norm(x, stats=fill)[1] is fill and torch.equal(fill, stats)
    assert torch.equal(fsp.layer_norm_backward(x, stats, x).view(30, 32), fsp.layer_norm_backward(x.view(30, 32), stats.view(30, 2), x.view(30, 32)))
    assert torch.equal(fsp.layer_norm(x[0, 0, 0]), y[0, 0, 0]) and fsp.layer_norm(x[:, :0]).shape == (2, 0, 5, 32)
    assert fsp.layer_norm(x[..., :0].contiguous()).shape == (2, 3, 5, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = fsp.layer_norm(x, stream=s)
    s.synchronize()
    assert torch.equal(z, y)


def test_empty_batches():
    x, stats = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, device="cuda")
    dw, db = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
    fsp.layer_norm_backward(x, stats, x, grad_weight=dw, grad_bias=db, accumulate=True)
    assert float(dw.sum() + db.sum()) == 16
    fsp.layer_norm_backward(x, stats, x, grad_weight=dw)
    assert float(dw.sum()) == 0 and float(db.sum()) == 8
    assert fsp.layer_norm_backward(x, stats, x).shape == (0, 8)


# both sides of what one CTA takes
@pytest.mark.parametrize("rows,dim", [(128, 40), (129, 40), (128, 100), (129, 101), (64, 256), (65, 255), (32, 512), (33, 512), (16, 1024), (17, 1001), (8, 2048),
                                      (9, 2048), (4, 4096), (5, 4095), (2, 8192), (3, 8192), (1, 8200), (2, 16384), (1, 20000)])
def test_gradients_of_few_rows(rows, dim):
    rng = np.random.default_rng(rows + dim)
    x, _ = matrix(rows, dim, "bf16", fill=_inputs(rows, dim, rng))
    dy, _ = matrix(rows, dim, "bf16", fill=rng.normal(0, 1, (rows, dim)))
    _, stats = fsp.layer_norm(x, stats=True)
    st = values(stats)
    want, tol = R.norm_gradients(values(x), st[:, 0], st[:, 1], values(dy), 1.0, 0.0, True)
    for accumulate in (False, True):
        dw, old = _vector(rng, dim, 0, 1, "bf16"), None
        db = _vector(rng, dim, 0, 1, "bf16")
        old = [values(t) if accumulate else 0.0 for t in (dw, db)]
        need = fsp.layer_norm_backward_workspace_bytes(rows, dim)
        work = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda") if accumulate else None
        dx = fsp.layer_norm_backward(x, stats, dy, grad_weight=dw, grad_bias=db, accumulate=accumulate, workspace=work)
        assert off_by(dx, want[0], tol[0], "bf16") == 0
        for g, o, v, t in zip((dw, db), old, want[1:], tol[1:]):
            assert off_by(g, v + o, t + R.U * (np.abs(v + o) + np.abs(v)), "bf16") == 0
    assert fsp.device_error() == 0


def test_offsets_past_32_bits():
    big = torch.zeros(2 ** 20 + 3, 4096, dtype=torch.bfloat16, device="cuda")   # rows 4096 apart: 2^32 elements and more
    x = big[:, :64]
    x[-1] = torch.randn(64, device="cuda")
    y, stats = fsp.layer_norm(x, eps=EPS, out=big[:, 64:128], stats=True)
    assert torch.equal(y[-1], fsp.layer_norm(x[-1:].clone(), eps=EPS)[0]) and float(y[:-1].abs().max()) == 0
    dw = torch.empty(64, device="cuda")
    dx = fsp.layer_norm_backward(x, stats, x, grad_weight=dw, out=big[:, 128:192])
    one = torch.empty(64, device="cuda")
    assert torch.equal(dx[-1], fsp.layer_norm_backward(x[-1:].clone(), stats[-1:].clone(), x[-1:].clone(), grad_weight=one)[0])
    assert torch.equal(one, dw) and float(big[:-1].abs().max()) == 0 and float(big[:, 192:].abs().max()) == 0


def test_captured_and_replayed():
    x, dy = torch.randn(2, 300, 520, device="cuda")
    w = torch.rand(520, device="cuda")
    dw, y, dx = torch.zeros(520, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    stats = torch.empty(300, 2, device="cuda")

    def both():
        fsp.layer_norm(x, w, out=y, stats=stats)
        fsp.layer_norm_backward(x, stats, dy, w, grad_weight=dw, accumulate=True, out=dx)
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        x.normal_()
        dw.zero_()
        graph.replay()
        got = [t.clone() for t in (y, dx, dw)]
        dw.zero_()
        both()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dw)))
    assert fsp.device_error() == 0


def test_refusals():
    x, w = torch.zeros(4, 16, device="cuda"), torch.ones(16, device="cuda")
    stats = torch.zeros(4, 2, device="cuda")
    for bad in (lambda: fsp.layer_norm(x.half()), lambda: fsp.layer_norm(x, w.half()), lambda: fsp.layer_norm(x, w, w.bfloat16()),
                lambda: fsp.layer_norm(x, out_dtype=torch.float16),
                lambda: fsp.layer_norm_backward(x, stats, x, grad_weight=w, grad_bias=w.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fsp.layer_norm(x.cpu()), lambda: fsp.layer_norm(x, w.cpu()), lambda: fsp.layer_norm(x.t()),
                lambda: fsp.layer_norm(x, w[:8]), lambda: fsp.layer_norm(x, torch.ones(32, device="cuda")[::2]),
                lambda: fsp.layer_norm(x, out=x[:2]), lambda: fsp.layer_norm(x, stats=stats[:3]),
                lambda: fsp.layer_norm(x, stats=stats.bfloat16()), lambda: fsp.layer_norm(torch.zeros(2, 8, 16, device="cuda")[:, ::2]),
                lambda: fsp.layer_norm_backward(x, stats, x[:3]), lambda: fsp.layer_norm_backward(x, stats[:3], x),
                lambda: fsp.layer_norm_backward(x, stats, x, add=x.bfloat16()), lambda: fsp.layer_norm_backward(x, stats, x, out=x.bfloat16()),
                lambda: fsp.layer_norm_backward(x, stats, x, need_grad_x=False, add=x),
                lambda: fsp.layer_norm_backward(x, stats, x, grad_weight=w[:8])):
        with pytest.raises(ValueError):
            bad()
    flat = torch.zeros(200, device="cuda")
    with pytest.raises(fsp.FspError, match="overlaps"):
        fsp.layer_norm(flat[:64].view(4, 16), out=flat[16:80].view(4, 16))
    with pytest.raises(fsp.FspError, match="overlaps"):
        fsp.layer_norm_backward(x, stats, x, grad_weight=x[0])
    with pytest.raises(fsp.FspError, match="workspace"):
        many = torch.zeros(500, 16, device="cuda")
        fsp.layer_norm_backward(many, many[:, :2].contiguous(), many, grad_weight=w, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fsp.FspError, match="eps"):
        fsp.layer_norm(x, eps=-1.0)
