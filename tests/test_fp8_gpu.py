"""Matrices in 8-bit floating point, their product, and the linear layer on them."""
import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp

from gpu_cases import Guarded, ensure_built
from ops_reference import fp8, rounds_to

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _values(x):
    return x.float().cpu().numpy()


def _wide(rng, rows, cols):
    """Values whose blocks differ by many powers of two, some zero blocks and zeros."""
    x = rng.normal(0, 1, (rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, (cols + 127) // 128)).repeat(128, 1)[:, :cols])
    x[rng.random((rows, cols)) < 0.05] = 0
    x[:, :128] *= rng.random((rows, 1)) < 0.8
    return x.astype(np.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad,shift", [(1, 1, 0, 0), (1, 128, 0, 0), (3, 5, 0, 0), (128, 128, 0, 0), (129, 513, 0, 0),
                                                 (64, 777, 0, 0), (200, 1024, 0, 0), (33, 130, 6, 0), (20, 640, 8, 8),
                                                 (20, 641, 0, 1), (300, 16, 0, 0), (65, 64, 0, 0)])
def test_codes_are_the_definition(rows, cols, pad, shift, dtype):
    rng = np.random.default_rng(rows + cols)
    buf = torch.zeros(rows * (cols + pad) + shift, dtype=DT[dtype], device="cuda")
    x = buf[shift:].view(rows, cols + pad)[:, :cols]
    x.copy_(torch.from_numpy(_wide(rng, rows, cols)))
    q, qt = fsp.quantize_fp8(x, True, True)
    h = _values(x)
    assert np.array_equal(_values(q.values()), fp8(h).astype(np.float32))
    assert np.array_equal(_values(qt.values()), fp8(h.T).astype(np.float32))
    assert np.array_equal(_values(fsp.quantize_fp8(x).values()), fp8(h).astype(np.float32))
    assert np.array_equal(_values(fsp.quantize_fp8(x, None, True).values()), fp8(h.T).astype(np.float32))


def test_scales_at_the_ends_of_their_range():
    x = torch.zeros(8, 128, device="cuda")
    for i, top in enumerate((448.0, 448.00003, 1.75, 1.7500001, 3.4e38, 2.0 ** -126, 1e-44, 2.0 ** -119 * 1.75)):
        x[i, 3], x[i, 9] = top, -top / 2
    got, want = _values(fsp.quantize_fp8(x).values()), fp8(_values(x))
    assert np.array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_non_finite_value_makes_its_block_nan(bad):
    x = torch.ones(3, 300, device="cuda")
    x[1, 130] = bad
    q, qt = fsp.quantize_fp8(x, True, True)
    v = _values(q.values())
    assert np.isnan(v[1, 128:256]).all() and np.isfinite(np.delete(v, 1, 0)).all() and np.isfinite(v[1, :128]).all()
    vt = _values(qt.values())
    assert np.isnan(vt[130]).all() and np.isfinite(np.delete(vt, 130, 0)).all()
    y = _values(fsp.matmul_fp8(q, fsp.quantize_fp8(torch.ones(5, 300, device="cuda")), out_dtype=torch.float32))
    assert np.isnan(y[1]).all() and (np.delete(y, 1, 0) == 300).all()
    z = _values(fsp.matmul_fp8(fsp.quantize_fp8(torch.ones(5, 300, device="cuda")), q, out_dtype=torch.float32))
    assert np.isnan(z[:, 1]).all() and (np.delete(z, 1, 1) == 300).all()


# one token, tiles' edges, odd sizes, many blocks of k, more tiles than SMs
SHAPES = [(1, 1, 1), (1, 2048, 1024), (2, 300, 128), (3, 5, 7), (16, 17, 129), (17, 128, 640), (33, 1000, 777), (64, 257, 2048),
          (65, 256, 384), (128, 128, 128), (129, 127, 513), (200, 600, 5632), (333, 1001, 777), (1000, 130, 96),
          (2500, 2100, 256), (2048, 4000, 128)]


def _product(a, b):
    x, y = fp8(a).astype(np.float64), fp8(b).astype(np.float64)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def _tolerance(k, mag):
    """k exact products added in fp32, in any order and with any rounding: each
    addition is off by at most 2^-23 of the magnitudes added so far."""
    return (k + 1) * 2.0 ** -23 * mag


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k):
    rng = np.random.default_rng(m + n + k)
    a, b = rng.normal(0, 1, (m, k)).astype(np.float32), (rng.normal(0, 1, (n, k)) * np.exp2(rng.integers(-6, 6, (n, 1)))).astype(np.float32)
    want, mag = _product(a, b)
    qa, qb = fsp.quantize_fp8(torch.from_numpy(a).cuda()), fsp.quantize_fp8(torch.from_numpy(b).cuda())
    tol = _tolerance(k, mag)
    got = _values(fsp.matmul_fp8(qa, qb, out_dtype=torch.float32))
    assert (np.abs(got - want) <= tol).all()
    # typical errors are far smaller: a 2^-24 step per addition, independent signs
    assert np.linalg.norm(got - want) <= 2.0 ** -20 * np.linalg.norm(want) + 1e-30
    assert rounds_to(_values(fsp.matmul_fp8(qa, qb)), want, tol).all()
    # accumulate, into rows with gaps, off alignment, between guards
    for pad, shift in ((0, 0), (3, 1), (8, 4)):
        g = Guarded(m * (n + pad) + shift, torch.float32, 0)
        c = g.t[shift:].view(m, n + pad)[:, :n]
        c.fill_(1.5)
        fsp.matmul_fp8(qa, qb, out=c, accumulate=True)
        assert (np.abs(_values(c) - (want + 1.5)) <= tol + 2.0 ** -23 * (mag + 1.5)).all()
        h = Guarded(m * (n + pad) + shift, torch.bfloat16, 0)
        d = h.t[shift:].view(m, n + pad)[:, :n]
        fsp.matmul_fp8(qa, qb, out=d)
        assert rounds_to(_values(d), want, tol).all()
        if pad:
            assert float(g.t[shift:].view(m, n + pad)[:, n:].abs().sum()) == 0
            assert float(h.t[shift:].view(m, n + pad)[:, n:].abs().sum()) == 0
        assert g.guards_intact() and h.guards_intact()
    assert fsp.device_error() == 0


def test_product_of_blocks_with_far_apart_scales():
    rng = np.random.default_rng(3)
    a, b = _wide(rng, 70, 1500), _wide(rng, 200, 1500)
    want, mag = _product(a, b)
    got = _values(fsp.matmul_fp8(fsp.quantize_fp8(torch.from_numpy(a).cuda()), fsp.quantize_fp8(torch.from_numpy(b).cuda()),
                                 out_dtype=torch.float32))
    assert (np.abs(got - want) <= _tolerance(1500, mag)).all()


def test_product_repeats_bit_for_bit_and_sums_nothing():
    qa, qb = fsp.quantize_fp8(torch.randn(300, 900, device="cuda")), fsp.quantize_fp8(torch.randn(400, 900, device="cuda"))
    a = fsp.matmul_fp8(qa, qb, out_dtype=torch.float32)
    assert all(torch.equal(a, fsp.matmul_fp8(qa, qb, out_dtype=torch.float32)) for _ in range(3))
    e = fsp.quantize_fp8(torch.zeros(4, 0, device="cuda"))
    assert float(fsp.matmul_fp8(e, fsp.quantize_fp8(torch.zeros(6, 0, device="cuda")), out=torch.ones(4, 6, device="cuda")).abs().sum()) == 0
    assert fsp.matmul_fp8(fsp.quantize_fp8(torch.zeros(0, 5, device="cuda")), fsp.quantize_fp8(torch.zeros(6, 5, device="cuda"))).shape == (0, 6)


@pytest.mark.parametrize("m,n,k", [(1, 64, 96), (1, 2048, 1024), (37, 130, 257), (256, 384, 512), (1030, 520, 200), (100, 3000, 300), (1024, 2300, 260)])
def test_linear_layer(m, n, k):
    rng = np.random.default_rng(m * n)
    bf = lambda *s: torch.from_numpy(rng.normal(0, 1, s).astype(np.float32)).cuda().bfloat16()  # noqa: E731
    x, w, dy = bf(m, k), bf(n, k), bf(m, n)
    layer = fsp.Fp8Linear(w, train=True)
    y = layer.forward(x)
    dw = torch.full((n, k), 2.0, device="cuda")
    dx = layer.backward(x, dy, dw)
    hx, hw, hd = _values(x), _values(w), _values(dy)
    for got, (p, q) in ((y, (hx, hw)), (dx, (hd, hw.T)), (dw, (hd.T, hx.T))):
        want, mag = _product(p, q)
        tol = _tolerance(p.shape[1], mag)
        if got.dtype == torch.bfloat16:
            assert rounds_to(_values(got), want, tol).all()
        else:
            assert (np.abs(_values(got) - want) <= tol).all()
    first = dw.clone()
    assert layer.backward(x, dy, dw, accumulate=True, need_grad_x=False) is None
    assert torch.allclose(dw, 2 * first, rtol=2.0 ** -22, atol=0)
    layer.update(w * 2)
    assert torch.equal(layer.forward(x), 2 * y)
    # leading dimensions, and a side stream
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = layer.forward(x.view(1, m, k), stream=s)
    s.synchronize()
    assert z.shape == (1, m, n) and torch.equal(z[0], 2 * y)


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,n,k,pad,shift", [(1, 1, 1, 0, 0), (1, 15, 128, 0, 0), (1, 2048, 1024, 0, 0), (2, 129, 777, 3, 1),
                                                (3, 1000, 5632, 0, 0), (4, 17, 130, 8, 8), (4, 33, 4096, 0, 0), (3, 40, 5461, 1, 1),
                                                (1, 30, 16384, 0, 0), (1, 30, 16385, 0, 0), (4, 30, 4097, 0, 0), (1, 20000, 96, 0, 0)])
def test_few_rows(rows, n, k, pad, shift, x, y):
    rng = np.random.default_rng(rows * n + k)
    buf = torch.zeros(rows * (k + pad) + shift, dtype=DT[x], device="cuda")
    xd = buf[shift:].view(rows, k + pad)[:, :k]
    xd.copy_(torch.from_numpy(_wide(rng, rows, k)))
    w = torch.from_numpy(rng.normal(0, 1, (n, k)).astype(np.float32)).cuda()
    g = Guarded(rows * (n + pad) + shift, DT[y], 0)
    out = g.t[shift:].view(rows, n + pad)[:, :n]
    assert fsp.Fp8Linear(w).forward(xd, out=out) is out
    want, mag = _product(_values(xd), _values(w))
    tol = _tolerance(k, mag)
    if y == "bf16":
        assert rounds_to(_values(out), want, tol).all()
    else:
        assert (np.abs(_values(out) - want) <= tol).all()
    if pad:
        assert float(g.t[shift:].view(rows, n + pad)[:, n:].abs().sum()) == 0
    assert g.guards_intact()


def test_few_rows_with_a_non_finite_value():
    x = torch.ones(2, 300, device="cuda")
    x[1, 200] = float("inf")
    y = _values(fsp.Fp8Linear(torch.ones(40, 300, device="cuda")).forward(x, out_dtype=torch.float32))
    assert (y[0] == 300).all() and np.isnan(y[1]).all()


def test_empty_layers():
    w = torch.ones(6, 5, device="cuda")
    layer = fsp.Fp8Linear(w, train=True)
    assert layer.forward(torch.ones(0, 5, device="cuda")).shape == (0, 6)
    dw = torch.ones(6, 5, device="cuda")
    e = torch.zeros(0, 5, device="cuda")
    assert layer.backward(e, torch.zeros(0, 6, device="cuda"), dw, accumulate=True).shape == (0, 5) and float(dw.sum()) == 30
    layer.backward(e, torch.zeros(0, 6, device="cuda"), dw)
    assert float(dw.abs().sum()) == 0
    none = fsp.Fp8Linear(torch.ones(6, 0, device="cuda"))
    assert float(none.forward(torch.ones(3, 0, device="cuda")).abs().sum()) == 0


def test_gradients_against_differences():
    """On values that 8 bits hold exactly the layer is linear, and so the
    difference quotients of L = sum(dy * y) are exact."""
    rng = np.random.default_rng(1)
    ints = lambda *s: rng.integers(-4, 5, s).astype(np.float64)  # noqa: E731
    x, w, dy, ex, ew = ints(20, 150), ints(30, 150), ints(20, 30), ints(20, 150), ints(30, 150)
    dev = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731

    def loss(x, w):
        return (dy * _values(fsp.Fp8Linear(dev(w)).forward(dev(x), out_dtype=torch.float32))).sum()
    layer = fsp.Fp8Linear(dev(w), train=True)
    dw, dx = torch.empty(30, 150, device="cuda"), torch.empty(20, 150, device="cuda")
    layer.backward(dev(x), dev(dy), dw, out=dx)
    assert loss(x + ex, w) - loss(x, w) == (_values(dx) * ex).sum()
    assert loss(x, w + ew) - loss(x, w) == (_values(dw) * ew).sum()


def test_refusals():
    x = torch.zeros(4, 256, device="cuda")
    q = fsp.quantize_fp8(x)
    for bad in (lambda: fsp.quantize_fp8(x.half()), lambda: fsp.matmul_fp8(q, q, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: fsp.quantize_fp8(x.cpu()), lambda: fsp.quantize_fp8(x.t()), lambda: fsp.quantize_fp8(x[0]),
                lambda: fsp.quantize_fp8(x, fsp.Fp8Matrix(4, 255)), lambda: fsp.matmul_fp8(q, fsp.quantize_fp8(x[:, :128])),
                lambda: fsp.matmul_fp8(q, q, accumulate=True), lambda: fsp.matmul_fp8(q, q, out=x),
                lambda: fsp.Fp8Linear(x).backward(x, x[:, :4]), lambda: fsp.Fp8Linear(x).forward(x[:, :255])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fsp.FspError, match="both NULL"):
        fsp.quantize_fp8(x, None, None)
    with pytest.raises(fsp.FspError, match="fp32 only"):
        fsp.matmul_fp8(q, q, out=torch.zeros(4, 4, dtype=torch.bfloat16, device="cuda"), accumulate=True)
    with pytest.raises(fsp.FspError, match="overlaps"):
        fsp.matmul_fp8(q, q, out=q.data[:64].view(torch.float32).view(4, 4))


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_few_rows_of_huge_and_tiny_values(rows, out):
    """The scales of x and w may lie anywhere: what a product stands for is in range
    although x's value times w's code is not."""
    rng = np.random.default_rng(rows)
    k, n = 700, 40
    x, w = rng.normal(0, 1, (rows, k)), rng.normal(0, 1, (n, k))
    ex = np.repeat([124, -120, 90, -122, 0, 60], 128)[:k].astype(np.float64)   # powers of two, by block
    x *= np.exp2(ex) * 0.5
    x = np.clip(x, -3.3e38, 3.3e38)
    w *= np.exp2(-ex)
    x[0, 5] = 3.4e38   # rounds to 2^128, beside a zero of w
    w[:, 5] = 0
    xd, wd = torch.from_numpy(x.astype(np.float32)).cuda(), torch.from_numpy(w.astype(np.float32)).cuda()
    want, mag = _product(_values(xd), _values(wd))
    assert np.isfinite(want).all() and np.abs(want).max() < 1e4
    got = _values(fsp.Fp8Linear(wd).forward(xd, out_dtype=DT[out]))
    tol = _tolerance(k, mag)
    if out == "bf16":
        assert rounds_to(got, want, tol).all()
    else:
        assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("m,n,k", [(257, 7680, 128), (300, 7680, 1), (384, 7700, 640), (700, 3457, 900), (300, 20000, 200)])
def test_launches_that_follow_pairs_with_an_idle_second_cta(m, n, k):
    """Tiles of 256 rows whose second half lies past the matrix: that CTA writes nothing
    and is done as soon as the last sum is, while the next launch waits for its place."""
    g = torch.Generator(device="cuda").manual_seed(m + n)
    a = torch.randint(-8, 9, (m, k), generator=g, device="cuda").float()
    b = torch.randint(-8, 9, (n, k), generator=g, device="cuda").float()
    want = a.double() @ b.double().t()   # 8 bits hold the operands, fp32 the sums: exact
    qa, qb = fsp.quantize_fp8(a), fsp.quantize_fp8(b)
    outs = [torch.full((m, n), float("nan"), device="cuda") for _ in range(40)]
    for y in outs:
        fsp.matmul_fp8(qa, qb, out=y)
    assert all(bool((y == want).all()) for y in outs) and fsp.device_error() == 0


@pytest.mark.parametrize("m,n,k", [(1500, 2600, 4100), (4099, 3001, 1030), (256, 40000, 8200)])
def test_pairs_read_what_both_ctas_copied(m, n, k):
    """Many rounds of the ring of stages, on operands written just before, each launch on
    others: a stage read before either CTA's copies have landed shows the last ones."""
    g = torch.Generator(device="cuda").manual_seed(k)
    y = torch.empty(m, n, device="cuda")
    for _ in range(8):
        a = torch.randint(-8, 9, (m, k), generator=g, device="cuda").float()
        b = torch.randint(-8, 9, (n, k), generator=g, device="cuda").float()
        fsp.matmul_fp8(fsp.quantize_fp8(a), fsp.quantize_fp8(b), out=y)
        # 8 bits hold the operands, fp32 the sums (below 64 x 8200): exact
        assert torch.equal(y, (a.double() @ b.double().t()).float())
    assert fsp.device_error() == 0


@pytest.mark.parametrize("m,n", [(64, 64), (200, 130)])
def test_waits_of_milliseconds(m, n):
    """One tile's sum over four million terms: its readers wait for it far longer than
    one attempt of the hardware's does."""
    k = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(m)
    a = torch.randint(-1, 2, (m, k), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    b = torch.randint(-1, 2, (n, k), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    y = fsp.matmul_fp8(fsp.quantize_fp8(a), fsp.quantize_fp8(b), out_dtype=torch.float32)
    want = torch.zeros(m, n, device="cuda")
    for c in range(0, k, 1 << 18):   # (each part, and their sum, is a whole number below 2^24)
        want += a[:, c:c + (1 << 18)].float() @ b[:, c:c + (1 << 18)].float().t()
    assert torch.equal(y, want) and fsp.device_error() == 0
