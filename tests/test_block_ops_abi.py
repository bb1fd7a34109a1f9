"""Layer norm, dropout and rotary positions on the host: what the C entry points refuse before any launch,
the sizes and tables they state, and the statements that the GPU tests compare with."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import fsdp_sharded_mixed_pass_gb300 as fsp
from fsdp_sharded_mixed_pass_gb300 import fsp as B
from fsdp_sharded_mixed_pass_gb300 import ops

import block_reference as R

FAKE = 1 << 44   # never dereferenced on the host
GAP = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from fsdp_sharded_mixed_pass_gb300 import build
        build.build()
    return B.lib()


def _norm(lib, x=FAKE, xd=0, rows=4, dim=8, xs=8, w=None, b=None, pd=0, eps=1e-5, center=1, out=FAKE + GAP, od=0, os_=8, stats=None):
    return lib.fsp_layer_norm(x, xd, rows, dim, xs, w, b, pd, eps, center, out, od, os_, stats, None)


def test_layer_norm_refusals(lib):
    assert _norm(lib, rows=0) == B.FSP_OK and _norm(lib, x=None, out=None, dim=0) == B.FSP_OK
    for kw in (dict(rows=-1), dict(dim=-1), dict(xd=2), dict(od=-1), dict(xs=7), dict(os_=7), dict(x=None), dict(out=None),
               dict(x=FAKE + 2), dict(w=FAKE + 1, pd=1), dict(w=FAKE, pd=5), dict(eps=-1e-9), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(stats=FAKE + 4), dict(out=FAKE + 4), dict(out=FAKE, os_=9), dict(out=FAKE, od=1),
               dict(out=FAKE + 64, w=FAKE + 64, x=FAKE + GAP), dict(stats=FAKE + 8), dict(stats=FAKE + GAP), dict(xs=1 << 57)):
        assert _norm(lib, **kw) == B.FSP_EINVAL, kw
        assert lib.fsp_last_error()
    assert _norm(lib, dim=(1 << 20) + 1, xs=1 << 21, os_=1 << 21) == B.FSP_EUNSUPPORTED
    assert _norm(lib, rows=1 << 31) == B.FSP_EUNSUPPORTED


def test_columns_of_their_own_within_the_same_rows(lib):
    """A result beside its input in one buffer's rows: past the checks of the arguments, only the memory is not there."""
    there = lambda status: status not in (B.FSP_OK, B.FSP_EINVAL) or b"allocation" in lib.fsp_last_error()  # noqa: E731
    for off in (32, 64, -32, 32 + 96, -64):
        assert there(_norm(lib, xs=24, os_=24, out=FAKE + off)) and there(_drop(lib, xs=24, os_=24, out=FAKE + off)), off
        assert there(_norm(lib, xs=24, os_=48, od=1, out=FAKE + off)) and there(_norm(lib, xs=24, os_=24, out=FAKE))
    for off in (28, 68, -28, -68, 96):
        assert _norm(lib, xs=24, os_=24, out=FAKE + off) == B.FSP_EINVAL and b"overlaps" in lib.fsp_last_error(), off
    assert _norm(lib, xs=24, os_=25, out=FAKE + 32) == B.FSP_EINVAL and _norm(lib, xs=24, os_=48, od=1, out=FAKE) == B.FSP_EINVAL


def _grad(lib, x=FAKE, xd=0, rows=4, dim=8, xs=8, stats=FAKE + GAP, dy=FAKE + 2 * GAP, gd=0, gs=8, w=None, wd=0, add=None, as_=8,
          dx=FAKE + 3 * GAP, ds=8, dw=FAKE + 4 * GAP, db=None, pd=0, acc=0, work=FAKE + 5 * GAP, work_bytes=1 << 20):
    return lib.fsp_layer_norm_backward(x, xd, rows, dim, xs, stats, 1, dy, gd, gs, w, wd, add, as_, dx, ds, dw, db, pd, acc, work,
                                       work_bytes, None)


def test_layer_norm_backward_refusals(lib):
    assert _grad(lib, rows=0, acc=1) == B.FSP_OK and _grad(lib, dim=0) == B.FSP_OK and _grad(lib, dx=None, dw=None) == B.FSP_OK
    for kw in (dict(rows=-1), dict(dim=-8), dict(xd=2), dict(gd=2), dict(xs=7), dict(gs=7), dict(x=None), dict(dy=None), dict(stats=None),
               dict(stats=FAKE + GAP + 4), dict(w=FAKE + 6 * GAP, wd=3), dict(pd=3), dict(add=FAKE + 6 * GAP, as_=7), dict(ds=7),
               dict(add=FAKE + 6 * GAP, dx=None), dict(rows=4000, work=None), dict(rows=4000, work_bytes=255), dict(rows=4000, work=FAKE + 5 * GAP + 8),
               dict(dx=FAKE + 4), dict(dx=FAKE, ds=9), dict(dw=FAKE), dict(db=FAKE + 4 * GAP + 4), dict(rows=4000, work=FAKE + 3 * GAP),
               dict(w=FAKE + 3 * GAP), dict(dw=FAKE + 4 * GAP + 2), dict(dx=FAKE + GAP)):
        assert _grad(lib, **kw) == B.FSP_EINVAL, kw
        assert lib.fsp_last_error()
    size = ctypes.c_size_t()
    bytes_of = lib.fsp_layer_norm_backward_workspace_bytes
    assert bytes_of(4, 8, None) == B.FSP_EINVAL and bytes_of(-1, 8, ctypes.byref(size)) == B.FSP_EINVAL
    assert bytes_of(4, (1 << 20) + 1, ctypes.byref(size)) == B.FSP_EUNSUPPORTED
    assert bytes_of(100000, 1024, ctypes.byref(size)) == B.FSP_OK and 1024 * 8 <= size.value <= 1024 * 8 * 1024
    for rows, dim in ((0, 1 << 20), (1, 8192), (2, 5000), (16, 1024), (128, 3)):   # what one CTA takes
        assert bytes_of(rows, dim, ctypes.byref(size)) == B.FSP_OK and size.value == 0
    for rows, dim in ((1, 8193), (3, 8192), (17, 1024), (129, 3)):
        assert bytes_of(rows, dim, ctypes.byref(size)) == B.FSP_OK and size.value >= dim * 8


def _drop(lib, x=FAKE, xd=0, rows=4, dim=8, xs=8, p=0.5, call=None, h=None, hd=0, hs=8, out=FAKE + GAP, od=0, os_=8):
    return lib.fsp_dropout(x, xd, rows, dim, xs, p, 1, 2, call, h, hd, hs, out, od, os_, None)


def test_dropout_refusals(lib):
    assert _drop(lib, rows=0) == B.FSP_OK and _drop(lib, dim=0) == B.FSP_OK
    for kw in (dict(rows=-1), dict(dim=-1), dict(xd=2), dict(od=3), dict(h=FAKE + 2 * GAP, hd=4), dict(h=FAKE + 2 * GAP, hs=7), dict(xs=7),
               dict(os_=7), dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(x=None), dict(out=None), dict(call=FAKE + 4),
               dict(out=FAKE + 4), dict(out=FAKE, od=1), dict(h=FAKE + GAP + 4), dict(call=FAKE + GAP)):
        assert _drop(lib, **kw) == B.FSP_EINVAL, kw
        assert lib.fsp_last_error()


def _rotary(lib, tensors=None, n=None, dtype=1, batch=1, tokens=4, pos=FAKE + 9 * GAP, size=8, ps=0, phases=FAKE + 8 * GAP, dim=64,
            layout=0, scale=1.0):
    tensors = [dict()] if tensors is None else tensors
    arr = (ops._RotaryTensor * max(1, len(tensors)))()
    for k, (t, kw) in enumerate(zip(arr, tensors)):
        kw = dict(dict(x=FAKE + k * GAP, out=FAKE + (k + 4) * GAP, heads=2, head_dim=64, xs=(512, 128, 64), os_=(512, 128, 64)), **kw)
        t.x, t.out, t.heads, t.head_dim = kw["x"], kw["out"], kw["heads"], kw["head_dim"]
        t.x_strides[:], t.out_strides[:] = kw["xs"], kw["os_"]
    return lib.fsp_rotary(arr, len(tensors) if n is None else n, dtype, batch, tokens, pos, size, ps, phases, dim, layout, scale, 0, None)


def test_rotary_refusals(lib):
    assert _rotary(lib, tokens=0) == B.FSP_OK and _rotary(lib, [dict(heads=0)]) == B.FSP_OK and _rotary(lib, batch=0) == B.FSP_OK
    for kw in (dict(n=0), dict(n=3), dict(dtype=2), dict(batch=-1), dict(tokens=-1), dict(size=2), dict(layout=2), dict(dim=0), dict(dim=63),
               dict(dim=66), dict(scale=float("nan")), dict(ps=3), dict(ps=1 << 60, batch=4), dict(pos=None), dict(phases=None), dict(pos=FAKE + 4),
               dict(phases=FAKE + 4), dict(pos=FAKE + 4 * GAP), dict(phases=FAKE + 4 * GAP + 64)):
        assert _rotary(lib, **kw) == B.FSP_EINVAL, kw
        assert lib.fsp_last_error()
    for t in (dict(x=None), dict(out=None), dict(x=FAKE + 1), dict(heads=-1), dict(head_dim=32), dict(head_dim=1 << 17), dict(heads=1 << 21),
              dict(xs=(0, -1, 64)), dict(xs=(0, 1 << 60, 64)), dict(os_=(0, 64, 64)), dict(os_=(0, 0, 64)), dict(os_=(512, 128, 32)),
              dict(out=FAKE + 2), dict(out=FAKE, os_=(512, 192, 64))):
        assert _rotary(lib, [t]) == B.FSP_EINVAL, t
        assert _rotary(lib, [dict(x=FAKE + 2 * GAP, out=FAKE + 3 * GAP), dict(dict(x=FAKE, out=FAKE + 4 * GAP), **t)]) == B.FSP_EINVAL, t
    # a batch of outputs that share their places
    assert _rotary(lib, [dict(os_=(0, 128, 64))], batch=2) == B.FSP_EINVAL
    # one's output within the other's input
    assert _rotary(lib, [dict(), dict(out=FAKE)]) == B.FSP_EINVAL
    assert _rotary(lib, [dict(out=FAKE, xs=(0, 192, 64), os_=(0, 192, 64)), dict(x=FAKE + 192, xs=(0, 192, 64))]) == B.FSP_EINVAL
    # an input that repeats its heads, under the output's span
    for xs in ((0, 128, 64), (512, 0, 64), (512, 128, 0), (0, 0, 0)):
        assert _rotary(lib, [dict(xs=xs, os_=(1024, 256, 64), out=FAKE + 64)], batch=2) == B.FSP_EINVAL and b"overlaps" in lib.fsp_last_error()
    assert _rotary(lib, tokens=1 << 30, batch=1 << 30) == B.FSP_EUNSUPPORTED


def test_rotary_accepts_heads_within_one_projection(lib):
    """Queries and keys in place within rows of one buffer: past the checks of the arguments, only the memory is not there."""
    inside = lambda off, heads: dict(x=FAKE + off, out=FAKE + off, heads=heads, xs=(4 * 384, 384, 64), os_=(4 * 384, 384, 64))  # noqa: E731
    for tensors, batch in (([inside(0, 3), inside(2 * 192, 1)], 1), ([inside(0, 3), inside(2 * 192, 1)], 3), ([inside(2 * 192, 1), inside(0, 3)], 1)):
        assert _rotary(lib, tensors, batch=batch) not in (B.FSP_OK, B.FSP_EINVAL) or b"allocation" in lib.fsp_last_error()
    assert _rotary(lib, [inside(0, 4), inside(2 * 192, 1)]) == B.FSP_EINVAL and b"overlaps" in lib.fsp_last_error()


# pi to 60 digits
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def test_phases_are_the_frequencies_in_turns(lib):
    f = [1.0, 1e-4, 0.0, 6.5, -0.25, 1234.5678, 2.0 ** -80, 10000.0 ** (-62 / 64)]
    got = (ctypes.c_uint64 * len(f))()
    assert lib.fsp_rotary_phases((ctypes.c_double * len(f))(*f), len(f), got) == B.FSP_OK
    for x, g in zip(f, got):
        turns = Fraction(x) / (2 * PI)
        off = (Fraction(g, 2 ** 64) - turns) % 1
        off = min(off, 1 - off)
        # 2 pi's and the division's rounding (2^-53 each, relative), and the cut below 2^-64
        assert off <= abs(turns) * Fraction(1, 2 ** 52) + Fraction(1, 2 ** 64)
    for bad in (float("inf"), float("nan")):
        assert lib.fsp_rotary_phases((ctypes.c_double * 1)(bad), 1, got) == B.FSP_EINVAL
    assert lib.fsp_rotary_phases(None, 1, got) == B.FSP_EINVAL and lib.fsp_rotary_phases(None, -1, None) == B.FSP_EINVAL
    assert lib.fsp_rotary_phases(None, 0, None) == B.FSP_OK


def test_rotary_frequencies():
    plain = fsp.Rotary(64, base=500.0, device="cpu")
    assert plain.frequencies == tuple(500.0 ** (-2 * j / 64) for j in range(32)) and plain.scale == 1.0
    assert fsp.Rotary(64, 500.0, scaling="linear", factor=4.0, device="cpu").frequencies == tuple(f / 4 for f in plain.frequencies)
    ntk = fsp.Rotary(64, 500.0, scaling="ntk", factor=4.0, device="cpu").frequencies
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], plain.frequencies[-1] / 4, rel_tol=1e-12)   # the slowest pair is stretched by the factor
    yarn = fsp.Rotary(64, 500.0, scaling="yarn", factor=4.0, original_length=1000, device="cpu")
    for f, g in zip(plain.frequencies, yarn.frequencies):
        t = 1000 * f / (2 * math.pi)
        assert math.isclose(g, f if t >= 32 else f / 4 if t <= 1 else f / 4 + (f - f / 4) * (t - 1) / 31, rel_tol=1e-12)
    assert yarn.scale == 0.1 * math.log(4.0) + 1 and yarn.frequencies[0] == 1.0
    own = fsp.Rotary(4, frequencies=[0.5, 0.25], scale=2.0, device="cpu")
    assert own.frequencies == (0.5, 0.25) and own.scale == 2.0
    for kw in (dict(dim=3), dict(dim=0), dict(layout="pairs"), dict(scaling="cubic"), dict(scaling="yarn", factor=2.0), dict(factor=0.0),
               dict(frequencies=[1.0]), dict(frequencies=[1.0, 2.0], scaling="linear"), dict(base=-1.0),
               dict(scaling="yarn", factor=2.0, original_length=10, turns=(2, 2))):
        with pytest.raises(ValueError):
            fsp.Rotary(**dict(dict(dim=4, device="cpu"), **kw))
    with pytest.raises(fsp.FspError, match="finite"):
        fsp.Rotary(4, frequencies=[1.0, float("inf")], device="cpu")


def test_the_generator_gives_its_authors_answers():
    """The three known answers published with Philox-4x32-10."""
    for counter, key, want in (
            ([0] * 4, [0] * 2, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
            ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0], "d16cfe09 94fdcceb 5001e420 24126ea1")):
        assert " ".join(f"{int(v):08x}" for v in R.philox(counter, key)) == want


def test_the_statements_agree_with_differences():
    """The gradients that the GPU tests compare with are those of the forward statement (central differences)."""
    rng = np.random.default_rng(0)
    x, dy, dirx = rng.normal(0, 1, (3, 4, 9))
    w, b, dirw = rng.normal(1, 0.3, (3, 9))
    for center in (True, False):
        f = lambda t: (R.norm(x + t * dirx, w + t * dirw, b + t, 1e-5, center)[0][0] * dy).sum()  # noqa: E731
        (_, m, r), _ = R.norm(x, w, b, 1e-5, center)
        (dx, dw, db), _ = R.norm_gradients(x, m, r, dy, w, 0.0, center)
        slope = (f(1e-5) - f(-1e-5)) / 2e-5
        assert abs(slope - ((dx * dirx).sum() + (dw * dirw).sum() + db.sum())) <= 1e-7 * np.abs(dy).sum()
    angle = rng.uniform(-3, 3, (4, 4))
    for half in (True, False):
        y = lambda v, a: R.rotate(v, a, 8, half, 1.5)[0]  # noqa: E731
        a, d = x[:, None, :], dy[:, None, :]
        assert np.isclose((y(a, angle) * d).sum(), (a * y(d, -angle))[..., :8].sum() + (a * d)[..., 8:].sum())


def test_tensors_elsewhere_than_the_current_device_are_refused():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 8)
    here = ops._current
    ops._current = lambda: 0
    try:
        rope = fsp.Rotary(8, device="cpu")
        for call in (lambda: fsp.layer_norm(x), lambda: fsp.layer_norm_backward(x, torch.zeros(4, 2), x), lambda: fsp.dropout(x, 0.1, 1),
                     lambda: rope.forward(x[:, None], torch.zeros(4, dtype=torch.int64))):
            with pytest.raises(ValueError, match="CUDA device"):
                call()
    finally:
        ops._current = here
