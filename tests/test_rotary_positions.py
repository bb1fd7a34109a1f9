"""Rotary phases and far positions against the frequencies themselves, in whole-number arithmetic."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import fsdp_sharded_mixed_pass_gb300 as fsp
from fsdp_sharded_mixed_pass_gb300 import fsp as B

import block_reference as R

# pi to 120 digits
PI = Fraction(int("3141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117067982148086513282306647"), 10 ** 120)
HALF_UNIT = Fraction(1, 2 ** 65) * (1 + Fraction(1, 2 ** 9))   # of 2^-64 turn, and what the product's cut leaves


@pytest.fixture(scope="module", autouse=True)
def _built():
    import os
    if not os.path.exists(B.LIB_PATH):
        from fsdp_sharded_mixed_pass_gb300 import build
        build.build()


def _off(turns):
    """Distance to the nearest whole turn."""
    turns %= 1
    return min(turns, 1 - turns)


def test_phases_are_rounded_once():
    rng = np.random.default_rng(0)
    f = [0.0, 1.0, -1.0, 2.0 ** -64, 2.0 ** -70, -5e-324, 1e-300, 6.283185307179586, 2.0 ** 63, -np.nextafter(2.0 ** 64, 0), 2.0 ** 53 + 2]
    f += [10000.0 ** (-2 * j / 128) for j in range(64)] + [500000.0 ** (-2 * j / 128) / 8 for j in range(64)]
    f += list(rng.normal(0, 1, 200) * 2.0 ** rng.integers(-80, 60, 200))
    got = (ctypes.c_uint64 * len(f))()
    assert B.lib().fsp_rotary_phases((ctypes.c_double * len(f))(*f), len(f), got) == B.FSP_OK
    for x, g in zip(f, got):
        assert _off(Fraction(g, 2 ** 64) - Fraction(x) / (2 * PI)) <= HALF_UNIT, x
    for bad in (2.0 ** 64, -2.0 ** 64, 1e300, float("inf"), float("nan")):
        assert B.lib().fsp_rotary_phases((ctypes.c_double * 1)(bad), 1, got) == B.FSP_EINVAL and B.lib().fsp_last_error()


@pytest.mark.gpu
def test_far_positions_against_the_frequencies():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pos = [1, 2 ** 31 - 1, 2 ** 31 + 7, 10 ** 12 + 3, 2 ** 40 + 12345, -2 ** 40 - 999, 2 ** 44]
    x = torch.randn(len(pos), 3, 128, device="cuda")
    for kw in (dict(), dict(base=500000.0, scaling="linear", factor=8.0, layout="interleaved")):
        rope = fsp.Rotary(128, **kw)
        turns = [[Fraction(f) * t / (2 * PI) for f in rope.frequencies] for t in pos]
        angle = np.array([[float((u + Fraction(1, 2)) % 1 - Fraction(1, 2)) for u in row] for row in turns]) * 2 * np.pi
        want, mag = R.rotate(x.double().cpu().numpy(), angle, 128, rope.layout == "half", 1.0)
        for i, t in enumerate(pos):
            # the phase's half unit, t times, beside what the rotation itself may be off
            tol = (R.ROTARY_TOL + float(HALF_UNIT * abs(t)) * 2 * np.pi) * mag[i]
            assert (np.abs(rope.forward(x, torch.tensor(pos, device="cuda")).double().cpu().numpy()[i] - want[i]) <= tol).all(), t
    assert fsp.device_error() == 0
