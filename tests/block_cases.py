"""Matrices in guarded device buffers, for the tests of the operators on rows."""
import numpy as np
import torch

from gpu_cases import Guarded

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def values(x):
    return x.detach().float().cpu().numpy().astype(np.float64)


def matrix(rows, cols, dtype, pad=0, shift=0, fill=None):
    """(rows x cols with `pad` elements between rows, `shift` elements off alignment; a check that
    nothing around its elements was written)."""
    g = Guarded(rows * (cols + pad) + shift, DT[dtype], 0)
    whole = g.t[shift:].view(rows, cols + pad)
    t = whole[:, :cols]
    if fill is not None:
        t.copy_(torch.from_numpy(np.asarray(fill, np.float32)))
    return t, lambda: g.guards_intact() and (not pad or float(whole[:, cols:].abs().sum()) == 0) and not bool(g.t[:shift].any())


def off_by(got, want, tol, dtype):
    """Elements outside `tol` of `want`, plus the one rounding of bf16 results (half a step, 2^-8 of the value)."""
    got = values(got) if isinstance(got, torch.Tensor) else got
    with np.errstate(invalid="ignore"):
        tol = tol + (2.0 ** -8 * (np.abs(want) + tol) if dtype == "bf16" else 0) + 1e-37   # (below the normal range steps are even)
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        bad = ~(same | (np.abs(got - want) <= tol))
    return int(bad.sum())
