"""Plain statements, in 64 bits (and, for the codes, in separately rounded fp32
operations), of the operators beside the sharded step.  Host only."""
import numpy as np

BLOCK = 256


# ---- AdamW's 8-bit states -----------------------------------------------------------

def codes(x, top, fourth_root):
    """(codes, scales) of whole blocks of fp32 values, every operation rounded to fp32."""
    b = np.asarray(x, np.float32).reshape(-1, BLOCK)
    s = np.abs(b).max(1)
    with np.errstate(invalid="ignore", divide="ignore"):
        r = np.sqrt(np.abs(b) / np.where(s > 0, s, np.float32(1))[:, None])
        if fourth_root:
            r = np.sqrt(r)
        q = np.rint(r * np.float32(top))
    if fourth_root:
        q = np.where((b > 0) & (q == 0), 1, q)
    return (np.sign(b) * q).astype(np.int32).reshape(-1), s


def code_values(q, s, top, fourth_root):
    x = q.astype(np.float32).reshape(-1, BLOCK) * np.float32(1.0 / top)
    x = x * np.abs(x)
    if fourth_root:
        x = x * x
    return (s[:, None] * x).astype(np.float32).reshape(-1)


def moments_rounded(m, v, g, hp):
    """m' and v' with each product and sum rounded to fp32."""
    f = {k: np.float32(hp[k]) for k in hp}
    c1, c2 = np.float32(1.0 - float(f["beta1"])), np.float32(1.0 - float(f["beta2"]))
    m = m * f["beta1"] + g * c1
    v = v * f["beta2"] + (g * g) * c2
    return m.astype(np.float32), v.astype(np.float32)


# ---- embedding -----------------------------------------------------------------------

def embedding_gradient(tokens, dy, vocab, scale, old=None, padding_idx=None):
    """(gradient, sum of magnitudes, terms per row) in 64 bits."""
    dw = np.zeros((vocab, dy.shape[1])) if old is None else old.astype(np.float64)
    mag = np.zeros((vocab, dy.shape[1]))
    n = np.zeros(vocab, np.int64)
    for i, t in enumerate(tokens):
        if 0 <= t < vocab and t != padding_idx:
            dw[t] += scale * dy[i].astype(np.float64)
            mag[t] += abs(scale) * np.abs(dy[i].astype(np.float64))
            n[t] += 1
    return dw, mag, n


# ---- 8-bit floating point ----------------------------------------------------------------

def e4m3(y):
    """Nearest e4m3 value (ties to even) of |y| <= 448."""
    mag = np.abs(y)
    step = np.exp2(np.floor(np.log2(np.maximum(mag, 2.0 ** -6))) - 3)
    return np.sign(y) * np.rint(mag / step) * step


def fp8(x):
    """What x's rows, cut into blocks of 128, stand for as codes and scales."""
    x = np.asarray(x, np.float64)
    r, k = x.shape
    b = np.pad(x, ((0, 0), (0, -k % 128))).reshape(r, -1, 128)
    top = np.abs(b).max(2, keepdims=True)
    # the smallest e in [-127, 127] with top <= 448 2^e
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.ceil(np.log2(np.where((top > 0) & np.isfinite(top), top, 2.0 ** -150) / 448))
    e += top > 448 * np.exp2(e)          # (log2's own rounding)
    e -= top <= 448 * np.exp2(e - 1)
    e = np.maximum(e, -127.0)
    s = np.exp2(e)
    with np.errstate(invalid="ignore"):
        v = np.where(np.isfinite(top), e4m3(np.where(np.isfinite(top), b, 0) / s) * s, np.nan)
    return v.reshape(r, -1)[:, :k]


# ---- bf16 results ------------------------------------------------------------------------

def _bf16(x):
    """64-bit values rounded once to bf16 (8 significant bits, ties to even; normal range)."""
    x = np.asarray(x, np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 7)
    return np.rint(x / step) * step


def rounds_to(got, want, tol):
    """Whether each of `got` is the bf16 rounding of a value within `tol` of `want`
    (rounding is monotone, so it lies between the roundings of the ends)."""
    return (got >= _bf16(want - tol)) & (got <= _bf16(want + tol))
