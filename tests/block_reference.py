"""Plain statements in 64 bits (the generator in whole numbers) of layer norm, dropout and
rotary positions, with what fp32 arithmetic may add to them.  Host only."""
import numpy as np

U = 2.0 ** -24   # half a step of fp32, relative


def depth(n):
    """Most additions that a term of a row's sum goes through.  Rows of up to 128 elements: at most 16 of a
    thread's own and four steps of its group; longer ones are shared by at least 16 threads, whose sums are joined in
    16 steps or, from 4097 elements on (256 and more of the first term), 5 among lanes and 16 or 32 warps."""
    return -(-n // 16) + 16


# ---- layer norm -----------------------------------------------------------------------

def norm(x, w, b, eps, center):
    """(y, mean, 1 / deviation) and fp32's bounds on the three."""
    x = np.asarray(x, np.float64)
    n = x.shape[1]
    m = x.mean(1, keepdims=True) if center else np.zeros((len(x), 1))
    c = x - m
    var = (c * c).mean(1, keepdims=True)
    r = 1 / np.sqrt(var + eps)
    h = c * r
    y = h * w + b
    # the mean: a term goes through `depth` additions, then the division, or 1 / n and a product
    em = (depth(n) + 2) * U * np.abs(x).mean(1, keepdims=True) if center else 0 * m
    ec = em + U * np.abs(c)
    # the variance: its terms' own error, the additions, the division, eps
    ev = (2 * np.abs(c) * ec + ec * ec).mean(1, keepdims=True) + (depth(n) + 4) * U * (var + eps)
    with np.errstate(divide="ignore", invalid="ignore"):
        er = 0.5 * ev / (var + eps - np.minimum(ev, 0.5 * (var + eps))) + 4 * U   # relative; root and division, or a root of two steps of 2^-23
    eh = ec * r * (1 + er) + np.abs(h) * (er + 2 * U)
    ey = np.abs(w) * eh + U * (np.abs(y) + np.abs(h * w) * 0) + 2 * U * np.abs(h * w)
    return (y, m[:, 0], r[:, 0]), (ey, em[:, 0] + U * np.abs(m[:, 0]), (er * r)[:, 0])


def norm_gradients(x, m, r, dy, w, add, center):
    """(dx, dw, db) of given fp32 statistics, and fp32's bounds on them."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    m, r = np.asarray(m, np.float64)[:, None], np.asarray(r, np.float64)[:, None]
    rows, n = x.shape
    h, g = (x - m) * r, dy * w
    eh, eg = 3 * U * np.abs(h), U * np.abs(g)
    mean = lambda t: t.mean(1, keepdims=True)  # noqa: E731
    mg = mean(g) if center else 0 * m
    mgh = mean(g * h)
    d = (depth(n) + 3) * U
    emg = (mean(eg) + d * mean(np.abs(g))) if center else 0 * m
    emgh = mean(np.abs(g) * eh + np.abs(h) * eg) + (d + U) * mean(np.abs(g * h))
    inner = g - mg - h * mgh
    size = np.abs(g) + np.abs(mg) + np.abs(h * mgh)
    einner = eg + emg + np.abs(h) * emgh + np.abs(mgh) * eh + 4 * U * size
    dx = r * inner + add
    edx = np.abs(r) * (einner + 2 * U * size) + U * (np.abs(dx) + np.abs(add))
    # over the rows: each of at most `rows` additions
    dw, db = (dy * h).sum(0), dy.sum(0)
    edw = (np.abs(dy) * eh + 2 * U * np.abs(dy * h)).sum(0) + rows * U * np.abs(dy * h).sum(0)
    edb = rows * U * np.abs(dy).sum(0)
    return (dx, dw, db), (edx, edw, edb)


# ---- dropout ----------------------------------------------------------------------------

def philox(counter, key):
    """Philox-4x32 of ten rounds: counter and key as lists of 4 and 2 words (arrays or numbers)."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        u, v = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        hi, lo = (lambda t: t >> np.uint64(32)), (lambda t: t & low)
        c = [hi(v) ^ c[1] ^ np.uint64(k[0]), lo(v), hi(u) ^ c[3] ^ np.uint64(k[1]), lo(u)]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def random16(n, seed, call):
    """The n numbers of 16 bits of (seed, call)."""
    i = np.arange((n + 7) // 8, dtype=np.uint64)
    one = np.ones_like(i)
    words = lambda v: ((v & 0xFFFFFFFF), ((v >> 32) & 0xFFFFFFFF))  # noqa: E731
    lo, hi = words(call)
    c = philox([i & np.uint64(0xFFFFFFFF), i >> np.uint64(32), one * np.uint64(lo), one * np.uint64(hi)], words(seed))
    w = np.stack(c, 1)
    return np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)[:n].astype(np.int64)


def dropout(x, p, seed, call, residual=0.0):
    """(y, keep) with the scale exact."""
    lost = int(np.floor(p * 65536 + 0.5))
    keep = (random16(x.size, seed, call) >= lost).reshape(x.shape)
    scale = 65536 / (65536 - lost) if lost < 65536 else 0.0
    with np.errstate(invalid="ignore"):
        return np.where(keep, np.asarray(x, np.float64) * scale, 0.0) + residual, keep


# ---- rotary positions ----------------------------------------------------------------------

def angles(positions, phases):
    """Radians in (-pi, pi] of whole-number phases (2^-64 turn), without rounding before the last step."""
    out = np.empty((len(positions), len(phases)))
    for i, t in enumerate(positions):
        for j, f in enumerate(phases):
            turn = int(t) * int(f) % 2 ** 64
            out[i, j] = (turn if turn < 2 ** 63 else turn - 2 ** 64) / 2.0 ** 64 * 2 * np.pi
    return out


def rotate(x, angle, dim, half, scale):
    """x (..., tokens, heads, head_dim) turned, and the sum of magnitudes of each result's terms."""
    x = np.asarray(x, np.float64)
    c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
    first, second = (slice(0, dim // 2), slice(dim // 2, dim)) if half else (slice(0, dim, 2), slice(1, dim, 2))
    a, b = x[..., first], x[..., second]
    y, mag = x.copy(), np.zeros_like(x)
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    mag[..., first] = mag[..., second] = abs(scale) * (np.abs(a) + np.abs(b))
    return y, mag


# the angle: its float rounding (2^-24 of at most pi) and the cut below 2^-32 turn (2 pi); sine and cosine: 2 steps
# of 2^-24; the scale, two products and the sum: 2^-24 each
ROTARY_TOL = (np.pi + 2 * np.pi * 2.0 ** -8 + 2 * 2 + 4) * U
