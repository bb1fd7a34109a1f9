"""Rotary positions: both layouts, part of the head, far positions, strides, the gradient."""
import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp

import block_reference as R
from block_cases import DT, off_by, values
from gpu_cases import Guarded, ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _phases(rope):
    return rope.phases.cpu().numpy().view(np.uint64)


def _want(rope, x, positions, inverse=False):
    """(rotated, tolerance) of x (..., tokens, heads, head_dim), positions (tokens,)."""
    a = R.angles(positions, _phases(rope))
    y, mag = R.rotate(values(x), -a if inverse else a, rope.dim, rope.layout == "half", rope.scale)
    return y, R.ROTARY_TOL * mag


# tokens, heads, head_dim, dim
SIZES = [(1, 1, 2, 2), (3, 1, 8, 8), (1, 24, 128, 128), (5, 3, 16, 16), (7, 2, 18, 10), (4, 5, 80, 20), (33, 6, 64, 32), (2, 1, 48, 48), (9, 4, 64, 64),
         (17, 3, 96, 96), (6, 7, 256, 64), (3, 9, 90, 90), (2, 33, 128, 96), (5, 2, 40, 16), (4, 3, 136, 128), (2, 2, 1024, 1024), (300, 1, 32, 32)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,head_dim,dim", SIZES)
def test_rotation(tokens, heads, head_dim, dim, layout, dtype):
    rng = np.random.default_rng(tokens + head_dim)
    rope = fsp.Rotary(dim, layout=layout, scaling="yarn", factor=4.0, original_length=64)
    for shift, index in ((0, torch.int64), (1, torch.int32)):
        n = tokens * heads * head_dim
        x = torch.from_numpy(rng.normal(0, 1, n + shift).astype(np.float32)).to("cuda", DT[dtype])[shift:].view(tokens, heads, head_dim)
        pos = rng.integers(-5, 2 ** 31 - 1, tokens)
        pos[0] = 0
        p = torch.from_numpy(pos).to("cuda", index)
        g = Guarded(n + shift, DT[dtype], 0)
        out = g.t[shift:].view(tokens, heads, head_dim)
        assert rope.forward(x, p, out=out) is out
        want, tol = _want(rope, x, pos)
        assert off_by(out, want, tol, dtype) == 0
        assert torch.equal(out[..., dim:], x[..., dim:]) and g.guards_intact()
        back = rope.backward(x, p)
        want, tol = _want(rope, x, pos, inverse=True)
        assert off_by(back, want, tol, dtype) == 0 and torch.equal(back[..., dim:], x[..., dim:])
        here = x.clone()
        assert rope.forward(here, p, out=here) is here and torch.equal(here, out)
    assert fsp.device_error() == 0


# enough tokens for threads that take several heads and several narrow accesses; batches, one tensor or two
@pytest.mark.parametrize("dtype,layout,batch,tokens,heads,kv,head_dim,dim", [
    ("bf16", "half", 2, 1601, 11, 3, 90, 90), ("f32", "half", 1, 3001, 9, 2, 192, 118), ("bf16", "interleaved", 1, 4003, 7, 5, 146, 60),
    ("f32", "interleaved", 3, 2001, 5, 1, 84, 20), ("bf16", "half", 1, 30011, 5, 0, 128, 128), ("bf16", "interleaved", 2, 12007, 1, 1, 72, 8),
    ("f32", "half", 1, 40001, 1, 0, 20, 12), ("bf16", "half", 1, 5003, 6, 6, 100, 40), ("f32", "interleaved", 1, 9001, 2, 3, 34, 34)])
def test_many_tokens(dtype, layout, batch, tokens, heads, kv, head_dim, dim):
    """Against 64 bits on the device, out of a projection's rows into tensors of their own."""
    rope = fsp.Rotary(dim, layout=layout, scaling="ntk", factor=8.0)
    qkv = torch.randn(batch, tokens, heads + 2 * kv, head_dim, device="cuda").to(DT[dtype])
    q, k = qkv[:, :, :heads], qkv[:, :, heads:heads + kv]
    pos = torch.randint(0, 100000, (batch, tokens), device="cuda")
    turn = pos[:, :, None, None].double() * torch.tensor(rope.frequencies, dtype=torch.float64, device="cuda")
    got = rope.forward((q, k), pos), rope.backward((q, k), pos)
    for x, fwd, bwd in ((q, got[0][0], got[1][0]), (k, got[0][1], got[1][1])):
        for y, sign in ((fwd, 1), (bwd, -1)):
            a, b = (x[..., :dim // 2], x[..., dim // 2:dim]) if layout == "half" else (x[..., 0:dim:2], x[..., 1:dim:2])
            a, b, c, s = a.double(), b.double(), turn.cos(), sign * turn.sin()
            u, v = (y[..., :dim // 2], y[..., dim // 2:dim]) if layout == "half" else (y[..., 0:dim:2], y[..., 1:dim:2])
            # the angle at 100000 in doubles: 2^-52 of 10^5, far below
            tol = R.ROTARY_TOL * (a.abs() + b.abs())
            for out, want in ((u, a * c - b * s), (v, b * c + a * s)):
                assert bool(((out - want).abs() <= tol + (2.0 ** -8 * (want.abs() + tol) if dtype == "bf16" else 0)).all())
            assert torch.equal(y[..., dim:], x[..., dim:])
    buf = qkv.clone()
    bq, bk = buf[:, :, :heads], buf[:, :, heads:heads + kv]
    rope.forward((bq, bk), pos, out=(bq, bk))
    assert torch.equal(bq, got[0][0]) and torch.equal(bk, got[0][1]) and torch.equal(buf[:, :, heads + kv:], qkv[:, :, heads + kv:])
    # one tensor in place, the other not: only the other's rest is copied
    if kv:
        buf = qkv.clone()
        out = torch.full((batch, tokens, kv, head_dim), float("nan"), device="cuda", dtype=DT[dtype])
        rope.forward((buf[:, :, :heads], k), pos, out=(buf[:, :, :heads], out))
        assert torch.equal(buf[:, :, :heads], got[0][0]) and torch.equal(out, got[0][1])
    assert fsp.device_error() == 0


def test_position_zero_and_far_positions():
    x = torch.randn(4, 2, 64, device="cuda")
    rope = fsp.Rotary(64)
    assert torch.equal(rope.forward(x, torch.zeros(4, dtype=torch.int64, device="cuda")), x)
    pos = [2 ** 40 + 12345, -2 ** 40 - 999, 2 ** 62 + 1, -2 ** 63]   # whole turns are taken off exactly
    want, tol = _want(rope, x, pos)
    assert off_by(rope.forward(x, torch.tensor(pos, device="cuda")), want, tol, "f32") == 0
    # a turn that is a power of two repeats without any error
    rope = fsp.Rotary(2, frequencies=[2 * np.pi / 1024], layout="interleaved")
    y = [rope.forward(x[..., :2], torch.full((4,), t, device="cuda")) for t in (3, 3 + 1024 * 7)]
    assert float((y[0] - y[1]).abs().max()) <= 8 * R.U * float(x.abs().max())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,head_dim,dim", [("bf16", 64, 64), ("f32", 64, 32), ("bf16", 20, 12)])
def test_queries_and_keys_of_one_projection(layout, dtype, head_dim, dim):
    """Both out of (and back into) one buffer's rows, for batches with positions of their own or shared ones."""
    b, t, hq, hk = 3, 11, 6, 2
    rope = fsp.Rotary(dim, layout=layout)
    qkv = torch.randn(b, t, hq + 2 * hk, head_dim, device="cuda").to(DT[dtype])
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    shared = torch.randint(0, 5000, (t,), device="cuda")
    own = torch.randint(0, 5000, (b, t), device="cuda")
    for pos in (shared, own):
        yq, yk = rope.forward((q, k), pos)
        assert yq.is_contiguous() and yk.shape == k.shape
        for i in range(b):
            p = (pos if pos.dim() == 1 else pos[i]).cpu().numpy()
            for x, y in ((q, yq), (k, yk)):
                want, tol = _want(rope, x[i], p)
                assert off_by(y[i], want, tol, dtype) == 0
        buf = qkv.clone()
        bq, bk = buf[:, :, :hq], buf[:, :, hq:hq + hk]
        rope.forward((bq, bk), pos, out=(bq, bk))
        assert torch.equal(bq, yq) and torch.equal(bk, yk) and torch.equal(buf[:, :, hq + hk:], qkv[:, :, hq + hk:])
        # each alone; heads ahead of tokens in memory; one's gradient into a projection's gradient
        assert torch.equal(rope.forward(q, pos), yq)
        heads_first = q.transpose(1, 2).contiguous().transpose(1, 2)
        into = torch.zeros(b, hq, t, head_dim, device="cuda", dtype=DT[dtype]).transpose(1, 2)
        assert torch.equal(rope.forward(heads_first, pos, out=into), yq)
        grad = torch.zeros_like(qkv)
        rope.backward((yq, yk), pos, out=(grad[:, :, :hq], grad[:, :, hq:hq + hk]))
        one = rope.backward(yq, pos)
        assert torch.equal(grad[:, :, :hq], one) and float(grad[:, :, hq + hk:].abs().max()) == 0


def test_the_gradient_undoes_and_matches_differences():
    rope = fsp.Rotary(32, base=100.0, layout="half", scaling="linear", factor=2.0)
    x, dy, d = torch.randn(3, 20, 4, 40, device="cuda")
    pos = torch.arange(20, device="cuda") * 31
    dx = rope.backward(dy, pos)
    # linear in x: <dy, y(x + d) - y(x)> = <dx, d>; 3200 products of size 1, each within some 2^-20
    diff = (rope.forward(x + d, pos).double() - rope.forward(x, pos).double())
    assert abs(float((diff * dy).sum() - (dx.double() * d).sum())) <= 3200 * 2.0 ** -20 * 3
    y = rope.backward(rope.forward(x, pos), pos)
    # the angle's error (2^-24 pi) moves both the same way; two rotations' other roundings
    assert float((y - x).abs().max()) <= 2 * R.ROTARY_TOL * 2 * float(x.abs().max()) * 2


@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, torch.int16), (torch.float32, torch.int32)])
@pytest.mark.parametrize("head_dim,dim", [(64, 32), (36, 10), (66, 34)])
def test_what_is_not_rotated_keeps_its_bits(dtype, bits, head_dim, dim):
    raw = torch.arange(50 * 3 * head_dim, device="cuda") * 40503
    x = raw.to(bits).view(dtype).view(50, 3, head_dim)   # NaNs of all kinds among them
    for layout in ("half", "interleaved"):
        y = fsp.Rotary(dim, layout=layout).forward(x, torch.arange(50, device="cuda"))
        assert torch.equal(y.view(bits)[..., dim:], x.view(bits)[..., dim:])


def test_inputs_that_repeat():
    """Broadcast heads, tokens and batches are read as they stand."""
    rope, pos = fsp.Rotary(32), torch.arange(6, device="cuda") * 11
    for shape in ((1, 1, 3, 40), (2, 1, 1, 40), (1, 6, 1, 40)):
        x = torch.randn(shape, device="cuda").expand(2, 6, 3, 40)
        assert torch.equal(rope.forward(x, pos), rope.forward(x.contiguous(), pos))
    buf = torch.randn(2 * 6 * 3 * 40, device="cuda")
    with pytest.raises(fsp.FspError, match="overlaps"):
        rope.forward(buf[:40].view(1, 1, 1, 40).expand(2, 6, 3, 40), pos, out=buf.view(2, 6, 3, 40))


def test_empties_streams_and_graphs():
    rope = fsp.Rotary(16)
    x, pos = torch.randn(6, 3, 16, device="cuda"), torch.arange(6, device="cuda")
    want = rope.forward(x, pos)
    assert rope.forward(x[:0], pos[:0]).shape == (0, 3, 16) and rope.forward(x[:, :0], pos).shape == (6, 0, 16)
    q, k = rope.forward((x, x[:, :0]), pos)
    assert torch.equal(q, want) and k.shape == (6, 0, 16)
    k, q = rope.forward((x[:, :0], x), pos)
    assert torch.equal(q, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = rope.forward(x, pos, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.forward(x, pos, out=out)
        pos.add_(1)
    pos.copy_(torch.arange(6, device="cuda"))
    for k in range(3):   # a decoding loop: the positions advance on the device
        graph.replay()
        assert torch.equal(out, rope.forward(x, torch.arange(6, device="cuda") + k))
    assert fsp.device_error() == 0


def test_offsets_past_32_bits():
    big = torch.zeros(2 ** 18 + 2, 1, 2 ** 14, dtype=torch.bfloat16, device="cuda")
    x = big[:, :, 64:128]
    x[-1] = torch.randn(64, device="cuda")
    pos = torch.full((2 ** 18 + 2,), 7, device="cuda")
    rope = fsp.Rotary(64)
    want = rope.forward(x[-1:].clone(), pos[:1])
    assert torch.equal(rope.forward(x, pos, out=big[:, :, :64])[-1:], want)
    assert float(big[:-1].abs().max()) == 0 and float(big[:, :, 128:].abs().max()) == 0


def test_refusals():
    rope = fsp.Rotary(16)
    x, pos = torch.zeros(4, 2, 16, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (lambda: rope.forward(x.half(), pos), lambda: rope.forward(x, pos.float()), lambda: rope.forward((x, x.bfloat16()), pos)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: rope.forward(x.cpu(), pos), lambda: rope.forward(x, pos.cpu()), lambda: rope.forward(x[0], pos), lambda: rope.forward(x, pos[:3]),
                lambda: rope.forward(x, torch.zeros(8, dtype=torch.int64, device="cuda")[::2]), lambda: rope.forward((x, x[:3]), pos),
                lambda: rope.forward((x, x, x), pos), lambda: rope.forward((x, x), pos, out=(x,)), lambda: rope.forward(x, pos, out=x[:3]),
                lambda: rope.forward(x.transpose(1, 2), pos), lambda: rope.forward((), pos)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fsp.FspError, match="smaller than rotary_dim"):
        rope.forward(x[..., :8].contiguous(), pos)
    with pytest.raises(fsp.FspError, match="overlaps"):
        rope.forward((x, torch.zeros_like(x)), pos, out=(torch.zeros_like(x), x))
    with pytest.raises(fsp.FspError, match="share a place"):
        rope.forward(x, pos, out=torch.zeros(1, 2, 16, device="cuda").expand(4, 2, 16))
