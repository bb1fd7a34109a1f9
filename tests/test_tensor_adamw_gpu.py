"""AdamW over a list of tensors, with fp32 and with 8-bit states."""
import numpy as np
import pytest
import torch

import fsdp_sharded_mixed_pass_gb300 as fsp
from oracle import step as OS

from gpu_cases import HP, Guarded, SCALED_BOUND, ensure_built, master_extra_scale, state_errors
from ops_reference import BLOCK, code_values, codes, moments_rounded, rounds_to

pytestmark = pytest.mark.gpu
OPT = dict(lr=HP["lr"], betas=(HP["beta1"], HP["beta2"]), eps=HP["eps"], weight_decay=HP["weight_decay"])
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ensure_built()


def _values(x):
    return x.detach().float().cpu().numpy()


class Lists:
    """Tensors of `sizes` inside guarded buffers, `shift` elements off alignment."""

    def __init__(self, sizes, param="f32", grad="f32", copies=False, shift=0, seed=0, bits=32, grad_std=1e-3, **kw):
        gen = np.random.default_rng(seed)
        pick = lambda d, i: d if isinstance(d, str) else d[i % len(d)]  # noqa: E731
        self.sizes, self.guards = sizes, []

        def make(n, dtype, values):
            g = Guarded(n + shift, DT[dtype], 0)
            self.guards.append(g)
            t = g.t[shift:]
            if values is not None:
                t.copy_(torch.from_numpy(values.astype(np.float32)))
            return t
        self.params = [make(n, pick(param, i), gen.normal(0, 0.02, n)) for i, n in enumerate(sizes)]
        self.grads = [make(n, pick(grad, i), gen.normal(0, grad_std, n)) for i, n in enumerate(sizes)]
        self.copies = [make(n, "bf16", None) if copies and i % 3 != 2 else None for i, n in enumerate(sizes)]
        self.opt = fsp.TensorAdamW(self.params, self.grads, self.copies if copies else None, state_bits=bits, **OPT, **kw)
        n = self.opt.state_len
        self.m, self.v = np.zeros(n, np.float32), np.zeros(n, np.float32)
        self.inside = np.zeros(n, bool)
        for o, k in zip(self.opt.offsets, sizes):
            self.m[o:o + k] = gen.normal(0, 1e-4, k)
            self.v[o:o + k] = gen.uniform(0, 1e-6, k) ** 2 * 1e6
            self.inside[o:o + k] = True
        self.opt.load_state(torch.from_numpy(self.m).cuda(), torch.from_numpy(self.v).cuda())

    def flat(self, tensors):
        out = np.zeros(self.opt.state_len, np.float32)
        for o, k, t in zip(self.opt.offsets, self.sizes, tensors):
            if t is not None:
                out[o:o + k] = _values(t)
        return out

    def intact(self):
        return all(g.guards_intact() for g in self.guards)


SIZES = [1, 255, 256, 257, 0, 2047, 2048, 2049, 5000, 3, 70001]


# enough tiles (2048 elements) for the ring of stages, most of them whole; the last
# tensors end off a multiple of 16, of 256 and of 2048, or are tiny
LONG = [4_000_000, 2_000_016, 1_234_567, 1, 700, 2048 * 9 + 256, 0, 17]
LONG32 = [17_000_016] + LONG   # (fp32 states take it from more tiles on)


def _bf16(x):
    return OS.bf16_bits_to_f32(OS.bf16_rne(x))


MIXED = (("f32", "bf16"), ("bf16", "f32", "f32"), True)


@pytest.mark.parametrize("param,grad,copies,sizes,shift",
                         [(*kinds, SIZES, shift) for shift in (0, 1, 2, 4)
                          for kinds in (("f32", "f32", False), ("f32", "bf16", True), ("bf16", "bf16", False), MIXED)]
                         + [("f32", "bf16", True, LONG32, 0), (*MIXED, LONG32, 0), (*MIXED, LONG32, 4)])
def test_fp32_states_match_the_oracle(param, grad, copies, sizes, shift):
    c = Lists(sizes, param, grad, copies, shift, seed=shift)
    c.opt.t = 9
    p, g = c.flat(c.params), c.flat(c.grads)
    c.opt.step()
    want = OS.adamw(p, c.m, c.v, g, HP, 10)
    got = [c.flat(c.params), _values(c.opt.exp_avg), _values(c.opt.exp_avg_sq)]
    ins = c.inside
    is_bf16 = c.flat([torch.full((n,), float(t.dtype == torch.bfloat16)) for n, t in zip(c.sizes, c.params)]) > 0
    errs = state_errors([x[ins] for x in got], [x[ins] for x in want], [x[ins] for x in (p, c.m, c.v)])
    assert (errs[1] <= SCALED_BOUND * 2 ** 24).all() and (errs[2] <= SCALED_BOUND * 2 ** 24).all()
    assert (errs[0][~is_bf16[ins]] <= SCALED_BOUND * 2 ** 24).all()
    # a bf16 parameter: the update in fp32 (within the bound above), rounded once
    tol = SCALED_BOUND * (np.abs(p) + np.abs(want[0]) + master_extra_scale(p, want[0], c.m, want[1]))
    assert rounds_to(got[0], want[0].astype(np.float64), tol)[is_bf16].all()
    for cp, q in zip(c.copies, c.params):
        if cp is not None and q.dtype == torch.float32:
            assert np.array_equal(_values(cp), _bf16(_values(q)))
    assert (got[1][~ins] == 0).all() and (got[2][~ins] == 0).all()
    assert c.intact() and c.opt.t == 10 and fsp.device_error() == 0


@pytest.mark.parametrize("sizes", [[4096, 513, 70000], [21_000_000, 513, 70000]])
def test_fp32_states_equal_the_sharded_step_bit_for_bit(sizes):
    c = Lists(sizes, copies=False, seed=5)
    plan = fsp.plan_layout([(n,) for n in sizes], 1, "fsdp2")
    seg = {s.param: s for s in plan.segments}
    gbuf = torch.zeros(plan.full_len_padded, device="cuda")
    pbuf = torch.zeros(plan.full_len_padded, device="cuda", dtype=torch.bfloat16)
    state = [torch.zeros(plan.state_len_total, device="cuda") for _ in range(3)]
    cut = lambda x, i: x[c.opt.offsets[i]:c.opt.offsets[i] + sizes[i]]  # noqa: E731
    for i, n in enumerate(sizes):
        gbuf[seg[i].full_off:seg[i].full_off + n] = c.grads[i]
        for buf, src in zip(state, (c.params[i], cut(c.opt.exp_avg, i), cut(c.opt.exp_avg_sq, i))):
            buf[seg[i].state_off:seg[i].state_off + n] = src
    for t in (1, 2, 3):
        fsp.sharded_step(plan, [gbuf], *state, [pbuf], HP, t)
        c.opt.step()
    for i, n in enumerate(sizes):
        for buf, mine in zip(state, (c.params[i], cut(c.opt.exp_avg, i), cut(c.opt.exp_avg_sq, i))):
            assert torch.equal(buf[seg[i].state_off:seg[i].state_off + n], mine)


@pytest.mark.parametrize("sizes,shift", [(SIZES, 0), (SIZES, 1), (SIZES, 4), (LONG, 0), (LONG, 4)])
@pytest.mark.parametrize("param,grad,copies,scale", [("f32", "f32", False, None), ("f32", "bf16", True, 0.37),
                                                     ("bf16", "bf16", False, None)])
def test_8_bit_states(param, grad, copies, scale, sizes, shift):
    c = Lists(sizes, param, grad, copies, shift, seed=10 + shift, bits=8)
    opt = c.opt
    q0, s0 = codes(c.m, 127, False)
    r0, t0 = codes(c.v, 255, True)
    assert np.array_equal(opt.exp_avg.cpu().numpy(), q0) and np.array_equal(opt.exp_avg_sq.cpu().numpy(), r0)
    assert np.array_equal(_values(opt.exp_avg_scale), s0) and np.array_equal(_values(opt.exp_avg_sq_scale), t0)
    m, v = code_values(q0, s0, 127, False), code_values(r0, t0, 255, True)
    got = opt.state_values()
    assert np.array_equal(_values(got[0]), m) and np.array_equal(_values(got[1]), v)
    opt.t = 9
    p, g = c.flat(c.params), c.flat(c.grads)
    coef = None
    if scale is not None:
        coef = torch.full((1,), scale, device="cuda")
        g = g * np.float32(scale)
    opt.step(grad_scale=coef)
    # codes and scales: exactly those of separately rounded fp32 operations
    m1, v1 = moments_rounded(m, v, g, HP)
    q1, s1 = codes(m1, 127, False)
    r1, t1 = codes(v1, 255, True)
    assert np.array_equal(opt.exp_avg.cpu().numpy(), q1) and np.array_equal(opt.exp_avg_sq.cpu().numpy(), r1)
    assert np.array_equal(_values(opt.exp_avg_scale), s1) and np.array_equal(_values(opt.exp_avg_sq_scale), t1)
    # and within half a code (and 2^-14, for fp32) of the definition in 64 bits
    want = OS.adamw(p, m, v, g, HP, 10)
    for x, q, s, top, root in ((want[1], q1, s1, 127, 2), (want[2], r1, t1, 255, 4)):
        big = np.repeat(s.astype(np.float64), BLOCK)
        near = np.where(big > 0, top * (np.abs(x) / np.where(big > 0, big, 1)) ** (1 / root), 0)
        off = np.abs(np.abs(q) - near)
        assert (off[np.abs(q) != 1] <= 0.5 + 2.0 ** -14).all() and (off <= 1).all()
    # the parameters: from m' and v' before they are rounded to codes
    now = c.flat(c.params)
    ins = c.inside
    if param == "f32":
        e = state_errors([now[ins], m1[ins], v1[ins]], [x[ins] for x in want], [x[ins] for x in (p, m, v)])
        assert (e[0] <= SCALED_BOUND * 2 ** 24).all()
        for cp, q in zip(c.copies, c.params):
            if cp is not None:
                assert np.array_equal(_values(cp), _bf16(_values(q)))
    else:
        tol = SCALED_BOUND * (np.abs(p) + np.abs(want[0]) + master_extra_scale(p, want[0], m, want[1]))
        assert rounds_to(now, want[0].astype(np.float64), tol)[ins].all()
    assert c.intact() and fsp.device_error() == 0


def test_8_bit_zero_and_tiny_blocks():
    c = Lists([1024], bits=8)
    c.opt.load_state(torch.zeros(1024, device="cuda"), torch.zeros(1024, device="cuda"))
    g = np.zeros(1024, np.float32)
    g[256:512] = 1e-18                     # v' = 1e-36 (1 - b2): normal; squares below 2^-126 vanish in fp32 too
    g[512], g[513] = 1.0, 1e-12            # a v' of 5e-26 beside one of 0.05: keeps the smallest code
    c.grads[0].copy_(torch.from_numpy(g))
    p = _values(c.params[0])
    c.opt.step()
    m, v = (_values(x) for x in c.opt.state_values())
    assert (m[:256] == 0).all() and (v[:256] == 0).all()
    assert (m[256:512] > 0).all() and (v[256:512] > 0).all()
    assert int(c.opt.exp_avg_sq[513]) == 1 and v[513] > 0 and (v[514:768] == 0).all()
    want = OS.adamw(p, np.zeros(1024), np.zeros(1024), g, HP, 1)[0]
    assert np.allclose(_values(c.params[0]), want, rtol=2.0 ** -20, atol=2.0 ** -24 * 0.1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_gradients_stay_in_their_element_or_block(bad):
    for bits in (32, 8):
        c = Lists([1000], bits=bits, seed=3)
        c.grads[0][300] = bad
        c.opt.step()
        m, v = (_values(x) for x in c.opt.state_values())
        p = _values(c.params[0])
        assert not np.isfinite(p[300]) and np.isfinite(np.delete(p, 300)).all()
        hit = slice(300, 301) if bits == 32 else slice(256, 512)
        assert not np.isfinite(m[300]) and not np.isfinite(v[300])
        rest = np.ones(1024, bool)
        rest[hit] = False
        assert np.isfinite(m[rest]).all() and np.isfinite(v[rest]).all()


@pytest.mark.parametrize("sizes", [[5000, 33], [21_000_000, 33]])
@pytest.mark.parametrize("bits", [32, 8])
def test_capturable_steps_replayed_from_a_graph_equal_host_steps(bits, sizes):
    a, b = (Lists(sizes, bits=bits, seed=8, capturable=cap) for cap in (False, True))
    b.opt.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.opt.step()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
    for _ in range(4):
        a.opt.step()
    torch.cuda.synchronize()
    assert a.opt.t == b.opt.t == 4
    for x, y in zip(a.params, b.params):
        assert torch.equal(x, y)
    assert torch.equal(a.opt.exp_avg, b.opt.exp_avg) and torch.equal(a.opt.exp_avg_sq, b.opt.exp_avg_sq)


def test_device_t_below_one_is_reported():
    c = Lists([10], capturable=True)
    c.opt._next_t.fill_(0)
    c.opt.step()
    assert fsp.device_error() == 8 and c.opt.t == 0


def test_step_on_another_stream_and_empty_lists():
    c = Lists([3000], bits=8, seed=4)
    d = Lists([3000], bits=8, seed=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.opt.step(stream=s)
    m = c.opt.state_values(stream=s)[0]
    s.synchronize()
    d.opt.step()
    assert torch.equal(c.params[0], d.params[0]) and torch.equal(m, d.opt.state_values()[0])
    for sizes in ([], [0, 0]):
        e = Lists(sizes, bits=8)
        e.opt.step()
        assert e.opt.t == 1 and e.opt.state_len == 0


def test_refusals():
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device="cuda")  # noqa: E731
    with pytest.raises(TypeError):
        fsp.TensorAdamW([f(4, torch.float16)], [f(4)])
    with pytest.raises(ValueError):
        fsp.TensorAdamW([f(4)], [f(5)])
    with pytest.raises(ValueError):
        fsp.TensorAdamW([f(8)[::2]], [f(4)])
    with pytest.raises(ValueError):
        fsp.TensorAdamW([f(4)], [f(4)], state_bits=16)
    with pytest.raises(ValueError):
        fsp.TensorAdamW([torch.zeros(4)], [f(4)])
    with pytest.raises(TypeError):
        fsp.TensorAdamW([f(4)], [f(4)], copies=[f(4)])
    x = f(64)
    with pytest.raises(fsp.FspError, match="overlaps"):
        fsp.TensorAdamW([x[:40]], [x[30:62].view(-1)[:32].new_zeros(40)], copies=[x.view(torch.bfloat16)[:40]])
    with pytest.raises(fsp.FspError, match="hyper-parameters"):
        fsp.TensorAdamW([f(4)], [f(4)], lr=-1.0).step()
    opt = fsp.TensorAdamW([f(4)], [f(4)])
    with pytest.raises(ValueError):
        opt.step(grad_scale=f(2))
    opt.exp_avg = opt.exp_avg_sq
    with pytest.raises(fsp.FspError, match="overlaps"):
        opt.step()
    assert opt.t == 0
    opt.exp_avg = opt._refs[1][0]   # a registered gradient in a state's place
    with pytest.raises(fsp.FspError):
        opt.step()


@pytest.mark.parametrize("bits", [32, 8])
def test_device_t_below_one_is_reported_on_long_lists(bits):
    n = 21_000_000   # enough tiles for the ring of stages
    a, b = (Lists([n], bits=bits, seed=6, capturable=cap) for cap in (True, False))
    a.opt._next_t.fill_(0)
    a.opt.step()
    assert fsp.device_error() == 8 and a.opt.t == 0
    b.opt.step()   # t = 1, which the step above was taken as
    assert fsp.device_error() == 0
    assert torch.equal(a.params[0], b.params[0]) and torch.equal(a.opt.exp_avg_sq, b.opt.exp_avg_sq)
