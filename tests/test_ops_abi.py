"""The operators' C entry points on the host: what they refuse before any launch,
and the sizes and layouts they state."""
import ctypes

import numpy as np
import pytest

from fsdp_sharded_mixed_pass_gb300 import fsp as B

from ops_reference import BLOCK, code_values, codes, e4m3, fp8, rounds_to

FAKE = 1 << 44   # 16-byte aligned, never dereferenced on the host
HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from fsdp_sharded_mixed_pass_gb300 import build
        build.build()
    return B.lib()


def _arr(ty, *xs):
    return (ty * max(1, len(xs)))(*xs)


def _create(lib, numels, params, pd, grads, gd, copies=None, n=None):
    out = ctypes.c_void_p(123)
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    st = lib.fsp_adamw_list_create(len(numels) if n is None else n, _arr(ctypes.c_int64, *numels), _arr(vp, *params),
                                   _arr(i32, *pd), _arr(vp, *grads), _arr(i32, *gd),
                                   None if copies is None else _arr(vp, *copies), ctypes.byref(out))
    return st, out


def test_adamw_list_refusals(lib):
    bad = [
        ([-1], [FAKE], [0], [2 * FAKE], [0]),                  # negative size
        ([4], [FAKE], [2], [2 * FAKE], [0]),                   # unknown dtypes
        ([4], [FAKE], [0], [2 * FAKE], [7]),
        ([4], [None], [0], [FAKE], [0]),                       # NULL
        ([4], [FAKE], [0], [None], [0]),
        ([4], [FAKE + 2], [0], [2 * FAKE], [0]),               # below the elements' alignment
        ([4], [FAKE + 1], [1], [2 * FAKE], [0]),
        ([4], [FAKE], [0], [FAKE + 12], [0]),                  # overlap
        ([4, 4], [FAKE, FAKE + 8], [0, 0], [2 * FAKE, 3 * FAKE], [0, 0]),
    ]
    for case in bad:
        st, out = _create(lib, *case)
        assert st == B.FSP_EINVAL and not out.value and lib.fsp_last_error()
    assert _create(lib, [], [], [], [], [], n=-1)[0] == B.FSP_EINVAL
    assert _create(lib, [4], [FAKE], [0], [2 * FAKE], [0], copies=[FAKE + 8])[0] == B.FSP_EINVAL
    assert lib.fsp_adamw_list_create(0, None, None, None, None, None, None, None) == B.FSP_EINVAL
    assert lib.fsp_adamw_list_create(1, None, None, None, None, None, None, ctypes.byref(ctypes.c_void_p())) == B.FSP_EINVAL


def test_adamw_list_of_nothing(lib):
    st, h = _create(lib, [0, 0], [None, None], [0, 1], [None, None], [0, 0])
    assert st == B.FSP_OK
    n, off = ctypes.c_int64(-1), (ctypes.c_int64 * 2)(-1, -1)
    assert lib.fsp_adamw_list_info(h, ctypes.byref(n), off) == B.FSP_OK and n.value == 0 and list(off) == [0, 0]
    step = lambda hp=HP, t=1, sd=0, ms=None: lib.fsp_adamw_list_step(h, sd, None, None, ms, None, ctypes.byref(B._hp(hp)), t, None, 0, None, None)  # noqa: E731
    assert step() == B.FSP_OK and step(sd=1) == B.FSP_OK
    assert step(t=0) == B.FSP_EINVAL and step(sd=2) == B.FSP_EINVAL and step(ms=FAKE) == B.FSP_EINVAL
    for k, x in (("lr", -1.0), ("beta1", 1.0), ("beta2", float("nan")), ("eps", float("inf"))):
        assert step(dict(HP, **{k: x})) == B.FSP_EINVAL
    assert lib.fsp_adamw_list_step(None, 0, None, None, None, None, ctypes.byref(B._hp(HP)), 1, None, 0, None, None) == B.FSP_EINVAL
    assert lib.fsp_adamw_list_info(None, ctypes.byref(n), None) == B.FSP_EINVAL
    assert lib.fsp_adamw_list_info(h, None, None) == B.FSP_EINVAL
    assert lib.fsp_adamw_list_state_values(h, *[None] * 7) == B.FSP_OK
    lib.fsp_adamw_list_destroy(h)
    lib.fsp_adamw_list_destroy(None)


def _embedding(lib, weight=None, wd=0, vocab=10, dim=8, ws=8, tokens=FAKE, size=8, n=0, out=None, od=0, os_=8):
    return lib.fsp_embedding(weight, wd, vocab, dim, ws, tokens, size, n, 1.0, out, od, os_, None)


def test_embedding_refusals(lib):
    assert _embedding(lib, vocab=0) == B.FSP_OK   # nothing to do
    for kw in (dict(size=2), dict(n=-1), dict(n=1 << 60), dict(vocab=-1), dict(dim=-1), dict(wd=3, vocab=0), dict(od=9),
               dict(ws=7), dict(os_=7), dict(n=4, tokens=None), dict(n=4, tokens=FAKE + 4), dict(weight=None), dict(weight=FAKE + 2),
               dict(ws=1 << 56)):
        assert _embedding(lib, **kw) == B.FSP_EINVAL, kw


def _backward(lib, n=0, vocab=10, dim=8, size=8, gd=0, wd=0, gs=8, ws=8, weight=None, work=None, work_bytes=0, accumulate=0):
    return lib.fsp_embedding_backward(None, size, n, None, gd, dim, gs, weight, wd, vocab, ws, 1.0, -1, accumulate, work,
                                      work_bytes, None)


def test_embedding_backward_refusals(lib):
    assert _backward(lib, vocab=0) == B.FSP_OK
    for kw in (dict(n=-1), dict(vocab=-1), dict(size=3), dict(gd=2), dict(wd=2), dict(gs=7), dict(ws=7), dict(n=4), dict()):
        assert _backward(lib, **kw) == B.FSP_EINVAL, kw
    for kw in (dict(n=(1 << 31)), dict(vocab=1 << 31), dict(dim=1 << 25)):
        assert _backward(lib, **kw) == B.FSP_EUNSUPPORTED, kw
    size = ctypes.c_size_t()
    assert lib.fsp_embedding_backward_workspace_bytes(10, 8, 100, None) == B.FSP_EINVAL
    assert lib.fsp_embedding_backward_workspace_bytes(10, -8, 100, ctypes.byref(size)) == B.FSP_EINVAL
    last = 0
    for n in (0, 1, 100, 10 ** 6):
        assert lib.fsp_embedding_backward_workspace_bytes(151936, 1024, n, ctypes.byref(size)) == B.FSP_OK
        assert size.value >= max(last, 16 * n)
        last = size.value


def test_fp8_sizes_and_refusals(lib):
    size, off = ctypes.c_size_t(), ctypes.c_size_t()
    for rows, cols in ((0, 0), (1, 1), (128, 128), (129, 513), (151936, 1024)):
        assert lib.fsp_fp8_bytes(rows, cols, ctypes.byref(size), ctypes.byref(off)) == B.FSP_OK
        tiles, blocks, pieces = -(-rows // 128), -(-cols // 128), -(-cols // 512)
        assert off.value == tiles * blocks * 16384 and size.value == off.value + tiles * pieces * 512
    assert lib.fsp_fp8_bytes(-1, 1, ctypes.byref(size), ctypes.byref(off)) == B.FSP_EINVAL
    assert lib.fsp_fp8_bytes(1, 1, None, ctypes.byref(off)) == B.FSP_EINVAL
    q = lib.fsp_fp8_quantize
    assert q(None, 0, 0, 8, 8, None, None, None) == B.FSP_OK
    for args in ((None, 0, 4, 8, 8, FAKE, None), (FAKE, 0, 4, 8, 7, FAKE, None), (FAKE, 2, 4, 8, 8, FAKE, None),
                 (FAKE, 0, 4, 8, 8, None, None), (FAKE + 2, 0, 4, 8, 8, FAKE, None), (FAKE, 0, 4, -8, 8, FAKE, None)):
        assert q(*args, None) == B.FSP_EINVAL, args
    mm = lib.fsp_fp8_matmul
    assert mm(None, None, 0, 8, 8, None, 0, 8, 0, None) == B.FSP_OK
    for args in ((FAKE, FAKE, 4, 8, 8, None, 0, 8, 0), (FAKE, FAKE, 4, 8, 8, FAKE, 0, 7, 0), (FAKE, FAKE, 4, 8, 8, FAKE, 5, 8, 0),
                 (FAKE, FAKE, 4, 8, -1, FAKE, 0, 8, 0), (FAKE, FAKE, 4, 8, 8, FAKE + 2, 0, 8, 0)):
        assert mm(*args, None) == B.FSP_EINVAL, args
    assert mm(FAKE, FAKE, 4, 8, 8, FAKE, 1, 8, 1, None) == B.FSP_EUNSUPPORTED
    assert lib.fsp_fp8_values(None, 4, 4, None, None) == B.FSP_EINVAL and lib.fsp_fp8_values(None, 0, 4, None, None) == B.FSP_OK


def test_fp8_linear_refusals(lib):
    size = ctypes.c_size_t()
    bytes_of = lambda r, i, o, b: (lib.fsp_fp8_linear_workspace_bytes(r, i, o, b, ctypes.byref(size)), size.value)  # noqa: E731
    assert bytes_of(1, 1024, 2048, 0) == (B.FSP_OK, 0) and bytes_of(0, 5, 5, 1) == (B.FSP_OK, 0)
    assert bytes_of(5, 1024, 2048, 0)[1] >= 5 * 1024 and bytes_of(300, 500, 700, 1)[1] >= 300 * (2 * 700 + 500)
    assert bytes_of(-1, 5, 5, 0)[0] == B.FSP_EINVAL and lib.fsp_fp8_linear_workspace_bytes(1, 1, 1, 0, None) == B.FSP_EINVAL
    f = lib.fsp_fp8_linear
    assert f(None, 0, 0, 8, 8, None, 8, None, 0, 8, None, 0, None) == B.FSP_OK
    for args in ((None, 0, 4, 8, 8, FAKE, 8, FAKE, 0, 8), (FAKE, 3, 4, 8, 8, FAKE, 8, FAKE, 0, 8),
                 (FAKE, 0, 4, 8, 7, FAKE, 8, FAKE, 0, 8), (FAKE, 0, 4, 8, 8, FAKE, 8, FAKE, 0, 7),
                 (FAKE, 0, -4, 8, 8, FAKE, 8, FAKE, 0, 8), (FAKE + 2, 0, 4, 8, 8, FAKE, 8, FAKE, 0, 8)):
        assert f(*args, None, 0, None) == B.FSP_EINVAL, args
    g = lib.fsp_fp8_linear_backward
    assert g(None, 0, 8, None, 0, 8, 0, 8, 8, None, None, 0, 8, None, 8, 0, None, 0, None) == B.FSP_OK
    assert g(FAKE, 0, 8, None, 0, 8, 4, 8, 8, FAKE, FAKE, 0, 8, None, 8, 0, None, 0, None) == B.FSP_EINVAL
    assert g(FAKE, 0, 8, FAKE, 0, 7, 4, 8, 8, FAKE, FAKE, 0, 8, None, 8, 0, None, 0, None) == B.FSP_EINVAL


# ---- the references themselves ---------------------------------------------------------

def test_reference_e4m3_against_torch():
    import torch
    x = np.concatenate([np.linspace(-448, 448, 20001), np.exp2(np.linspace(-12, 8, 5000))]).astype(np.float32)
    assert np.array_equal(e4m3(x.astype(np.float64)), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_reference_fp8_scale_is_the_smallest_that_fits():
    x = np.zeros((3, 200))
    x[0, 5], x[1, 150], x[2, 7] = 448.0, -449.0, 1e-3
    v = fp8(x)
    assert v[0, 5] == 448 and v[1, 150] == -448 and abs(v[2, 7] - 1e-3) <= 1e-3 * 2.0 ** -4 and (fp8(v) == v).all()


def test_reference_codes_worked_block():
    x = np.zeros(BLOCK, np.float32)
    x[:4] = 1.0, -0.25, 1e-9, 0.5
    q, s = codes(x, 127, False)
    assert s[0] == 1 and list(q[:5]) == [127, -64, 0, 90, 0]   # 63.5 rounds to even; 127 sqrt(1/2) = 89.8
    r, t = codes(np.abs(x), 255, True)
    assert list(r[:5]) == [255, 180, 1, 214, 0]                # 255 (1/4)^(1/4) = 180.3; 1e-9: 1.43; 255 (1/2)^(1/4) = 214.4
    assert abs(code_values(q, s, 127, False)[3] - 0.5) < 0.5 * 2 / 90 and abs(code_values(r, t, 255, True)[1] - 0.25) < 0.25 * 4 / 180


def test_reference_rounding_of_bf16():
    want = np.array([1.0, 1.0 + 2.0 ** -8, 7.50974])
    assert rounds_to(np.array([1.0, 1.0, 7.5]), want, np.zeros(3)).all()
    assert not rounds_to(np.array([1.0 + 2.0 ** -7, 1.0 + 2.0 ** -7, 7.53125]), want, np.zeros(3)).any()


def test_embedding_backward_takes_no_more_tokens_than_its_sort_can_count(lib):
    """The sort counts tokens in 32 bits and steps by up to 16384 past the last one."""
    size = ctypes.c_size_t()
    bytes_of = lambda n: lib.fsp_embedding_backward_workspace_bytes(10, 1, n, ctypes.byref(size))  # noqa: E731
    most = 2 ** 31 - 1 - 16384
    assert bytes_of(most) == B.FSP_OK and size.value >= 16 * most
    for n in (most + 1, 2 ** 31 - 4098, 2 ** 31 - 1, 2 ** 31):
        assert bytes_of(n) == B.FSP_EUNSUPPORTED, n
        assert _backward(lib, n=n) == B.FSP_EUNSUPPORTED, n


# ---- tensors of another device -------------------------------------------------------------

def _refused_elsewhere():
    """Every tensor argument of the binding's calls, each in turn on another device than
    the current one.  Host tensors stand in for device 0's (`here`) and device 1's."""
    import torch
    import fsdp_sharded_mixed_pass_gb300 as fsp

    class Here(torch.Tensor):
        def get_device(self):
            return 0

    class There(torch.Tensor):
        def get_device(self):
            return 1

    def make(there, name, *shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(There if name == there else Here)

    def matrix(there, name, rows, cols):
        q = fsp.Fp8Matrix(rows, cols, device="cpu")
        q.data = make(there, name, q.data.numel(), dtype=torch.uint8)
        return q

    def layer(there):
        m = fsp.Fp8Linear.__new__(fsp.Fp8Linear)
        m.out_features, m.in_features, m.train = 6, 4, True
        m.codes, m.codes_t = matrix(there, "weight", 6, 4), matrix(there, "weight", 4, 6)
        return m
    i64 = torch.int64
    calls = {
        "embedding": (("weight", "tokens", "out"), lambda t: fsp.embedding(
            make(t, "weight", 5, 4), make(t, "tokens", 3, dtype=i64), out=make(t, "out", 3, 4))),
        "embedding_backward": (("tokens", "grad_out", "grad_weight", "workspace"), lambda t: fsp.embedding_backward(
            make(t, "tokens", 3, dtype=i64), make(t, "grad_out", 3, 4), make(t, "grad_weight", 5, 4),
            workspace=make(t, "workspace", 100000, dtype=torch.uint8))),
        "TensorAdamW": (("param", "grad", "copy"), lambda t: fsp.TensorAdamW(
            [make(t, "param", 8)], [make(t, "grad", 8)], [make(t, "copy", 8, dtype=torch.bfloat16)])),
        "quantize_fp8": (("x", "rows", "transposed"), lambda t: fsp.quantize_fp8(
            make(t, "x", 6, 4), matrix(t, "rows", 6, 4), matrix(t, "transposed", 4, 6))),
        "matmul_fp8": (("a", "b", "out"), lambda t: fsp.matmul_fp8(
            matrix(t, "a", 6, 4), matrix(t, "b", 5, 4), out=make(t, "out", 6, 5))),
        "values": (("matrix",), lambda t: matrix(t, "matrix", 6, 4).values()),
        "forward": (("x", "weight", "out"), lambda t: layer(t).forward(make(t, "x", 3, 4), out=make(t, "out", 3, 6))),
        "backward": (("x", "grad_out", "weight", "grad_weight", "out"), lambda t: layer(t).backward(
            make(t, "x", 3, 4), make(t, "grad_out", 3, 6), make(t, "grad_weight", 6, 4), out=make(t, "out", 3, 4))),
    }
    return [(name, arg, call) for name, (args, call) in calls.items() for arg in args]


def test_tensors_of_another_device_are_refused(lib, monkeypatch):
    from fsdp_sharded_mixed_pass_gb300 import ops
    ops._ready()
    monkeypatch.setattr(ops, "_device", lambda: 0)

    def launched(*args):
        raise AssertionError("the library was called")
    quiet = type("Lib", (), {n: staticmethod(launched) for n in ops.EXPORTS})
    for n in ("fsp_fp8_bytes", "fsp_fp8_linear_workspace_bytes", "fsp_embedding_backward_workspace_bytes"):
        setattr(quiet, n, staticmethod(getattr(lib, n)))
    monkeypatch.setattr(ops, "_lib", quiet)
    monkeypatch.setattr(ops._fsp, "lib", lambda: quiet)
    monkeypatch.setattr(ops, "_handle", lambda *a: 0)
    for name, arg, call in _refused_elsewhere():
        with pytest.raises(ValueError, match="cuda:1"):
            call(arg)
        with pytest.raises(AssertionError, match="was called"):   # all of them here: nothing is refused
            call(None)
