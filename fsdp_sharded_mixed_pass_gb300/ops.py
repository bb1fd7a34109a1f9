"""The operators of ``include/fsp_ops.h`` on torch tensors: AdamW over a list
of tensors, the embedding with its gradient, matrices in 8-bit floating point,
layer norm with its gradients, dropout and rotary positions.  Argument marshalling and output buffers only; everything is computed by
the library's kernels, asynchronously on ``stream`` (None: the current one) and the
current device, where every tensor of a call has to be.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct

from . import fsp as _fsp
from .optim import _on_stream

STATE_BLOCK = 256   # elements of a tensor that share a scale in 8-bit AdamW states

EXPORTS = ("fsp_adamw_list_create", "fsp_adamw_list_info", "fsp_adamw_list_destroy", "fsp_adamw_list_step",
           "fsp_adamw_list_state_values", "fsp_adamw_list_state_load", "fsp_embedding",
           "fsp_embedding_backward_workspace_bytes", "fsp_embedding_backward", "fsp_fp8_bytes", "fsp_fp8_quantize",
           "fsp_fp8_values", "fsp_fp8_matmul", "fsp_fp8_linear", "fsp_fp8_linear_backward",
           "fsp_fp8_linear_workspace_bytes", "fsp_layer_norm", "fsp_layer_norm_backward_workspace_bytes",
           "fsp_layer_norm_backward", "fsp_dropout", "fsp_rotary_phases", "fsp_rotary")


class _RotaryTensor(ctypes.Structure):   # ten words of 64 bits (Rotary passes them as such)
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("x_strides", ctypes.c_int64 * 3), ("out_strides", ctypes.c_int64 * 3)]


def bind(L) -> None:
    """Declares the argument types of ``EXPORTS`` on the loaded library."""
    vp, i32, i64, f32, P = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.POINTER
    size = ctypes.c_size_t
    for name, args in {
        "fsp_adamw_list_create": [i32, P(i64), P(vp), P(i32), P(vp), P(i32), P(vp), P(vp)],
        "fsp_adamw_list_info": [vp, P(i64), P(i64)],
        "fsp_adamw_list_destroy": [vp],
        "fsp_adamw_list_step": [vp, i32, vp, vp, vp, vp, P(_fsp._HParams), i64, vp, i32, vp, vp],
        "fsp_adamw_list_state_values": [vp] * 8,
        "fsp_adamw_list_state_load": [vp] * 8,
        "fsp_embedding": [vp, i32, i64, i64, i64, vp, i32, i64, f32, vp, i32, i64, vp],
        "fsp_embedding_backward_workspace_bytes": [i64, i64, i64, P(size)],
        "fsp_embedding_backward": [vp, i32, i64, vp, i32, i64, i64, vp, i32, i64, i64, f32, i64, i32, vp, size, vp],
        "fsp_fp8_bytes": [i64, i64, P(size), P(size)],
        "fsp_fp8_quantize": [vp, i32, i64, i64, i64, vp, vp, vp],
        "fsp_fp8_values": [vp, i64, i64, vp, vp],
        "fsp_fp8_matmul": [vp, vp, i64, i64, i64, vp, i32, i64, i32, vp],
        "fsp_fp8_linear": [vp, i32, i64, i64, i64, vp, i64, vp, i32, i64, vp, size, vp],
        "fsp_fp8_linear_backward": [vp, i32, i64, vp, i32, i64, i64, i64, i64, vp, vp, i32, i64, vp, i64, i32, vp, size,
                                    vp],
        "fsp_fp8_linear_workspace_bytes": [i64, i64, i64, i32, P(size)],
        "fsp_layer_norm": [vp, i32, i64, i64, i64, vp, vp, i32, f32, i32, vp, i32, i64, vp, vp],
        "fsp_layer_norm_backward_workspace_bytes": [i64, i64, P(size)],
        "fsp_layer_norm_backward": [vp, i32, i64, i64, i64, vp, i32, vp, i32, i64, vp, i32, vp, i64, vp, i64, vp, vp, i32,
                                    i32, vp, size, vp],
        "fsp_dropout": [vp, i32, i64, i64, i64, ctypes.c_double, ctypes.c_uint64, i64, vp, vp, i32, i64, vp, i32, i64, vp],
        "fsp_rotary_phases": [P(ctypes.c_double), i64, P(ctypes.c_uint64)],
        "fsp_rotary": [vp, i32, i32, i64, i64, vp, i32, i64, vp, i64, i32, f32, i32, vp],
    }.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = None if name == "fsp_adamw_list_destroy" else ctypes.c_int


# What every call needs, looked up once: a call on one token is a few microseconds
# of the GPU's time, so the host's share is kept as small.
_torch = _lib = _raw_stream = _device = None
_CODES, _INDEX = {}, {}   # dtype -> the library's code; index dtype -> bytes


def _ready():
    global _torch, _lib, _raw_stream, _device
    import torch
    _lib = _fsp.lib()
    _CODES.update({torch.float32: _fsp.DTYPES["f32"], torch.bfloat16: _fsp.DTYPES["bf16"]})
    _INDEX.update({torch.int64: 8, torch.int32: 4})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    return _lib


def _current() -> int:
    """The current device's index, on which a call's kernels run."""
    if _torch is None:
        _ready()
    return _device()


def _on(device: int, x, what: str) -> None:
    """Refuses a tensor that is not on ``device``: a kernel must not be given another
    device's memory."""
    at = x.get_device()
    if at != device:
        raise ValueError(f"{what} is not on a CUDA device" if at < 0 else
                         f"{what} is on cuda:{at}, the current device is cuda:{device}")


def _handle(stream, device: int):
    """The cudaStream_t of a stream argument (None: the current stream of ``device``,
    the current device)."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _fsp._stream_handle(stream)


def _dtype(x, what: str, device: int) -> int:
    """The library's code of the dtype (fp32 or bf16) of a tensor on ``device``."""
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {x.dtype}")
    if x.get_device() != device:
        _on(device, x, what)
    return code


def _rows(x, what: str):
    """A 2-D tensor's (rows, columns, row stride); its columns must be adjacent."""
    if x.dim() != 2:
        raise ValueError(f"{what} must have 2 dimensions")
    rows, cols = x.shape
    stride, step = x.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}: the elements of a row must be adjacent")
    return rows, cols, stride if rows > 1 and cols > 0 else max(1, cols)


def _flat(x, features: int, what: str):
    """(rows, row stride) of a tensor of any leading dimensions as rows x features."""
    if x.dim() == 2:
        rows, cols, stride = _rows(x, what)
        if cols != features:
            raise ValueError(f"{what}'s last dimension must be {features}")
        return rows, stride
    if x.dim() < 1 or x.shape[-1] != features:
        raise ValueError(f"{what}'s last dimension must be {features}")
    if not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous unless it has 2 dimensions")
    rows = 1
    for d in x.shape[:-1]:
        rows *= d
    return rows, max(1, features)


def _tokens(tokens, device: int) -> int:
    """Bytes per index of a token tensor on ``device``."""
    size = _INDEX.get(tokens.dtype)
    if size is None:
        raise TypeError(f"tokens: unsupported dtype {tokens.dtype}")
    if tokens.get_device() != device:
        _on(device, tokens, "tokens")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return size


def _workspace_bytes(workspace, device: int) -> int:
    """Bytes of a workspace tensor on ``device``; they must be its own, one after the other
    (an expanded tensor has more elements than memory)."""
    if workspace.get_device() != device:
        _on(device, workspace, "workspace")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _empty(shape, dtype, device, stream):
    """A buffer whose memory is handed out (and later taken back) in the order
    of the stream the call runs on."""
    if _torch is None:
        _ready()
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _on_stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


# ---- AdamW over a list of tensors ----------------------------------------------

class TensorAdamW:
    """AdamW over a list of tensors, one launch per step: ``params[i]`` (fp32 or
    bf16), ``grads[i]`` (fp32 or bf16) and, with ``copies``, ``copies[i]`` (bf16 or
    None: receives the new parameter rounded) are contiguous CUDA tensors
    registered once and read and written in place.

    ``state_bits=32`` keeps fp32 moments; ``state_bits=8`` keeps them in 8-bit
    codes with an fp32 scale per block of 256 elements (``exp_avg``: int8,
    ``exp_avg_sq``: uint8, ``exp_avg_scale``, ``exp_avg_sq_scale``), a quarter of
    the memory and traffic; ``state_values()`` reads such states as fp32 and
    ``load_state(m, v)`` writes them.  Tensor i's states are slots
    ``offsets[i]`` ... of the state buffers.

    ``step(grad_scale=None)`` applies update t + 1; ``grad_scale``, a device fp32
    tensor, multiplies every gradient (a clip coefficient).  ``capturable=True``
    keeps t on the device, as for ``ShardedAdamW``.
    """

    def __init__(self, params, grads, copies=None, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, state_bits: int = 32, capturable: bool = False):
        import torch
        self._h = None
        params, grads = list(params), list(grads)
        copies = [None] * len(params) if copies is None else list(copies)
        if not len(params) == len(grads) == len(copies):
            raise ValueError("params, grads and copies must be as many")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        n = len(params)
        here = _current()
        for i, (p, g, c) in enumerate(zip(params, grads, copies)):
            for x, what in ((p, "param"), (g, "grad"), (c, "copy")):
                if x is None and what == "copy":
                    continue
                if x.numel() != p.numel():
                    raise ValueError(f"{what} {i} has {x.numel()} elements, its parameter {p.numel()}")
                if not x.is_contiguous():
                    raise ValueError(f"{what} {i} must be contiguous")
            if c is not None:
                if c.dtype != torch.bfloat16:
                    raise TypeError(f"copy {i} must be bf16")
                _on(here, c, f"copy {i}")
        self._refs = (params, grads, copies)
        arr = lambda ty, xs: (ty * max(1, n))(*xs)  # noqa: E731
        ptrs = lambda xs: arr(ctypes.c_void_p, [None if x is None else x.data_ptr() for x in xs])  # noqa: E731
        out = ctypes.c_void_p()
        _fsp._check(_fsp.lib().fsp_adamw_list_create(
            n, arr(ctypes.c_int64, [p.numel() for p in params]), ptrs(params),
            arr(ctypes.c_int32, [_dtype(p, f"param {i}", here) for i, p in enumerate(params)]), ptrs(grads),
            arr(ctypes.c_int32, [_dtype(g, f"grad {i}", here) for i, g in enumerate(grads)]), ptrs(copies),
            ctypes.byref(out)), "fsp_adamw_list_create")
        self._h = out
        state_len, offsets = ctypes.c_int64(), (ctypes.c_int64 * max(1, n))()
        _fsp._check(_fsp.lib().fsp_adamw_list_info(out, ctypes.byref(state_len), offsets), "fsp_adamw_list_info")
        self.state_len, self.offsets = state_len.value, tuple(offsets[:n])
        device = params[0].device if n else "cuda"
        self.state_bits = state_bits
        zeros = lambda k, dt: torch.zeros(k, dtype=dt, device=device)  # noqa: E731
        if state_bits == 32:
            self.exp_avg, self.exp_avg_sq = zeros(self.state_len, torch.float32), zeros(self.state_len, torch.float32)
            self.exp_avg_scale = self.exp_avg_sq_scale = None
        else:
            self.exp_avg, self.exp_avg_sq = zeros(self.state_len, torch.int8), zeros(self.state_len, torch.uint8)
            self.exp_avg_scale = zeros(self.state_len // STATE_BLOCK, torch.float32)
            self.exp_avg_sq_scale = zeros(self.state_len // STATE_BLOCK, torch.float32)
        self.hparams = dict(lr=float(lr), beta1=float(betas[0]), beta2=float(betas[1]), eps=float(eps),
                            weight_decay=float(weight_decay))
        self._next_t = torch.ones(1, dtype=torch.int64, device=device) if capturable else None
        self._t = 0

    @property
    def capturable(self) -> bool:
        return self._next_t is not None

    @property
    def t(self) -> int:
        """Index of the last update applied (0 before the first)."""
        return self._t if self._next_t is None else int(self._next_t.item()) - 1

    @t.setter
    def t(self, value: int) -> None:
        if value < 0:
            raise ValueError("t must be >= 0")
        if self._next_t is not None:
            self._next_t.fill_(int(value) + 1)
        else:
            self._t = int(value)

    def _states(self):
        if self.state_bits == 32:
            return self.exp_avg.data_ptr(), self.exp_avg_sq.data_ptr(), None, None
        return (self.exp_avg.data_ptr(), self.exp_avg_sq.data_ptr(), self.exp_avg_scale.data_ptr(),
                self.exp_avg_sq_scale.data_ptr())

    def step(self, grad_scale=None, stream=None) -> None:
        here = _current()
        if grad_scale is not None and (_dtype(grad_scale, "grad_scale", here) != 0 or grad_scale.numel() != 1):
            raise ValueError("grad_scale must be one fp32 element")
        if self._next_t is not None:
            _on(here, self._next_t, "the update index")
        status = _lib.fsp_adamw_list_step(
            self._h, 0 if self.state_bits == 32 else 1, *self._states(), ctypes.byref(_fsp._hp(self.hparams)),
            self._t + 1, None if self._next_t is None else self._next_t.data_ptr(), 1,
            None if grad_scale is None else grad_scale.data_ptr(), _handle(stream, here))
        if status:
            _fsp._check(status, "fsp_adamw_list_step")
        if self._next_t is None:
            self._t += 1   # only once the step was accepted

    def _fp32_states(self, m, v, device: int):
        for x, what in ((m, "exp_avg"), (v, "exp_avg_sq")):
            if _dtype(x, what, device) != 0 or x.numel() != self.state_len or not x.is_contiguous():
                raise ValueError(f"{what} must be {self.state_len} contiguous fp32 elements")
        return m.data_ptr(), v.data_ptr()

    def state_values(self, out=None, stream=None):
        """(exp_avg, exp_avg_sq) as fp32 tensors of ``state_len`` elements: the
        states themselves with 32 bits, what the codes stand for with 8."""
        import torch
        if self.state_bits == 32:
            return self.exp_avg, self.exp_avg_sq
        here = _current()
        m, v = out if out is not None else [_empty((self.state_len,), torch.float32, self.exp_avg.device, stream)
                                            for _ in range(2)]
        _fsp._check(_fsp.lib().fsp_adamw_list_state_values(self._h, *self._states(), *self._fp32_states(m, v, here),
                                                           _handle(stream, here)), "fsp_adamw_list_state_values")
        return m, v

    def load_state(self, exp_avg, exp_avg_sq, stream=None) -> None:
        """Sets the states from fp32 tensors of ``state_len`` elements."""
        here = _current()
        pm, pv = self._fp32_states(exp_avg, exp_avg_sq, here)
        if self.state_bits == 32:
            with _on_stream(stream):
                self.exp_avg.copy_(exp_avg)
                self.exp_avg_sq.copy_(exp_avg_sq)
            return
        _fsp._check(_fsp.lib().fsp_adamw_list_state_load(self._h, pm, pv, *self._states(),
                                                         _handle(stream, here)), "fsp_adamw_list_state_load")

    def close(self):
        if self._h is not None and self._h.value:
            _fsp.lib().fsp_adamw_list_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- embedding -----------------------------------------------------------------

def embedding(weight, tokens, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """``out[..., :] = scale * weight[tokens[...], :]``, multiplied in fp32 and
    rounded once to ``out_dtype`` (default: the weight's).  A token outside the
    table gives zeros and sets bit 16 of ``device_error()``.  Nothing is recorded for
    autograd: the gradient is ``embedding_backward``'s."""
    here = _current()
    size = _tokens(tokens, here)
    code = _dtype(weight, "weight", here)
    vocab, dim, stride = _rows(weight, "weight")
    if out is None:
        out = _empty((*tokens.shape, dim), out_dtype or weight.dtype, weight.device, stream)
        out_stride = max(1, dim)
    else:
        if tuple(out.shape) != (*tokens.shape, dim) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out has another shape or dtype")
        out_stride = _flat(out, dim, "out")[1]
    status = _lib.fsp_embedding(weight.data_ptr(), code, vocab, dim, stride, tokens.data_ptr(), size, tokens.numel(),
                                scale, out.data_ptr(), _dtype(out, "out", here), out_stride, _handle(stream, here))
    if status:
        _fsp._check(status, "fsp_embedding")
    return out


def embedding_backward_workspace_bytes(vocab: int, dim: int, n_tokens: int) -> int:
    """Device workspace bytes ``embedding_backward`` needs."""
    out = ctypes.c_size_t(0)
    _fsp._check((_lib or _ready()).fsp_embedding_backward_workspace_bytes(vocab, dim, n_tokens, ctypes.byref(out)),
                "fsp_embedding_backward_workspace_bytes")
    return out.value


def embedding_backward(tokens, grad_out, grad_weight, scale: float = 1.0, padding_idx: int | None = None,
                       accumulate: bool = False, workspace=None, stream=None):
    """Writes (``accumulate``: adds) ``scale`` times the sum of ``grad_out``'s rows
    per token into ``grad_weight`` (vocab x dim) - a tensor of its own, or the
    embedding's slice of a rank's main-grad buffer.  ``padding_idx`` gets no
    gradient.  ``workspace``: a device tensor of at least
    ``embedding_backward_workspace_bytes`` bytes (None: allocated here)."""
    here = _current()
    size, n = _tokens(tokens, here), tokens.numel()
    vocab, dim, stride = _rows(grad_weight, "grad_weight")
    if tuple(grad_out.shape) != (*tokens.shape, dim):
        raise ValueError(f"grad_out must have shape {(*tokens.shape, dim)}")
    grad_stride = _flat(grad_out, dim, "grad_out")[1]
    if padding_idx is not None and not 0 <= padding_idx < vocab:
        raise ValueError("padding_idx is not a row of grad_weight")
    grad_code, code = _dtype(grad_out, "grad_out", here), _dtype(grad_weight, "grad_weight", here)
    if workspace is None:
        workspace = _empty(embedding_backward_workspace_bytes(vocab, dim, n), _torch.uint8, grad_weight.device, stream)
    work_bytes = _workspace_bytes(workspace, here)
    status = _lib.fsp_embedding_backward(
        tokens.data_ptr(), size, n, grad_out.data_ptr(), grad_code, dim, grad_stride,
        grad_weight.data_ptr(), code, vocab, stride, scale,
        -1 if padding_idx is None else padding_idx, 1 if accumulate else 0, workspace.data_ptr(),
        work_bytes, _handle(stream, here))
    if status:
        _fsp._check(status, "fsp_embedding_backward")
    return grad_weight


# ---- 8-bit floating point --------------------------------------------------------

class Fp8Matrix:
    """``rows`` x ``cols`` values as 8-bit codes with one power-of-two scale per
    block of 128 of a row, in the library's tile layout (``fsp_fp8_bytes``)."""

    def __init__(self, rows: int, cols: int, device="cuda", stream=None):
        nbytes, off = ctypes.c_size_t(), ctypes.c_size_t()
        _fsp._check((_lib or _ready()).fsp_fp8_bytes(rows, cols, ctypes.byref(nbytes), ctypes.byref(off)),
                    "fsp_fp8_bytes")
        self.rows, self.cols, self.scale_offset = rows, cols, off.value
        self.data = _empty(nbytes.value, _torch.uint8, device, stream)

    def values(self, stream=None):
        """What the codes stand for, as an fp32 tensor."""
        here = _current()
        _on(here, self.data, "the matrix")
        out = _empty((self.rows, self.cols), _torch.float32, self.data.device, stream)
        _fsp._check(_lib.fsp_fp8_values(self.data.data_ptr(), self.rows, self.cols, out.data_ptr(), _handle(stream, here)),
                    "fsp_fp8_values")
        return out


def quantize_fp8(x, rows=True, transposed=None, stream=None):
    """The 8-bit matrix of a 2-D tensor (fp32 or bf16), of its transpose, or both
    in one pass: ``rows`` and ``transposed`` are each True (a new ``Fp8Matrix``), an
    ``Fp8Matrix`` to fill, or None / False (not wanted).  Returns the wanted one, or
    the pair."""
    here = _current()
    code = _dtype(x, "x", here)
    r, c, stride = _rows(x, "x")
    got = []
    for want, shape in ((rows, (r, c)), (transposed, (c, r))):
        if want is True:
            want = Fp8Matrix(*shape, device=x.device, stream=stream)
        elif want is False:
            want = None
        if want is not None:
            if (want.rows, want.cols) != shape:
                raise ValueError(f"the matrix to fill is {want.rows} x {want.cols}, not {shape[0]} x {shape[1]}")
            _on(here, want.data, "the matrix to fill")
        got.append(want)
    _fsp._check(_lib.fsp_fp8_quantize(x.data_ptr(), code, r, c, stride,
                                      *[None if q is None else q.data.data_ptr() for q in got], _handle(stream, here)),
                "fsp_fp8_quantize")
    if got[0] is None:
        return got[1]
    return got[0] if got[1] is None else tuple(got)


def matmul_fp8(a: Fp8Matrix, b: Fp8Matrix, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """``out[m, n] = sum_k a[m, k] b[n, k]`` in fp32, rounded once to bf16 (the
    default) or fp32; ``accumulate`` adds to an fp32 ``out``."""
    if a.cols != b.cols:
        raise ValueError(f"the operands sum over {a.cols} and {b.cols} elements")
    here = _current()
    _on(here, a.data, "a")
    _on(here, b.data, "b")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = _empty((a.rows, b.rows), out_dtype or _torch.bfloat16, a.data.device, stream)
    elif tuple(out.shape) != (a.rows, b.rows) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has another shape or dtype")
    m, n, stride = _rows(out, "out")
    _fsp._check(_lib.fsp_fp8_matmul(a.data.data_ptr(), b.data.data_ptr(), m, n, a.cols, out.data_ptr(),
                                    _dtype(out, "out", here), stride, 1 if accumulate else 0, _handle(stream, here)),
                "fsp_fp8_matmul")
    return out


class Fp8Linear:
    """A linear layer ``y = x W^T`` whose products run on 8-bit operands: x, W and
    the output gradient are each quantised in blocks of 128 along the axis that
    the product sums over.

    ``Fp8Linear(weight)`` lays the out x in weight out for ``forward``; with
    ``train=True`` for ``backward`` too.  ``update(weight)`` does so again after an
    optimizer step.  Nothing is recorded for autograd: the gradients are
    ``backward``'s.
    """

    def __init__(self, weight, train: bool = False, stream=None):
        self.out_features, self.in_features, _ = _rows(weight, "weight")
        self.train = bool(train)
        self.codes = Fp8Matrix(self.out_features, self.in_features, weight.device, stream)
        self.codes_t = Fp8Matrix(self.in_features, self.out_features, weight.device, stream) if train else None
        self.update(weight, stream=stream)

    def update(self, weight, stream=None) -> None:
        """Lays out a new weight of the same shape."""
        quantize_fp8(weight, self.codes, self.codes_t, stream=stream)

    def _workspace(self, rows: int, backward: int, device, stream):
        size = ctypes.c_size_t(0)
        _fsp._check(_lib.fsp_fp8_linear_workspace_bytes(rows, self.in_features, self.out_features, backward,
                                                        ctypes.byref(size)), "fsp_fp8_linear_workspace_bytes")
        return _empty(size.value, _torch.uint8, device, stream) if size.value else None

    def forward(self, x, out=None, out_dtype=None, stream=None):
        """``x W^T`` (bf16 unless ``out`` or ``out_dtype`` says fp32)."""
        here = _current()
        code = _dtype(x, "x", here)
        w = self.codes.data
        if w.get_device() != here:
            _on(here, w, "the layer's weight")
        rows, stride = _flat(x, self.in_features, "x")
        n = self.out_features
        if out is None:
            out = _empty((*x.shape[:-1], n), out_dtype or _torch.bfloat16, x.device, stream)
            out_stride = max(1, n)
        else:
            if out.shape[:-1] != x.shape[:-1] or (out_dtype is not None and out.dtype != out_dtype):
                raise ValueError("out has another shape or dtype")
            out_stride = _flat(out, n, "out")[1]
        work = self._workspace(rows, 0, x.device, stream)
        status = _lib.fsp_fp8_linear(x.data_ptr(), code, rows, self.in_features, stride, w.data_ptr(), n,
                                     out.data_ptr(), _dtype(out, "out", here), out_stride,
                                     None if work is None else work.data_ptr(), 0 if work is None else work.numel(),
                                     _handle(stream, here))
        if status:
            _fsp._check(status, "fsp_fp8_linear")
        return out

    def backward(self, x, grad_out, grad_weight=None, accumulate: bool = False, need_grad_x: bool = True, out=None,
                 stream=None):
        """The gradient of x, ``grad_out W`` (bf16, or ``out``), and, into the fp32
        ``grad_weight`` where it is given, ``grad_out^T x`` (``accumulate``: added
        to it, as micro-batches add to a main gradient)."""
        if not self.train:
            raise ValueError("this layer was laid out for forward only (train=False)")
        k, n = self.in_features, self.out_features
        rows, stride = _flat(x, k, "x")
        dy_rows, dy_stride = _flat(grad_out, n, "grad_out")
        if rows != dy_rows:
            raise ValueError("x and grad_out must have as many rows")
        if not need_grad_x and grad_weight is None:
            return None
        here = _current()
        x_code, dy_code = _dtype(x, "x", here), _dtype(grad_out, "grad_out", here)
        w = self.codes_t.data
        _on(here, w, "the layer's weight")
        dx = dw = None
        dx_stride = dw_stride = max(1, k)
        dx_code = 1
        if need_grad_x:
            dx = out if out is not None else _empty(x.shape, _torch.bfloat16, x.device, stream)
            if dx.shape != x.shape:
                raise ValueError("out must have x's shape")
            dx_stride, dx_code = _flat(dx, k, "out")[1], _dtype(dx, "out", here)
        if grad_weight is not None:
            if _dtype(grad_weight, "grad_weight", here) != 0:
                raise TypeError("grad_weight must be fp32")
            if tuple(grad_weight.shape) != (n, k):
                raise ValueError(f"grad_weight must have shape {(n, k)}")
            dw, dw_stride = grad_weight, _rows(grad_weight, "grad_weight")[2]
        work = self._workspace(rows, 1, x.device, stream)
        _fsp._check(_lib.fsp_fp8_linear_backward(
            x.data_ptr(), x_code, stride, grad_out.data_ptr(), dy_code, dy_stride, rows, k, n, w.data_ptr(),
            None if dx is None else dx.data_ptr(), dx_code, dx_stride, None if dw is None else dw.data_ptr(), dw_stride, 1 if accumulate else 0,
            None if work is None else work.data_ptr(), 0 if work is None else work.numel(), _handle(stream, here)),
            "fsp_fp8_linear_backward")
        return dx


# ---- layer norm ------------------------------------------------------------------------

def _rows_of(x, what: str):
    """(rows, columns, row stride) of a tensor as rows of its last dimension (a number: of one)."""
    shape = x.shape
    dim = shape[-1] if shape else 1
    if dim and x.is_contiguous():
        return x.numel() // dim, dim, dim
    rows, stride = _flat(x, dim, what)
    return rows, dim, stride


def _row_stride(x, like, dim: int, what: str, dtype=None) -> int:
    """The row stride of a tensor (of ``dtype``, where one is given) that has the shape of ``like``."""
    if x.shape != like.shape or (dtype is not None and x.dtype != dtype):
        raise ValueError(f"{what} has another shape{'' if dtype is None else ' or dtype'}")
    return dim if dim and x.is_contiguous() else _flat(x, dim, what)[1] if x.shape else 1


def _param(x, dim: int, what: str, device: int) -> int:
    """The library's code of a parameter's dtype, a vector of ``dim`` adjacent elements."""
    code = _dtype(x, what, device)
    if x.shape != (dim,) or not x.is_contiguous():
        raise ValueError(f"{what} must be {dim} adjacent elements")
    return code


def _two_params(x, y, names, dim: int, device: int):
    """The one dtype code of two parameters, each of which may be None."""
    a = None if x is None else _param(x, dim, names[0], device)
    b = a if y is None else _param(y, dim, names[1], device)
    if a is not None and a != b:
        raise TypeError(f"{names[0]} and {names[1]} must have the same dtype")
    return b or 0


def _stats(stats, rows: int, device: int):
    """The address of the (mean, 1 / deviation) pairs of ``rows`` rows."""
    if _dtype(stats, "stats", device) != 0 or stats.numel() != 2 * rows or stats.size(-1) != 2 or not stats.is_contiguous():
        raise ValueError(f"stats must be contiguous fp32 pairs of {rows} rows")
    return stats.data_ptr()


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, center: bool = True, out=None, out_dtype=None, stats=None,
               stream=None):
    """``(x - m) / sqrt(mean((x - m)^2) + eps) * weight + bias`` over the last dimension,
    ``m`` its mean, or 0 with ``center=False`` (the norm by the root mean square); in
    fp32, rounded once to ``out_dtype`` (default: x's).  ``out`` may be ``x``.

    ``stats``: True (a new tensor), an fp32 tensor of shape ``(*x.shape[:-1], 2)`` to fill,
    or None; with it the call returns ``(out, stats)``, what ``layer_norm_backward``
    reads.  Nothing is recorded for autograd."""
    here = _current()
    code = _dtype(x, "x", here)
    rows, dim, stride = _rows_of(x, "x")
    param = _two_params(weight, bias, ("weight", "bias"), dim, here)
    if out is None:
        out = _empty(x.shape, out_dtype or x.dtype, x.device, stream)
        out_stride = dim or 1
    else:
        out_stride = _row_stride(out, x, dim, "out", out_dtype)
    if stats is True:
        stats = _empty((*x.shape[:-1], 2), _torch.float32, x.device, stream)
        stats_ptr = stats.data_ptr()
    elif stats is None or stats is False:
        stats = stats_ptr = None
    else:
        stats_ptr = _stats(stats, rows, here)
    status = _lib.fsp_layer_norm(x.data_ptr(), code, rows, dim, stride, None if weight is None else weight.data_ptr(),
                                 None if bias is None else bias.data_ptr(), param, eps, 1 if center else 0,
                                 out.data_ptr(), _dtype(out, "out", here), out_stride, stats_ptr, _handle(stream, here))
    if status:
        _fsp._check(status, "fsp_layer_norm")
    return out if stats is None else (out, stats)


@functools.lru_cache(maxsize=256)
def layer_norm_backward_workspace_bytes(rows: int, dim: int) -> int:
    """Device workspace bytes ``layer_norm_backward`` needs for the parameters' gradients."""
    out = ctypes.c_size_t(0)
    _fsp._check((_lib or _ready()).fsp_layer_norm_backward_workspace_bytes(rows, dim, ctypes.byref(out)),
                "fsp_layer_norm_backward_workspace_bytes")
    return out.value


def layer_norm_backward(x, stats, grad_out, weight=None, center: bool = True, grad_weight=None, grad_bias=None,
                        accumulate: bool = False, need_grad_x: bool = True, add=None, out=None, workspace=None,
                        stream=None):
    """The gradient of x (x's dtype, or ``out``'s buffer) from the forward pass's ``x``,
    ``stats`` and ``center``; ``add``, a tensor like x (the residual stream's gradient), is
    added to it.  ``grad_weight`` and ``grad_bias`` (fp32 or bf16, where given) receive
    (``accumulate``: are increased by) the sums over the rows.  ``out`` may be ``x``,
    ``grad_out`` or ``add``.  ``workspace``: a device tensor of at least
    ``layer_norm_backward_workspace_bytes`` bytes (None: allocated here)."""
    here = _current()
    code, dy_code = _dtype(x, "x", here), _dtype(grad_out, "grad_out", here)
    rows, dim, stride = _rows_of(x, "x")
    dy_stride = _row_stride(grad_out, x, dim, "grad_out")
    stats_ptr = _stats(stats, rows, here)
    weight_ptr = add_ptr = out_ptr = dw_ptr = db_ptr = work_ptr = None
    w_code = work_bytes = 0
    if weight is not None:
        w_code, weight_ptr = _param(weight, dim, "weight", here), weight.data_ptr()
    grad_code = _two_params(grad_weight, grad_bias, ("grad_weight", "grad_bias"), dim, here)
    if grad_weight is not None:
        dw_ptr = grad_weight.data_ptr()
    if grad_bias is not None:
        db_ptr = grad_bias.data_ptr()
    columns = grad_weight is not None or grad_bias is not None
    add_stride = dx_stride = dim or 1
    if not need_grad_x:
        if add is not None or out is not None:
            raise ValueError("add and out need need_grad_x")
        if not columns:
            return None
    else:
        if add is not None:
            _on(here, add, "add")
            add_stride, add_ptr = _row_stride(add, x, dim, "add", x.dtype), add.data_ptr()
        if out is None:
            out = _empty(x.shape, x.dtype, x.device, stream)
        else:
            _on(here, out, "out")
            dx_stride = _row_stride(out, x, dim, "out", x.dtype)
        out_ptr = out.data_ptr()
    if columns:
        if workspace is None:
            work_bytes = layer_norm_backward_workspace_bytes(rows, dim)
            if work_bytes:
                workspace = _empty(work_bytes, _torch.uint8, x.device, stream)
        else:
            work_bytes = _workspace_bytes(workspace, here)
        if work_bytes:
            work_ptr = workspace.data_ptr()
    status = _lib.fsp_layer_norm_backward(
        x.data_ptr(), code, rows, dim, stride, stats_ptr, 1 if center else 0, grad_out.data_ptr(), dy_code, dy_stride,
        weight_ptr, w_code, add_ptr, add_stride, out_ptr, dx_stride, dw_ptr, db_ptr, grad_code, 1 if accumulate else 0,
        work_ptr, work_bytes, _handle(stream, here))
    if status:
        _fsp._check(status, "fsp_layer_norm_backward")
    return out


# ---- dropout ---------------------------------------------------------------------------

def dropout(x, p: float, seed: int, call=0, residual=None, out=None, out_dtype=None, stream=None):
    """``x`` with each element dropped with probability ``p`` (a multiple of 2^-16, the
    nearest) or divided by 1 - p, plus ``residual`` where it is given; in fp32, rounded
    once to ``out_dtype`` (default: the residual's, or x's).  ``out`` may be ``x`` or
    ``residual``.

    Which elements go is a function of ``seed`` (64 bits), ``call`` (an int of 64 bits, or a device
    int64 tensor of one element: the form to capture in a CUDA graph) and the element's
    index, so no mask is stored: ``dropout_backward`` takes the same seed and call, and
    any two calls of a run should differ in one of them."""
    here = _current()
    code = _dtype(x, "x", here)
    rows, dim, stride = _rows_of(x, "x")
    call_ptr = None
    if isinstance(call, int):
        if not -1 << 63 <= call < 1 << 63:
            raise ValueError("call must be within 64 bits")   # (another call's masks otherwise)
    else:
        if call.dtype != _torch.int64 or call.numel() != 1:
            raise ValueError("call must be an int or one int64 element")
        _on(here, call, "call")
        call, call_ptr = 0, call.data_ptr()
    r_code, r_stride = 0, stride
    if residual is not None:
        r_code = _dtype(residual, "residual", here)
        r_stride = _row_stride(residual, x, dim, "residual")
    if out is None:
        out = _empty(x.shape, out_dtype or (x if residual is None else residual).dtype, x.device, stream)
        out_stride = dim or 1
    else:
        out_stride = _row_stride(out, x, dim, "out", out_dtype)
    status = _lib.fsp_dropout(x.data_ptr(), code, rows, dim, stride, p, seed & 0xFFFFFFFFFFFFFFFF, call, call_ptr,
                              None if residual is None else residual.data_ptr(), r_code, r_stride, out.data_ptr(),
                              _dtype(out, "out", here), out_stride, _handle(stream, here))
    if status:
        _fsp._check(status, "fsp_dropout")
    return out


def dropout_backward(grad_out, p: float, seed: int, call=0, out=None, out_dtype=None, stream=None):
    """The gradient of ``dropout``'s x, with the forward pass's ``p``, ``seed`` and ``call``
    (that of its residual is ``grad_out`` itself)."""
    return dropout(grad_out, p, seed, call, out=out, out_dtype=out_dtype, stream=stream)


# ---- rotary positions ------------------------------------------------------------------

class Rotary:
    """Rotary positions over the first ``dim`` elements of each head: pair j turns by its
    token's position times ``frequencies[j]``.

    ``layout``: ``"half"`` (pair j is elements j and j + dim / 2) or ``"interleaved"``
    (2 j and 2 j + 1).  The frequencies are ``base^(-2 j / dim)``, or for contexts longer
    than the trained one scaled by ``factor``: ``"linear"`` divides them by it, ``"ntk"``
    raises the base to ``base * factor^(dim / (dim - 2))``, and ``"yarn"`` (Peng, Quesnelle,
    Fan and Shippole, "YaRN: Efficient context window extension of large language models",
    2023) divides those that turn fewer than ``turns[0]`` times over ``original_length``
    positions, keeps those that turn more than ``turns[1]`` times, goes linearly from one
    to the other, and multiplies the rotated elements by ``0.1 ln(factor) + 1``.
    ``frequencies`` (radians per position) takes their place, ``scale`` that of the
    multiplier.

    ``forward`` and ``backward`` take a tensor, or a pair (queries and keys, one launch), of
    shape (tokens, heads, head_dim) or (batch, tokens, heads, head_dim), its last
    dimension adjacent and the others of any strides, and int32 or int64 positions of shape
    (tokens,) or (batch, tokens).  Nothing is recorded for autograd."""

    def __init__(self, dim: int, base: float = 10000.0, layout: str = "half", scaling: str | None = None, factor: float = 1.0,
                 original_length: int | None = None, turns=(1.0, 32.0), scale: float | None = None, frequencies=None,
                 device="cuda"):
        if _torch is None:
            _ready()
        if dim < 2 or dim % 2:
            raise ValueError("dim must be even and at least 2")
        if layout not in ("half", "interleaved"):
            raise ValueError("layout must be 'half' or 'interleaved'")
        if frequencies is None:
            frequencies = _frequencies(dim, base, scaling, factor, original_length, turns)
            if scale is None and scaling == "yarn":
                scale = 0.1 * math.log(factor) + 1.0
        elif scaling is not None:
            raise ValueError("frequencies and scaling exclude each other")
        self.frequencies = tuple(float(f) for f in frequencies)
        if len(self.frequencies) != dim // 2:
            raise ValueError(f"{dim // 2} frequencies are needed")
        self.dim, self.layout, self.scale = dim, layout, 1.0 if scale is None else float(scale)
        host = (ctypes.c_uint64 * (dim // 2))()
        _fsp._check(_lib.fsp_rotary_phases((ctypes.c_double * (dim // 2))(*self.frequencies), dim // 2, host),
                    "fsp_rotary_phases")
        self.phases = _torch.frombuffer(host, dtype=_torch.int64).to(device)

    def forward(self, x, positions, out=None, stream=None):
        """x (or the pair) rotated, in a new tensor or in ``out`` (a pair for a pair; x
        itself: in place).  Elements past ``dim`` are copied."""
        return self._run(x, positions, out, 0, stream)

    def backward(self, grad_out, positions, out=None, stream=None):
        """The gradient of ``forward``'s x: rotated back."""
        return self._run(grad_out, positions, out, 1, stream)

    def _run(self, x, positions, out, inverse: int, stream):
        here = _current()
        pair = isinstance(x, (tuple, list))
        xs = x if pair else (x,)
        n = len(xs)
        if not 1 <= n <= 2:
            raise ValueError("one tensor or a pair is rotated by a call")
        outs = (None,) * n if out is None else out if pair else (out,)
        if len(outs) != n:
            raise ValueError("out must be as many tensors")
        lead = xs[0].shape[:-2]
        dims, dtype = len(lead), xs[0].dtype
        if not 1 <= dims <= 2:
            raise ValueError("x must have 3 or 4 dimensions")
        batch, tokens = lead if dims == 2 else (1, lead[0])
        words, got = [], []
        for x_i, o in zip(xs, outs):
            shape = x_i.shape
            if shape[:-2] != lead:
                raise ValueError("the tensors must have the same batch and tokens")
            code = _dtype(x_i, "x", here)
            if x_i.dtype != dtype:
                raise TypeError("the tensors must have the same dtype")
            heads, head_dim = shape[-2:]
            strides = _head_strides(x_i, "x")
            if o is None:
                o = _empty(shape, dtype, x_i.device, stream)
                token = heads * head_dim
                out_strides = (tokens * token, token, head_dim)
            else:
                if o.shape != shape or o.dtype != dtype:
                    raise ValueError("out has another shape or dtype")
                if o.get_device() != here:
                    _on(here, o, "out")
                out_strides = _head_strides(o, "out")
            words += (x_i.data_ptr(), o.data_ptr(), heads, head_dim, *strides, *out_strides)
            got.append(o)
        if positions.get_device() != here:
            _on(here, positions, "positions")
        index = _INDEX.get(positions.dtype)
        if index is None:
            raise TypeError(f"positions: unsupported dtype {positions.dtype}")
        if positions.shape == lead:
            positions_stride = tokens
        elif positions.shape == (tokens,):
            positions_stride = 0
        else:
            raise ValueError(f"positions must have shape {tuple(lead)} or {(tokens,)}")
        if not positions.is_contiguous():
            raise ValueError("positions must be contiguous")
        phases = self.phases
        if phases.get_device() != here:
            _on(here, phases, "the frequencies")
        status = _lib.fsp_rotary(_WORDS[n](*words), n, code, batch, tokens, positions.data_ptr(), index, positions_stride,
                                 phases.data_ptr(), self.dim, 0 if self.layout == "half" else 1, self.scale, inverse,
                                 _handle(stream, here))
        if status:
            _fsp._check(status, "fsp_rotary")
        return tuple(got) if pair else got[0]


_WORDS = (None, struct.Struct("=10q").pack, struct.Struct("=20q").pack)   # one fsp_rotary_tensor, two


def _head_strides(x, what: str):
    """Strides of the batches, tokens and heads of a tensor whose heads' elements are adjacent."""
    strides = x.stride()
    if strides[-1] != 1 and x.shape[-1] > 1:
        raise ValueError(f"{what}: the elements of a head must be adjacent")
    return strides[:3] if len(strides) == 4 else (0, *strides[:2])


def _frequencies(dim: int, base: float, scaling, factor: float, length, turns):
    """Radians per position of each pair."""
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError("scaling must be 'linear', 'ntk', 'yarn' or None")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be above 0")
    if scaling == "ntk" and dim > 2:
        base *= factor ** (dim / (dim - 2))
    f = [base ** (-2 * j / dim) for j in range(dim // 2)]
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling != "yarn":
        return f
    if not length or length < 0:
        raise ValueError("yarn needs original_length")
    few, many = turns
    if not few < many:
        raise ValueError("turns must increase")
    kept = [min(max((x * length / math.tau - few) / (many - few), 0.0), 1.0) for x in f]
    return [x / factor * (1 - k) + x * k for x, k in zip(f, kept)]
