"""The operators of ``include/fsp_ops.h`` on torch tensors: AdamW over a list
of tensors, the embedding with its gradient, and matrices in 8-bit floating
point.  Argument marshalling and output buffers only; everything is computed by
the library's kernels, asynchronously on ``stream`` (None: the current one) and the
current device, where every tensor of a call has to be.
"""
from __future__ import annotations

import ctypes

from . import fsp as _fsp
from .optim import _on_stream

STATE_BLOCK = 256   # elements of a tensor that share a scale in 8-bit AdamW states

EXPORTS = ("fsp_adamw_list_create", "fsp_adamw_list_info", "fsp_adamw_list_destroy", "fsp_adamw_list_step",
           "fsp_adamw_list_state_values", "fsp_adamw_list_state_load", "fsp_embedding",
           "fsp_embedding_backward_workspace_bytes", "fsp_embedding_backward", "fsp_fp8_bytes", "fsp_fp8_quantize",
           "fsp_fp8_values", "fsp_fp8_matmul", "fsp_fp8_linear", "fsp_fp8_linear_backward",
           "fsp_fp8_linear_workspace_bytes")


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
    if workspace is not None:
        _on(here, workspace, "workspace")
    else:
        workspace = _empty(embedding_backward_workspace_bytes(vocab, dim, n), _torch.uint8, grad_weight.device, stream)
    status = _lib.fsp_embedding_backward(
        tokens.data_ptr(), size, n, grad_out.data_ptr(), grad_code, dim, grad_stride,
        grad_weight.data_ptr(), code, vocab, stride, scale,
        -1 if padding_idx is None else padding_idx, 1 if accumulate else 0, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _handle(stream, here))
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
