"""Running a solved layer on 8-bit integer tensor cores.

A layer solved with ``group_size=-1`` becomes an ``Int8Layer``; activations
become ``Int8Tokens``.  The functions without the ``gptq_`` prefix allocate
their outputs and run on the current stream; those with it carry the C ABI's
names (``include/gptq.h``, where the formulas and limits stand) and write into
tensors the caller owns.

    layer = int8_layer(solve_layer(W, X, dict(bits=8, sym=True, group_size=-1)), bits=8)
    y = linear_int8(x, layer)                      # x [tokens, in], 16 or 32 bits
    a = gated_int8(x, gate, up, act="silu")        # act(gate projection) * up projection
    h, xq = norm_tokens(h, y, weight, quantize=True)
    h, y = mlp_int8(h, y, weight, gate, up, down)  # a decoder block's MLP half

Activations are 2-D, tokens in rows, rows contiguous (any row stride).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _check, _dt, _i64, _p, _ptr, _rowmajor, _stream, lib

_NORMS = {"rms": 0, "layer": 1}
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_int = ctypes.c_int


class _Tokens(ctypes.Structure):
    _fields_ = [("q", _p), ("ldq", _i64), ("scale", _p), ("sum", _p)]


class _Layer(ctypes.Structure):
    _fields_ = [("w", _p), ("ldw", _i64), ("scale", _p), ("zero", _p)]


class _Norm(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("d", _i64), ("ht", _int), ("yt", _int), ("kind", _int),
                ("eps", ctypes.c_float), ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("h", _p), ("ldh", _i64), ("y", _p), ("ldy", _i64), ("post_weight", _p), ("post_bias", _p),
                ("gate", _p), ("ldgate", _i64), ("weight", _p), ("bias", _p), ("h_out", _p), ("ldh_out", _i64),
                ("x", _p), ("ldx", _i64), ("q", _p), ("ldq", _i64), ("scale", _p), ("sum", _p)]


lib.gptq_layout_int8.argtypes = [_p, _p, _i64, _i64, _int, _p, _i64, _p, _p]
lib.gptq_layout_int8.restype = _int
lib.gptq_quantize_tokens.argtypes = [_p, _int, _i64, _i64, _i64, _p, _i64, _p, _p, _p]
lib.gptq_quantize_tokens.restype = _int
lib.gptq_norm_tokens.argtypes = [ctypes.POINTER(_Norm), _p]
lib.gptq_norm_tokens.restype = _int
lib.gptq_matmul_int8.argtypes = [ctypes.POINTER(_Tokens), _i64, _i64, ctypes.POINTER(_Layer), _i64, _p, _p, _int,
                                 _i64, _p]
lib.gptq_matmul_int8.restype = _int
lib.gptq_matmul_int8_gated.argtypes = [ctypes.POINTER(_Tokens), _i64, _i64, ctypes.POINTER(_Layer),
                                       ctypes.POINTER(_Layer), _i64, _int, _p, _int, _i64, _p]
lib.gptq_matmul_int8_gated.restype = _int
lib.gptq_int8_status.argtypes = [_p]
lib.gptq_int8_status.restype = _int


class Int8Layer(NamedTuple):
    """A layer of weights scale[n] * (weight[n][k] - zero[n])."""
    weight: torch.Tensor                  # int8 [out, in], row stride a multiple of 16
    scale: torch.Tensor                   # float32 [out]
    zero: Optional[torch.Tensor] = None   # int32 [out], |zero| <= 255; None: all zero


class Int8Tokens(NamedTuple):
    """Activations scale[t] * q[t][k], with the sum of each token's codes."""
    q: torch.Tensor                       # int8 [tokens, in], row stride a multiple of 16
    scale: torch.Tensor                   # float32 [tokens]
    sum: torch.Tensor                     # int32 [tokens]


# ------------------------------------------------------------------ checks
# The library sees addresses only: types, shapes and devices are checked here.
def _vector(t, n, dtype, device, name):
    if t.dtype is not dtype or t.shape != (n,) or (n > 1 and t.stride(0) != 1) or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} elements on {device}")


def _matrix(t, rows, cols, dtype, device, name):
    if t.dtype is not dtype or t.shape != (rows, cols) or t.device != device:
        raise ValueError(f"{name} must be a {dtype} matrix of {rows} x {cols} on {device}")
    _rows(t, name)


def _rows(t, name):
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")


def _ld(t):
    """The row stride; a single row's is of no account."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _ld8(t):
    return t.stride(0) if t.shape[0] > 1 else _round16(t.shape[1])


def _round16(n):
    return (n + 15) // 16 * 16


def _int8_rows(rows, cols, device):
    """A rows x cols int8 matrix with 16-byte aligned rows."""
    return torch.empty((rows, _round16(cols)), dtype=torch.int8, device=device)[:, :cols]


def _c_tokens(x):
    q = x.q
    if q.dtype is not torch.int8:
        raise ValueError(f"x.q must be int8, got {q.dtype}")
    _rows(q, "x.q")
    _vector(x.scale, q.shape[0], torch.float32, q.device, "x.scale")
    _vector(x.sum, q.shape[0], torch.int32, q.device, "x.sum")
    return _Tokens(q.data_ptr(), _ld8(q), x.scale.data_ptr(), x.sum.data_ptr())


def _c_layer(layer, in_, device, name):
    weight, scale, zero = layer if len(layer) == 3 else (*layer, None)
    if weight.dim() != 2:
        raise ValueError(f"{name}: the weight must be a 2-D tensor")
    out = weight.shape[0]
    _matrix(weight, out, in_, torch.int8, device, f"{name}: the weight")
    _vector(scale, out, torch.float32, device, f"{name}: the scale")
    if zero is not None:
        _vector(zero, out, torch.int32, device, f"{name}: the zero")
    return _Layer(weight.data_ptr(), _ld8(weight), scale.data_ptr(), None if zero is None else zero.data_ptr()), out


class _on:
    """The tensors' device as the current one for a call."""

    def __init__(self, t):
        if not t.is_cuda:
            raise ValueError(f"the tensors must be on a CUDA device, not {t.device}")
        index = t.device.index
        self.guard = None if index == torch.cuda.current_device() else torch.cuda.device(index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


# --------------------------------------------------------------- ABI calls
def gptq_layout_int8(qweight, zeros, bits, weight, zero=None, stream=None) -> None:
    """weight (int8, out x in) and zero (int32, out) of a layer solved with
    one group per row, from its packed codes and zeros (int32, out or out x 1)."""
    _rows(weight, "weight")
    out, in_ = weight.shape
    dev = weight.device
    if weight.dtype is not torch.int8:
        raise ValueError(f"weight must be int8, got {weight.dtype}")
    if qweight.dtype not in (torch.int32, torch.uint32) or not qweight.is_contiguous() or \
            qweight.numel() != out * in_ * bits // 32 or qweight.device != dev:
        raise ValueError(f"qweight must hold {out} contiguous rows of {in_ * bits // 32} words on {dev}")
    _vector(zeros.reshape(-1), out, torch.int32, dev, "zeros")
    if zero is not None:
        _vector(zero, out, torch.int32, dev, "zero")
    with _on(weight):
        _check(lib.gptq_layout_int8(_ptr(qweight), _ptr(zeros), out, in_, int(bits), _ptr(weight), _ld8(weight),
                                    _ptr(zero), _stream(stream)))


def gptq_quantize_tokens(X, q, scale, sum, stream=None) -> None:
    """q (int8), scale (float32) and sum (int32) <- X [tokens, in]."""
    _rows(X, "X")
    _matrix(q, *X.shape, torch.int8, X.device, "q")
    _vector(scale, X.shape[0], torch.float32, X.device, "scale")
    _vector(sum, X.shape[0], torch.int32, X.device, "sum")
    with _on(X):
        _check(lib.gptq_quantize_tokens(X.data_ptr(), _dt(X), *X.shape, _ld(X), q.data_ptr(), _ld8(q),
                                        scale.data_ptr(), sum.data_ptr(), _stream(stream)))


def gptq_norm_tokens(h, y=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, alpha=1.0,
                     beta=1.0, kind="rms", eps=1e-6, h_out=None, x=None, tokens=None, dtype=None,
                     stream=None) -> None:
    """h_out, x and/or tokens (an Int8Tokens) <- the norms around a block.
    h_out may be h.  ``dtype`` names the type of weight and bias where neither
    y nor x is given."""
    _rows(h, "h")
    T, d = h.shape
    dev, ht = h.device, h.dtype
    yt = next((t.dtype for t in (y, x, weight) if t is not None), dtype or ht)
    if kind not in _NORMS:
        raise ValueError(f"kind must be one of {sorted(_NORMS)}, got {kind!r}")
    for name, t, dt in (("y", y, yt), ("x", x, yt), ("h_out", h_out, ht)):
        if t is not None:
            _matrix(t, T, d, dt, dev, name)
    for name, t in (("weight", weight), ("bias", bias), ("post_weight", post_weight), ("post_bias", post_bias)):
        if t is not None:
            _vector(t, d, yt, dev, name)
    ldgate = 0
    if gate is not None and gate.dim() == 2:
        _matrix(gate, T, d, yt, dev, "gate")
        ldgate = _ld(gate)
    elif gate is not None:
        _vector(gate, d, yt, dev, "gate")
    a = _Norm(T, d, _dt(h), _dt_of(yt), _NORMS[kind], eps, alpha, beta, h.data_ptr(), _ld(h),
              _at(y), 0 if y is None else _ld(y), _at(post_weight), _at(post_bias), _at(gate), ldgate,
              _at(weight), _at(bias), _at(h_out), 0 if h_out is None else _ld(h_out),
              _at(x), 0 if x is None else _ld(x), None, 0, None, None)
    if tokens is not None:
        _matrix(tokens.q, T, d, torch.int8, dev, "tokens.q")
        _vector(tokens.scale, T, torch.float32, dev, "tokens.scale")
        _vector(tokens.sum, T, torch.int32, dev, "tokens.sum")
        a.q, a.ldq, a.scale, a.sum = tokens.q.data_ptr(), _ld8(tokens.q), tokens.scale.data_ptr(), \
            tokens.sum.data_ptr()
    with _on(h):
        _check(lib.gptq_norm_tokens(a, _stream(stream)))


def gptq_matmul_int8(x, layer, Y, bias=None, stream=None) -> None:
    """Y [tokens, out] <- the product of x (Int8Tokens) with an Int8Layer."""
    xs = _c_tokens(x)
    T, in_ = x.q.shape
    w, out = _c_layer(layer, in_, x.q.device, "layer")
    _matrix(Y, T, out, Y.dtype, x.q.device, "Y")
    if bias is not None:
        _vector(bias, out, torch.float32, x.q.device, "bias")
    yt = _dt(Y)
    with _on(x.q):
        _check(lib.gptq_matmul_int8(xs, T, in_, w, out, _at(bias), Y.data_ptr(), yt, _ld(Y), _stream(stream)))


def gptq_matmul_int8_gated(x, gate, up, Y, act="silu", stream=None) -> None:
    """Y [tokens, out] <- act(x gate^T) * (x up^T)."""
    xs = _c_tokens(x)
    T, in_ = x.q.shape
    dev = x.q.device
    wg, out = _c_layer(gate, in_, dev, "gate")
    wu, out_up = _c_layer(up, in_, dev, "up")
    if out_up != out:
        raise ValueError(f"gate and up differ in size: {out} and {out_up} channels")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    _matrix(Y, T, out, Y.dtype, dev, "Y")
    yt = _dt(Y)
    with _on(x.q):
        _check(lib.gptq_matmul_int8_gated(xs, T, in_, wg, wu, out, _ACTS[act], Y.data_ptr(), yt, _ld(Y),
                                          _stream(stream)))


def gptq_int8_status(stream=None) -> None:
    """Wait for the stream and raise GptqError if a bounded device-side wait
    of an int8 product on this device has given up since the last call."""
    _check(lib.gptq_int8_status(_stream(stream)))


def _at(t):
    return None if t is None else t.data_ptr()


_DTYPE_CODES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _dt_of(dtype):
    if dtype not in _DTYPE_CODES:
        raise TypeError(f"unsupported dtype {dtype}")
    return _DTYPE_CODES[dtype]


# ---------------------------------------------------------- allocating calls
def int8_layer(r, bits: int) -> Int8Layer:
    """The Int8Layer of a layer solved with ``group_size=-1``: r is the dict
    solve_layer or solve_block returned (or any with its qweight, scales and
    zeros), bits the width it was solved with.  A symmetric 8-bit layer has
    only zeros in ``zero``; pass ``layer._replace(zero=None)`` to skip them."""
    qweight, scales, zeros = r["qweight"], r["scales"], r["zeros"]
    if qweight is None:
        raise ValueError("the layer has no packed codes (in * bits is not a multiple of 32)")
    if scales.dim() != 2 or scales.shape[1] != 1:
        raise ValueError("an int8 layer needs one scale per output channel: solve with group_size=-1")
    out, in_ = scales.shape[0], qweight.shape[1] * 32 // bits
    weight = _int8_rows(out, in_, scales.device)
    zero = torch.empty(out, dtype=torch.int32, device=scales.device) if bits == 8 else None
    gptq_layout_int8(qweight, zeros, bits, weight, zero)
    return Int8Layer(weight, scales.reshape(-1), zero)


def quantize_tokens(X) -> Int8Tokens:
    """X [tokens, in] (f16, bf16 or f32) with a scale for each token."""
    _rows(X, "X")
    T, in_ = X.shape
    x = Int8Tokens(_int8_rows(T, in_, X.device), torch.empty(T, dtype=torch.float32, device=X.device),
                   torch.empty(T, dtype=torch.int32, device=X.device))
    gptq_quantize_tokens(X, *x)
    return x


def norm_tokens(h, y=None, weight=None, *, bias=None, post_weight=None, post_bias=None, gate=None, alpha=1.0,
                beta=1.0, kind="rms", eps=1e-6, quantize=False, inplace=False):
    """(h', x): h' = alpha h + beta gate * post(y) and x = pre(h'), the norms
    before and after a block with its gate and residual scale.

    h is the residual stream (float32 or y's type), y the block's output
    (None for the first block's norm), weight and bias the pre-norm's,
    post_weight and post_bias the post-norm's (None: no post-norm), gate a
    vector over channels or a [tokens, d] matrix.  kind is "rms" or "layer".
    ``quantize`` returns x as Int8Tokens; ``inplace`` writes h' over h.
    Without y and with alpha 1, h' is h and h itself is returned."""
    _rows(h, "h")
    if weight is None:
        raise ValueError("weight (the pre-norm's) is needed")
    T, d = h.shape
    h_out = h if inplace else None if y is None and alpha == 1.0 else torch.empty((T, d), dtype=h.dtype,
                                                                                  device=h.device)
    if quantize:
        x, tokens = None, Int8Tokens(_int8_rows(T, d, h.device), torch.empty(T, dtype=torch.float32, device=h.device),
                                     torch.empty(T, dtype=torch.int32, device=h.device))
    else:
        x, tokens = torch.empty((T, d), dtype=weight.dtype, device=h.device), None
    gptq_norm_tokens(h, y, weight, bias, post_weight, post_bias, gate, alpha, beta, kind, eps, h_out, x, tokens)
    return (h if h_out is None else h_out), (tokens if quantize else x)


def linear_int8(x, layer, bias=None, dtype=None):
    """x [tokens, in] times an Int8Layer (or (weight, scale[, zero])), plus
    bias (float32).  A floating x is quantized by token first; the result has
    ``dtype``, by default x's (bfloat16 for Int8Tokens)."""
    if not isinstance(x, Int8Tokens):
        dtype = dtype or x.dtype
        x = quantize_tokens(x)
    Y = torch.empty((x.q.shape[0], layer[0].shape[0]), dtype=dtype or torch.bfloat16, device=x.q.device)
    gptq_matmul_int8(x, layer, Y, bias)
    return Y


def gated_int8(x, gate, up, act="silu", dtype=None):
    """act(x gate^T) * (x up^T) in one kernel; x, gate, up and dtype as in
    linear_int8, act one of "silu", "gelu", "gelu_tanh"."""
    if not isinstance(x, Int8Tokens):
        dtype = dtype or x.dtype
        x = quantize_tokens(x)
    Y = torch.empty((x.q.shape[0], gate[0].shape[0]), dtype=dtype or torch.bfloat16, device=x.q.device)
    gptq_matmul_int8_gated(x, gate, up, Y, act)
    return Y


def mlp_int8(h, y, weight, gate, up, down, act="silu", **norm):
    """The MLP half of a solved decoder block: (h', z) with h' the residual
    stream after the attention output y and z = down(act(gate x) * up x), x
    the pre-norm of h'.  ``norm`` takes norm_tokens' keywords.  Feed (h', z)
    to the next block's norm_tokens."""
    h, x = norm_tokens(h, y, weight, quantize=True, **norm)
    a = gated_int8(x, gate, up, act, dtype=weight.dtype)
    return h, linear_int8(a, down)
