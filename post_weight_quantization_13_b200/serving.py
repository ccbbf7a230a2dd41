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

Only layers with one scale for each output channel run here: one solved in
groups of columns (``group_size`` 64 or 128, as a 4-bit checkpoint has it) is
refused by ``int8_layer``.  Activations are 2-D, tokens in rows, rows contiguous
(any row stride).  These are inference calls: a solved layer is frozen, and no
gradient flows through them, whatever ``requires_grad`` says.  They do not wait
for the device: a wait inside a kernel that gave up, and left a result
incomplete, shows in ``gptq_int8_status`` only.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import GptqError, _check, _i64, _p, lib
from . import _serving  # type: ignore[attr-defined]  (built beside libgptq.so; there is no fallback)

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
lib.gptq_linear_int8_ws_bytes.argtypes = [_i64, _i64]
lib.gptq_linear_int8_ws_bytes.restype = ctypes.c_size_t
lib.gptq_linear_int8.argtypes = [_p, _int, _i64, _i64, _i64, ctypes.POINTER(_Layer), _i64, _p, _p, _int, _i64, _p,
                                 ctypes.c_size_t, _p]
lib.gptq_linear_int8.restype = _int
lib.gptq_linear_int8_gated.argtypes = [_p, _int, _i64, _i64, _i64, ctypes.POINTER(_Layer), ctypes.POINTER(_Layer),
                                       _i64, _int, _p, _int, _i64, _p, ctypes.c_size_t, _p]
lib.gptq_linear_int8_gated.restype = _int
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


_serving.init(GptqError, Int8Tokens)


# ------------------------------------------------------------------ checks
# The library sees addresses only: types, shapes and devices are checked here.
# (The allocating calls below go through _serving.so, which makes the same
# checks: at decode these lines cost more than the kernels they launch.)
_CODES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _code(dtype):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _vector(t, n, dtype, device, name):
    """The address of a contiguous vector."""
    if t.dtype is not dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} elements on {device}")
    return t.data_ptr()


def _matrix(t, shape, dtype, device, name):
    """The address and row stride of a matrix with contiguous rows."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be a {dtype} matrix of {shape[0]} x {shape[1]} on {device}")
    return t.data_ptr(), _ld(t, name)


def _ld(t, name):
    """The row stride; a single row's is of no account, and is given as the
    shortest any call accepts."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    ld, one = t.stride()
    rows, cols = t.shape
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    return ld if rows > 1 else _round16(cols)


def _round16(n):
    return (n + 15) & ~15


def _int8_rows(rows, cols, device):
    """A rows x cols int8 matrix with 16-byte aligned rows."""
    return torch.empty((rows, _round16(cols)), dtype=torch.int8, device=device)[:, :cols]


def _c_tokens(x):
    q = x.q
    if q.dtype is not torch.int8:
        raise ValueError(f"x.q must be int8, got {q.dtype}")
    ld, n, dev = _ld(q, "x.q"), q.shape[0], q.device
    return _Tokens(q.data_ptr(), ld, _vector(x.scale, n, torch.float32, dev, "x.scale"),
                   _vector(x.sum, n, torch.int32, dev, "x.sum"))


def _c_layer(layer, in_, device, name):
    """(the C struct, the channels) of an Int8Layer or (weight, scale[, zero])."""
    weight, scale = layer[0], layer[1]
    zero = layer[2] if len(layer) > 2 else None
    if weight.dim() != 2:
        raise ValueError(f"{name}: the weight must be a 2-D tensor")
    out = weight.shape[0]
    w, ld = _matrix(weight, (out, in_), torch.int8, device, f"{name}.weight")
    return _Layer(w, ld, _vector(scale, out, torch.float32, device, f"{name}.scale"),
                  None if zero is None else _vector(zero, out, torch.int32, device, f"{name}.zero")), out


def _call(device, stream, fn, *args):
    """fn on the tensors' device and the stream (None: its current one)."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, not {device}")
    index = device.index
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status:
        _check(status)


# --------------------------------------------------------------- ABI calls
def gptq_layout_int8(qweight, zeros, bits, weight, zero=None, stream=None) -> None:
    """weight (int8, out x in) and zero (int32, out) of a layer solved with
    one group per row, from its packed codes and zeros (int32, out or out x 1)."""
    dev = weight.device
    if weight.dtype is not torch.int8:
        raise ValueError(f"weight must be int8, got {weight.dtype}")
    ld = _ld(weight, "weight")
    out, in_ = weight.shape
    if qweight.dtype not in (torch.int32, torch.uint32) or not qweight.is_contiguous() or \
            qweight.numel() != out * in_ * bits // 32 or qweight.device != dev:
        raise ValueError(f"qweight must hold {out} contiguous rows of {in_ * bits // 32} words on {dev}")
    if not zeros.is_contiguous():
        raise ValueError("zeros must be contiguous")
    z = _vector(zeros.view(-1), out, torch.int32, dev, "zeros")
    z8 = None if zero is None else _vector(zero, out, torch.int32, dev, "zero")
    _call(dev, stream, lib.gptq_layout_int8, qweight.data_ptr(), z, out, in_, int(bits), weight.data_ptr(), ld, z8)


def gptq_quantize_tokens(X, q, scale, sum, stream=None) -> None:
    """q (int8), scale (float32) and sum (int32) <- X [tokens, in]."""
    ldx, code, dev = _ld(X, "X"), _code(X.dtype), X.device
    T, in_ = X.shape
    qp, ldq = _matrix(q, (T, in_), torch.int8, dev, "q")
    _call(dev, stream, lib.gptq_quantize_tokens, X.data_ptr(), code, T, in_, ldx, qp, ldq,
          _vector(scale, T, torch.float32, dev, "scale"), _vector(sum, T, torch.int32, dev, "sum"))


def gptq_norm_tokens(h, y=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, alpha=1.0,
                     beta=1.0, kind="rms", eps=1e-6, h_out=None, x=None, tokens=None, stream=None) -> None:
    """h_out, x and/or tokens (an Int8Tokens) <- the norms around a block.
    h_out may be h."""
    ldh, dev, ht = _ld(h, "h"), h.device, h.dtype
    T, d = shape = h.shape
    yt = y.dtype if y is not None else weight.dtype if weight is not None else ht
    if kind not in _NORMS:
        raise ValueError(f"kind must be one of {sorted(_NORMS)}, got {kind!r}")

    def matrix(t, dtype, name):
        return (None, 0) if t is None else _matrix(t, shape, dtype, dev, name)

    def vector(t, name):
        return None if t is None else _vector(t, d, yt, dev, name)

    if gate is not None and gate.dim() == 2:
        g, ldgate = _matrix(gate, shape, yt, dev, "gate")
    else:
        g, ldgate = vector(gate, "gate"), 0
    a = _Norm(T, d, _code(ht), _code(yt), _NORMS[kind], eps, alpha, beta, h.data_ptr(), ldh, *matrix(y, yt, "y"),
              vector(post_weight, "post_weight"), vector(post_bias, "post_bias"), g, ldgate,
              vector(weight, "weight"), vector(bias, "bias"), *matrix(h_out, ht, "h_out"), *matrix(x, yt, "x"))
    if tokens is not None:
        a.q, a.ldq = _matrix(tokens.q, shape, torch.int8, dev, "tokens.q")
        a.scale = _vector(tokens.scale, T, torch.float32, dev, "tokens.scale")
        a.sum = _vector(tokens.sum, T, torch.int32, dev, "tokens.sum")
    _call(dev, stream, lib.gptq_norm_tokens, a)


def gptq_matmul_int8(x, layer, Y, bias=None, stream=None) -> None:
    """Y [tokens, out] <- the product of x (Int8Tokens) with an Int8Layer."""
    xs, dev = _c_tokens(x), x.q.device
    T, in_ = x.q.shape
    w, out = _c_layer(layer, in_, dev, "layer")
    yt = _code(Y.dtype)
    y, ldy = _matrix(Y, (T, out), Y.dtype, dev, "Y")
    b = None if bias is None else _vector(bias, out, torch.float32, dev, "bias")
    _call(dev, stream, lib.gptq_matmul_int8, xs, T, in_, w, out, b, y, yt, ldy)


def gptq_matmul_int8_gated(x, gate, up, Y, act="silu", stream=None) -> None:
    """Y [tokens, out] <- act(x gate^T) * (x up^T)."""
    xs, dev = _c_tokens(x), x.q.device
    T, in_ = x.q.shape
    wg, wu, out, code = _c_pair(gate, up, in_, dev, act)
    yt = _code(Y.dtype)
    y, ldy = _matrix(Y, (T, out), Y.dtype, dev, "Y")
    _call(dev, stream, lib.gptq_matmul_int8_gated, xs, T, in_, wg, wu, out, code, y, yt, ldy)


def gptq_linear_int8_ws_bytes(tokens: int, in_: int) -> int:
    return lib.gptq_linear_int8_ws_bytes(tokens, in_)


def gptq_linear_int8(X, layer, Y, ws=None, bias=None, stream=None) -> None:
    """Y [tokens, out] <- the product of floating activations X [tokens, in],
    quantized by token, with an Int8Layer.  ws: a workspace tensor of
    gptq_linear_int8_ws_bytes bytes (none where that is 0)."""
    ldx, xt, dev = _ld(X, "X"), _code(X.dtype), X.device
    T, in_ = X.shape
    w, out = _c_layer(layer, in_, dev, "layer")
    yt = _code(Y.dtype)
    y, ldy = _matrix(Y, (T, out), Y.dtype, dev, "Y")
    b = None if bias is None else _vector(bias, out, torch.float32, dev, "bias")
    wsp, nws = _workspace(ws, dev)
    _call(dev, stream, lib.gptq_linear_int8, X.data_ptr(), xt, T, in_, ldx, w, out, b, y, yt, ldy, wsp, nws)


def gptq_linear_int8_gated(X, gate, up, Y, ws=None, act="silu", stream=None) -> None:
    """Y [tokens, out] <- act(X gate^T) * (X up^T), X as in gptq_linear_int8."""
    ldx, xt, dev = _ld(X, "X"), _code(X.dtype), X.device
    T, in_ = X.shape
    wg, wu, out, code = _c_pair(gate, up, in_, dev, act)
    yt = _code(Y.dtype)
    y, ldy = _matrix(Y, (T, out), Y.dtype, dev, "Y")
    wsp, nws = _workspace(ws, dev)
    _call(dev, stream, lib.gptq_linear_int8_gated, X.data_ptr(), xt, T, in_, ldx, wg, wu, out, code, y, yt, ldy, wsp,
          nws)


def _c_pair(gate, up, in_, dev, act):
    wg, out = _c_layer(gate, in_, dev, "gate")
    wu, out_up = _c_layer(up, in_, dev, "up")
    if out_up != out:
        raise ValueError(f"gate and up differ in size: {out} and {out_up} channels")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return wg, wu, out, _ACTS[act]


def _workspace(ws, dev):
    if ws is None:
        return None, 0
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def gptq_int8_status(stream=None) -> None:
    """Wait for the stream and raise GptqError if a bounded device-side wait
    of any of these calls on its device has given up since the last time.
    The calls themselves do not wait for the device and cannot tell."""
    _call(torch.device("cuda", torch.cuda.current_device()) if stream is None else stream.device, stream,
          lib.gptq_int8_status)


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
    return _serving.quantize(X)


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
    if weight is None:
        raise ValueError("weight (the pre-norm's) is needed")
    if kind not in _NORMS:
        raise ValueError(f"kind must be one of {sorted(_NORMS)}, got {kind!r}")
    return _serving.norm(h, y, weight, bias, post_weight, post_bias, gate, alpha, beta, _NORMS[kind], eps, quantize,
                         inplace)


def linear_int8(x, layer, bias=None, dtype=None):
    """x [tokens, in] times an Int8Layer (or (weight, scale[, zero])), plus
    bias (float32).  A floating x is quantized by token first; the result has
    ``dtype``, by default x's (bfloat16 for Int8Tokens)."""
    return _serving.linear(x, layer, bias, dtype)


def gated_int8(x, gate, up, act="silu", dtype=None):
    """act(x gate^T) * (x up^T) in one kernel; x, gate, up and dtype as in
    linear_int8, act one of "silu", "gelu", "gelu_tanh"."""
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return _serving.gated(x, gate, up, _ACTS[act], dtype)


def mlp_int8(h, y, weight, gate, up, down, act="silu", **norm):
    """The MLP half of a solved decoder block: (h', z) with h' the residual
    stream after the attention output y and z = down(act(gate x) * up x), x
    the pre-norm of h'.  ``norm`` takes norm_tokens' keywords.  Feed (h', z)
    to the next block's norm_tokens.  Refused layers leave h as it was."""
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    if norm.get("inplace"):     # the products' own checks come when h is overwritten
        d = h.shape[-1]
        _, _, inter, _ = _c_pair(gate, up, d, h.device, act)
        _c_layer(down, inter, h.device, "down")
        for name, layer, in_ in (("gate", gate, d), ("up", up, d), ("down", down, inter)):
            w = layer[0]
            if w.data_ptr() % 16 or (w.shape[0] > 1 and (w.stride(0) % 16 or w.stride(0) < in_)):
                raise ValueError(f"{name}.weight must have rows on 16-byte boundaries")
            if not 1 <= in_ <= 32768 or w.shape[0] > 65535:
                raise ValueError(f"{name}: {w.shape[0]} x {in_} exceeds 65535 x 32768")
    h, x = norm_tokens(h, y, weight, quantize=True, **norm)
    a = gated_int8(x, gate, up, act, dtype=weight.dtype)
    return h, linear_int8(a, down)
