"""The 8-bit serving calls against plain float64 forms, at the sizes, types
and layouts where they can go wrong."""
import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _rng(*seed):
    return np.random.default_rng([17, *seed])


def _values(rng, tokens, d, dtype, spread=1.0):
    """Normal activations with lognormal scales of the channels, on the CPU."""
    x = rng.standard_normal((tokens, d)) * np.exp(spread * rng.standard_normal(d))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def _within(got, want, tol, what=""):
    got = got.detach().cpu().double().numpy()
    off = np.abs(got - want)
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(off / tol)), np.argwhere(bad)[:3].tolist())


def _padded(rows, cols, dtype, pad, fill=7.0):
    buf = torch.full((rows + 2, cols + pad), fill, dtype=dtype, device="cuda")
    return buf, buf[1:rows + 1, :cols]


def _untouched(buf, rows, cols, fill=7.0):
    assert bool((buf[0] == fill).all()) and bool((buf[rows + 1] == fill).all())
    assert bool((buf[:, cols:] == fill).all())


# -------------------------------------------------------------- quantize_tokens
@pytest.mark.parametrize("tokens,d,dtype,pad", [
    (1, 1, F32, 0), (1, 4096, BF16, 0), (3, 7, F16, 0), (5, 512, F16, 0), (9, 513, BF16, 3), (2, 1000, F32, 1),
    (33, 4096, F16, 8), (4, 11008, F16, 0), (2, 16384, BF16, 0), (3, 16385, F32, 0), (2, 32768, F32, 0),
    (1001, 77, BF16, 0), (6, 32767, F16, 0),
    # many rows: the streaming kernel, its ring going round, and what it leaves to the other
    (3100, 4096, BF16, 0), (3100, 4001, F16, 0), (12000, 1025, BF16, 3), (601, 8192, F32, 0), (700, 9001, F32, 0),
    (3001, 1024, BF16, 8), (1500, 4096, F32, 4), (2000, 11008, F16, 0), (700, 32768, F32, 0), (900, 1032, F16, 1),
    (40000, 512, BF16, 0), (1300, 1025, F16, 0), (700, 4001, BF16, 0), (601, 11007, F32, 0), (800, 2000, BF16, 3),
    (3, 32768, F16, 3), (3, 16383, BF16, 0), (2500, 509, F16, 0), (2500, 254, BF16, 1), (900, 32765, F16, 0),
])
def test_quantize_tokens_is_the_definition(lib, tokens, d, dtype, pad):
    x = _values(_rng(1, tokens, d), tokens, d, dtype)
    buf = torch.zeros((tokens, d + pad), dtype=dtype, device="cuda")
    buf[:, :d] = x
    rows = torch.full((tokens, (d + 15) // 16 * 16 + 16), 99, dtype=torch.int8, device="cuda")
    scale = torch.empty(tokens, device="cuda")
    total = torch.empty(tokens, dtype=torch.int32, device="cuda")
    lib.gptq_quantize_tokens(buf[:, :d], rows[:, :d], scale, total)
    q, s = R.quantize(x.float().numpy())
    assert np.array_equal(rows[:, :d].cpu().numpy(), q)
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(total.cpu().numpy(), q.sum(1, dtype=np.int64))
    assert bool((rows[:, d:] == 99).all())


def test_quantize_tokens_odd_rows(lib):
    """Zero rows, NaN, infinities, halfway cases, denormal scales: each stays
    inside its own row."""
    d = 300
    x = _rng(2).standard_normal((10, d)).astype(np.float32)
    x[0] = 0
    x[1, 17] = np.nan
    x[2, 299] = np.inf
    x[3, 0] = -np.inf
    x[4] = np.arange(d) % 255 - 127          # scale exactly 1
    x[5] = (np.arange(d) % 253 - 126) + 0.5  # halfway between codes
    x[5, 0] = 127
    x[6] *= 1e-40                            # denormal
    x[7] = 0
    x[7, 5] = 2.0 ** -149                    # scale rounds to zero
    x[8] *= 1e37
    x[9, 3] = 3e38
    t = lib.quantize_tokens(torch.from_numpy(x).cuda())
    q, s = R.quantize(x)
    assert np.array_equal(t.q.cpu().numpy(), q)
    assert np.array_equal(t.scale.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(t.sum.cpu().numpy(), q.sum(1, dtype=np.int64))


# -------------------------------------------------------------------- products
SIZES = [  # tokens, in, out
    (1, 1, 1), (1, 16, 5), (1, 4096, 4096), (2, 100, 127), (3, 129, 300), (4, 11008, 260), (5, 1000, 128),
    (8, 4096, 129), (15, 777, 64), (16, 128, 4096), (17, 256, 1), (31, 3000, 513), (64, 4096, 1030), (100, 2000, 2731),
    (127, 127, 127), (128, 1024, 256), (129, 640, 384), (200, 4096, 255), (300, 100, 900), (513, 2048, 2049),
    (1000, 300, 520), (2050, 1152, 1024), (7, 32768, 40), (300, 32767, 130),
    (20, 1, 40), (600, 5, 300), (2, 17, 3), (1, 12288, 300), (2, 12287, 149), (2, 12289, 33), (1, 32768, 9), (1, 15, 1000),
    (2, 15, 149), (400, 8192, 2048), (130, 4096, 1024), (3, 2000, 11008),
]


@pytest.mark.parametrize("tokens,in_,out", SIZES)
def test_linear_sizes(lib, tokens, in_, out):
    rng = _rng(3, tokens, in_, out)
    zero, dtype = bool((tokens + out) & 1), (F16, BF16, F32)[(tokens + in_) % 3]
    layer = R.random_layer(rng, out, in_, zero)
    bias = rng.standard_normal(out).astype(np.float32) if out & 1 else None
    x = _values(rng, tokens, in_, BF16)
    buf, Y = _padded(tokens, out, dtype, 5 if in_ & 1 else 16)
    xt = lib.quantize_tokens(x.cuda())
    lib.gptq_matmul_int8(xt, R.on_device(lib, layer), Y, None if bias is None else torch.from_numpy(bias).cuda())
    q, s = R.quantize(x.float().numpy())
    p = R.product(q, s, layer)
    _within(Y, p + (0 if bias is None else bias), R.linear_tol(p, bias, dtype))
    _untouched(buf, tokens, out)
    lib.gptq_int8_status()


@pytest.mark.parametrize("tokens,in_,out", SIZES)
def test_gated_sizes(lib, tokens, in_, out):
    rng = _rng(4, tokens, in_, out)
    kind, dtype = ("silu", "gelu", "gelu_tanh")[tokens % 3], (F16, BF16, F32)[(tokens + out) % 3]
    gate, up = R.random_layer(rng, out, in_, bool(in_ & 1)), R.random_layer(rng, out, in_, bool(out & 1))
    # gate values of a few units, where the activations bend
    gate = (gate[0], (gate[1] * 2e-2 / np.sqrt(in_)).astype(np.float32), gate[2])
    up = (up[0], (up[1] * 2e-2 / np.sqrt(in_)).astype(np.float32), up[2])
    x = _values(rng, tokens, in_, F16)
    buf, Y = _padded(tokens, out, dtype, 5 if in_ & 1 else 16)
    xt = lib.quantize_tokens(x.cuda())
    lib.gptq_matmul_int8_gated(xt, R.on_device(lib, gate), R.on_device(lib, up), Y, kind)
    q, s = R.quantize(x.float().numpy())
    y, tol = R.gated(q, s, gate, up, kind, dtype)
    _within(Y, y, tol, kind)
    _untouched(buf, tokens, out)
    lib.gptq_int8_status()


@pytest.mark.parametrize("tokens", [1, 6, 20, 140, 600])
def test_extreme_codes_do_not_overflow(lib, tokens):
    """The largest sums the limits allow: every code at its bound, in 32768."""
    in_, out = 32768, 136
    q = np.full((tokens, in_), -128, np.int8)
    w = np.full((out, in_), -128, np.int8)
    z = np.full(out, 255, np.int32)
    layer = (w, np.full(out, 1e-6, np.float32), z)
    x = lib.Int8Tokens(torch.from_numpy(q).cuda(), torch.full((tokens,), 0.5, device="cuda"),
                       torch.full((tokens,), -128 * in_, dtype=torch.int32, device="cuda"))
    got = lib.linear_int8(x, R.on_device(lib, layer), dtype=F32)
    p = R.product(q, np.full(tokens, 0.5, np.float32), layer)
    assert np.isclose(p[0, 0], (128 * 128 + 255 * 128) * 32768 * 0.5 * np.float64(np.float32(1e-6)))
    _within(got, p, R.linear_tol(p, None, F32))


@pytest.mark.parametrize("tokens", [1, 4, 30, 200, 700])
def test_a_bad_token_spoils_its_own_row_only(lib, tokens):
    rng = _rng(5, tokens)
    x = _values(rng, tokens, 300, F32)
    row = tokens // 2
    x[row, 12] = float("nan")
    layer, up = R.random_layer(rng, 140, 300), R.random_layer(rng, 140, 300)
    for y in (lib.linear_int8(x.cuda(), R.on_device(lib, layer)),
              lib.gated_int8(x.cuda(), R.on_device(lib, layer), R.on_device(lib, up))):
        nan = torch.isnan(y).cpu()
        assert bool(nan[row].all()) and int(nan.sum()) == 140


def test_no_tokens_and_no_channels(lib):
    layer = R.on_device(lib, R.random_layer(_rng(6), 8, 32))
    assert lib.linear_int8(torch.empty(0, 32, dtype=BF16, device="cuda"), layer).shape == (0, 8)
    none = lib.Int8Layer(layer.weight[:0], layer.scale[:0])
    assert lib.linear_int8(torch.ones(3, 32, dtype=BF16, device="cuda"), none).shape == (3, 0)
    h, x = lib.norm_tokens(torch.empty(0, 32, device="cuda"), torch.empty(0, 32, device="cuda"),
                           torch.ones(32, device="cuda"), quantize=True)
    assert h.shape == (0, 32) and x.q.shape == (0, 32)


def test_strided_operands(lib):
    """Columns of wider buffers as x, weight and Y; one row of a matrix."""
    rng = _rng(7)
    layer = R.random_layer(rng, 96, 160)
    big = torch.zeros(96, 512, dtype=torch.int8, device="cuda")
    big[:, 64:224] = torch.from_numpy(layer[0])
    x = _values(rng, 40, 160, BF16)
    wide = torch.full((40, 333), float("nan"), dtype=BF16, device="cuda")
    wide[:, 5:165] = x
    dl = lib.Int8Layer(big[:, 64:224], torch.from_numpy(layer[1]).cuda())
    for rows in (slice(0, 40), slice(11, 12)):
        q, s = R.quantize(x[rows].float().numpy())
        p = R.product(q, s, layer)
        _within(lib.linear_int8(wide[rows, 5:165], dl), p, R.linear_tol(p, None, BF16))


@pytest.mark.parametrize("tokens,in_,out", [(2, 64, 100), (40, 96, 300), (300, 256, 520), (700, 384, 1000), (1000, 128, 513)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,first", [(16, 0), (24, 8), (7, 3), (32, 16)])
def test_results_into_wider_buffers(lib, tokens, in_, out, dtype, pad, first):
    """Y's rows on 32-byte, 16-byte and no boundaries; what lies around them is
    left alone."""
    rng = _rng(tokens, out, pad)
    layer = R.random_layer(rng, out, in_)
    dl = lib.Int8Layer(*(torch.from_numpy(a).cuda() for a in layer[:2]))
    x = _values(rng, tokens, in_, BF16)
    q, s = R.quantize(x.float().numpy())
    t = lib.quantize_tokens(x.cuda())
    ld = (out + 15) // 16 * 16 + pad + first
    for gated in (False, True):
        buf = torch.full((tokens + 2, ld), 7.0, dtype=dtype, device="cuda")
        Y = buf[1:-1, first:first + out]
        if gated:
            lib.gptq_matmul_int8_gated(t, dl, dl, Y)
            want = lib.gated_int8(t, dl, dl, dtype=dtype)
        else:
            lib.gptq_matmul_int8(t, dl, Y)
            want = lib.linear_int8(t, dl, dtype=dtype)
            p = R.product(q, s, layer)
            _within(Y, p, R.linear_tol(p, None, dtype))
        assert torch.equal(Y, want)
        Y.fill_(7.0)
        assert bool((buf == 7.0).all())


def test_offsets_beyond_32_bits(lib):
    """70000 tokens of 32768: the codes' last rows lie past 2^31 bytes, the
    result's past 2^32."""
    T, in_, out = 70000, 32768, 40000
    layer = R.random_layer(_rng(8), out, 32)
    w = torch.zeros(out, in_, dtype=torch.int8, device="cuda")
    w[:, -32:] = torch.from_numpy(layer[0])
    q = torch.zeros(T, in_, dtype=torch.int8, device="cuda")
    tail = np.random.default_rng(9).integers(-127, 128, (T, 32)).astype(np.int8)
    q[:, -32:] = torch.from_numpy(tail)
    x = lib.Int8Tokens(q, torch.full((T,), 0.25, device="cuda"), q.sum(1, dtype=torch.int32))
    y = lib.linear_int8(x, lib.Int8Layer(w, torch.from_numpy(layer[1]).cuda()), dtype=F16)
    for rows in (slice(0, 40), slice(T // 2, T // 2 + 40), slice(T - 40, T)):
        p = R.product(tail[rows], np.full(40, 0.25, np.float32), layer)
        _within(y[rows], p, R.linear_tol(p, None, F16))


# ----------------------------------------------------------------------- norms
NORMS = [  # tokens, d, type, residual type, kind, post, gate, alpha, beta, pad
    (1, 1, F32, F32, "rms", False, None, 1.0, 1.0, 0), (1, 4096, BF16, BF16, "rms", False, None, 1.0, 1.0, 0),
    (5, 77, F16, F16, "layer", True, "token", 0.7, 0.5, 0), (64, 512, BF16, F32, "rms", True, "channel", 1.0, 0.25, 8),
    (33, 513, F16, F32, "layer", False, "channel", 1.0, 1.0, 3), (7, 4096, F16, F16, "layer", True, None, 1.0, 1.0, 0),
    (9, 11008, BF16, F32, "layer", True, "token", 0.7, 1.0, 0), (3, 16384, F32, F32, "rms", True, "token", 1.0, 1.0, 0),
    (2, 16392, BF16, BF16, "layer", True, "channel", 1.0, -1.0, 0), (2, 32768, F32, F32, "layer", True, "token", 1, 1, 0),
    # many rows: the streaming kernel's rings go round, with and without a gate for each token, and with a tail
    (1500, 512, BF16, BF16, "rms", True, "channel", 1.0, 0.5, 0), (5000, 264, F16, F32, "layer", True, "token", 1, 1, 8),
    (1203, 11008, F16, F32, "layer", True, "token", 0.7, 1.0, 0), (700, 16384, BF16, BF16, "rms", False, None, 1, 1, 0),
    (601, 32768, BF16, F32, "rms", True, "channel", 1, 1, 0), (999, 4096, F32, F32, "rms", True, "token", 1, 1, 0),
    (2000, 4100, BF16, BF16, "rms", True, "channel", 1, 1, 0), (700, 4001, BF16, BF16, "layer", True, "token", 1, 1, 0),
    (650, 9001, BF16, BF16, "layer", True, "token", 1, 1, 0), (700, 12289, F16, F32, "layer", True, None, 1, 1, 0),
    (601, 8200, F32, F32, "rms", True, "token", 1, 1, 0), (640, 9003, F16, F16, "rms", True, "channel", 1, 1, 5),
    (600, 14000, F16, F16, "layer", True, "token", 1, 1, 0), (610, 8193, F32, F32, "layer", True, "channel", 1, 1, 0),
    (601, 11007, F16, F32, "rms", True, "channel", 0.7, 1, 0), (650, 1031, F32, F32, "layer", False, "token", 1, 1, 1),
    (600, 16383, BF16, F32, "rms", False, None, 1, 1, 0), (3, 32768, BF16, F32, "rms", True, "token", 1, 1, 3),
    (3, 16380, F16, F16, "layer", True, None, 1, 1, 1), (4, 8190, F16, F16, "rms", True, "channel", 1, 1, 1),
    (2500, 249, BF16, BF16, "rms", True, "channel", 1, 1, 0), (2500, 511, F16, F32, "layer", True, "token", 1, 1, 0),
 (640, 2056, F16, F16, "rms", True, "token", 1, 1, 5),
    (1001, 300, F16, F32, "rms", True, "channel", 1.0, 1.0, 1), (3, 32767, F16, F16, "rms", False, "token", 0.0, 1.0, 0),
]


@pytest.mark.parametrize("tokens,d,dtype,htype,kind,post,gate,alpha,beta,pad", NORMS)
@pytest.mark.parametrize("quantize", [False, True])
def test_norm(lib, tokens, d, dtype, htype, kind, post, gate, alpha, beta, pad, quantize):
    rng = _rng(10, tokens, d)
    layer = kind == "layer"
    y, h = _values(rng, tokens, d, dtype) + (3 if layer else 0), _values(rng, tokens, d, htype, 0.3)
    y = y.to(dtype)
    vec = lambda m: torch.from_numpy((m + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(dtype)  # noqa: E731
    weight, bias = vec(1), vec(0) if layer else None
    pw, pb = (vec(1) if post else None), (vec(0) if post and layer else None)
    g = None if gate is None else (vec(0.5) if gate == "channel" else _values(rng, tokens, d, dtype, 0.1))
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    wide = lambda t: torch.cat([t, torch.full((t.shape[0], pad), float("nan"), dtype=t.dtype)], 1).cuda()[:, :d]  # noqa: E731
    h1, x = lib.norm_tokens(wide(h), wide(y), cuda(weight), bias=cuda(bias), post_weight=cuda(pw), post_bias=cuda(pb),
                            gate=cuda(g), alpha=alpha, beta=beta, kind=kind, eps=1e-5, quantize=quantize)
    f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    wh, dh, wx, dx = R.norm(f(h), f(y), f(weight), f(bias), f(pw), f(pb), f(g), alpha, beta, kind, float(np.float32(1e-5)))
    _within(h1, wh, dh * 1.01 + R.U[htype] * np.abs(wh) * 1.01 + R.FLOOR[htype], "h")
    if not quantize:
        _within(x, wx, dx * 1.01 + R.U[dtype] * np.abs(wx) * 1.01 + R.FLOOR[dtype], "x")
        return
    q, scale = x.q.cpu().numpy().astype(np.float64), x.scale.cpu().numpy().astype(np.float64)
    assert np.array_equal(x.sum.cpu().numpy(), q.sum(1))
    top, at = np.abs(wx).max(1), dx.max(1)
    assert np.all(np.abs(scale * 127 - top) <= at * 1.01 + 2 * R.U32 * top)
    # a code is the nearest one to a value within dx of the exact one
    assert np.all(np.abs(q * scale[:, None] - wx) <= (0.5 * (1 + 1e-4) * scale)[:, None] + dx * 1.01)


def test_norm_first_block_and_in_place(lib):
    rng = _rng(11)
    a, b = (_values(rng, 20, 264, BF16).cuda() for _ in range(2))
    w = _values(rng, 1, 264, BF16)[0].cuda()
    same, x = lib.norm_tokens(a, None, w)
    assert same is a
    _, _, wx, dx = R.norm(a.double().cpu().numpy(), None, w.double().cpu().numpy(), None, None, None, None, 1, 1, "rms",
                          float(np.float32(1e-6)))
    _within(x, wx, dx * 1.01 + R.U[BF16] * np.abs(wx) * 1.01 + R.FLOOR[BF16])
    want, wx = lib.norm_tokens(a, b, w)
    c = a.clone()
    got, gx = lib.norm_tokens(c, b, w, inplace=True)
    assert got is c and torch.equal(got, want) and torch.equal(gx, wx)


@pytest.mark.parametrize("tokens,d,offset", [(7, 333, 1), (5, 40, 3), (700, 1024, 1), (601, 4001, 5), (650, 2051, 7),
                                             (601, 9001, 5), (620, 8203, 7), (3000, 4099, 1)])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_rows_that_start_anywhere(lib, tokens, d, offset, dtype):
    """Tensors that begin and end inside a 16-byte unit, their surroundings
    NaN, and outputs that do: first and last rows whole, nothing else written.
    In place as well."""
    rng = _rng(20, tokens, d)

    def inside(t=None):
        buf = torch.full((tokens * d + 32,), float("nan"), dtype=dtype, device="cuda")
        view = buf[offset:offset + tokens * d].view(tokens, d)
        if t is not None:
            view.copy_(t)
        return buf, view

    h, y = _values(rng, tokens, d, dtype), _values(rng, tokens, d, dtype)
    w = _values(rng, 1, d, dtype, 0.1)[0]
    f = lambda t: t.double().numpy()  # noqa: E731
    wh, dh, wx, dx = R.norm(f(h), f(y), f(w), None, f(w), None, None, 1, 1, "rms", float(np.float32(1e-6)))
    (_, hv), (_, yv), (hb, ho), (xb, xo) = inside(h), inside(y), inside(), inside()
    wbuf = torch.full((d + 16,), float("nan"), dtype=dtype, device="cuda")
    wv = wbuf[offset:offset + d]
    wv.copy_(w)
    lib.gptq_norm_tokens(hv, yv, wv, post_weight=wv, h_out=ho, x=xo)
    _within(ho, wh, dh * 1.01 + R.U[dtype] * np.abs(wh) * 1.01 + R.FLOOR[dtype], "h")
    _within(xo, wx, dx * 1.01 + R.U[dtype] * np.abs(wx) * 1.01 + R.FLOOR[dtype], "x")
    for b in (hb, xb):
        assert bool(torch.isnan(b[:offset]).all()) and bool(torch.isnan(b[offset + tokens * d:]).all())
    want, x1 = ho.clone(), xo.clone()
    lib.gptq_norm_tokens(hv, yv, wv, post_weight=wv, h_out=hv, x=xo)
    assert torch.equal(hv, want) and torch.equal(xo, x1)
    t = lib.quantize_tokens(yv)
    q, scale = R.quantize(y.float().numpy())
    assert np.array_equal(t.q.cpu().numpy(), q) and np.array_equal(t.scale.cpu().numpy(), scale)
    assert np.array_equal(t.sum.cpu().numpy(), q.sum(1, dtype=np.int64))
    layer = R.random_layer(rng, 40, d)
    p = R.product(q, scale, layer)
    _within(lib.linear_int8(yv, R.on_device(lib, layer), dtype=F32), p, R.linear_tol(p, None, F32))
    lib.gptq_int8_status()


def test_norm_all_outputs_at_once(lib):
    """h_out, x and the tokens of one call equal those of calls for each."""
    rng = _rng(12)
    h, y, w = _values(rng, 30, 1000, F32).cuda(), _values(rng, 30, 1000, F16).cuda(), _values(rng, 1, 1000, F16)[0].cuda()
    h1, x1 = lib.norm_tokens(h, y, w)
    _, t1 = lib.norm_tokens(h, y, w, quantize=True)
    h2, x2 = torch.empty_like(h), torch.empty_like(y)
    t2 = lib.Int8Tokens(torch.empty(30, 1008, dtype=torch.int8, device="cuda")[:, :1000], torch.empty_like(t1.scale),
                        torch.empty_like(t1.sum))
    lib.gptq_norm_tokens(h, y, w, h_out=h2, x=x2, tokens=t2)
    assert torch.equal(h1, h2) and torch.equal(x1, x2)
    assert all(torch.equal(a, b) for a, b in zip(t1, t2))


# ------------------------------------------------------------- a solved layer
@pytest.mark.parametrize("bits,sym", [(8, True), (8, False), (4, False), (3, True), (2, False)])
def test_int8_layer_of_a_solved_layer(lib, bits, sym):
    """The layout stands for the weights gptq_dequantize_layer gives, and a
    product with it for the product with those."""
    rng = _rng(13, bits)
    W = torch.from_numpy((0.02 * rng.standard_normal((70, 288))).astype(np.float32)).cuda()
    X = _values(rng, 900, 288, F16)
    r = lib.solve_layer(W, X.t().contiguous().cuda(), dict(bits=bits, group_size=-1, sym=sym))
    layer = lib.int8_layer(r, bits)
    deq = torch.empty(70, 288, device="cuda")
    lib.gptq_dequantize_layer(r["qweight"], r["scales"], r["zeros"], r["g_idx"], bits, deq)
    z = torch.zeros(70, dtype=torch.int32, device="cuda") if layer.zero is None else layer.zero
    assert torch.equal(layer.scale[:, None] * (layer.weight.int() - z[:, None]).float(), deq)
    if bits == 8 and sym:
        assert int(layer.zero.abs().max()) == 0
    y = lib.linear_int8(X.cuda(), layer, dtype=F32)
    q, s = R.quantize(X.float().numpy())
    want = (q * s.astype(np.float64)[:, None]) @ deq.double().cpu().numpy().T
    p = R.product(q, s, (layer.weight.cpu().numpy(), layer.scale.cpu().numpy(), z.cpu().numpy()))
    _within(y, p, R.linear_tol(p, None, F32))
    assert np.abs(want - p).max() <= 1e-6 * np.abs(p).max()


def _mlp_reference(h, y, w, gate, up, down):
    f = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    h1, _, x, _ = R.norm(f(h), f(y), f(w), None, None, None, None, 1, 1, "rms", float(np.float32(1e-6)))
    q, s = R.quantize(x.astype(np.float32))
    a, _ = R.gated(q, s, gate, up, "silu", w.dtype)
    q, s = R.quantize(torch.from_numpy(a.astype(np.float32)).to(w.dtype).float().numpy())
    return h1, R.product(q, s, down)


@pytest.mark.parametrize("tokens", [1, 5, 40, 333])
def test_mlp_of_a_solved_block(lib, tokens):
    """Two blocks' MLP halves in a row on layers solve_block quantized.  A code
    may differ by one where a value lies at the border of two, so the run is
    compared in norm: one code in the 8-bit grid is at most 1/127 of a token's
    largest value, and the output's own rounding is 2^-8."""
    rng = _rng(14)
    d, inter = 256, 704
    weights = {n: torch.from_numpy((0.05 * rng.standard_normal(s)).astype(np.float32)).cuda()
               for n, s in (("gate", (inter, d)), ("up", (inter, d)), ("down", (d, inter)))}
    acts = {"mlp": _values(rng, 1024, d, F16, 0.3).t().contiguous().cuda(),
            "down": _values(rng, 1024, inter, F16, 0.3).t().contiguous().cuda()}
    res = lib.solve_block([("gate", weights["gate"], "mlp"), ("up", weights["up"], "mlp"),
                           ("down", weights["down"], "down")], acts, dict(bits=8, sym=True, group_size=-1))
    layers = {n: lib.int8_layer(res[n], 8) for n in weights}
    host = {n: (l.weight.cpu().numpy(), l.scale.cpu().numpy(), l.zero.cpu().numpy()) for n, l in layers.items()}
    h, y = _values(rng, tokens, d, BF16, 0.3).cuda(), _values(rng, tokens, d, BF16, 0.3).cuda()
    w = (1 + 0.1 * torch.randn(d)).to(BF16).cuda()
    for _ in range(2):
        wh, wz = _mlp_reference(h, y, w, host["gate"], host["up"], host["down"])
        h1, z = lib.mlp_int8(h, y, w, layers["gate"], layers["up"], layers["down"])
        _within(h1, wh, 1.02 * R.U[BF16] * np.abs(wh) + 1e-6)
        off = np.linalg.norm(z.double().cpu().numpy() - wz) / np.linalg.norm(wz)
        assert off < 2.0 ** -8 + 1 / 127, off
        h, y = h1, z
    lib.gptq_int8_status()


# ------------------------------------------------------- streams, graphs, reuse
def _case(lib, tokens, seed):
    rng = _rng(15, seed)
    d, out = 520, 264
    h, y = _values(rng, tokens, d, BF16).cuda(), _values(rng, tokens, d, BF16).cuda()
    w = _values(rng, 1, d, BF16, 0.1)[0].cuda()
    gate, up = (R.on_device(lib, R.random_layer(rng, out, d, True)) for _ in range(2))
    down = R.on_device(lib, R.random_layer(rng, d, out))
    scale = 1e-3
    gate, up = gate._replace(scale=gate.scale * scale), up._replace(scale=up.scale * scale)
    return h, y, w, gate, up, down


@pytest.mark.parametrize("tokens", [1, 3, 48, 400])
def test_repeated_and_concurrent_calls_give_the_same_bits(lib, tokens):
    cases = [_case(lib, tokens, s) for s in range(3)]
    want = [lib.mlp_int8(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(4):
        for c, s, g in zip(cases, streams, got):
            with torch.cuda.stream(s):
                g.append(lib.mlp_int8(*c))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for r in g for a, b in zip(r, w))


@pytest.mark.parametrize("tokens", [1, 3, 48, 400])
def test_captured_runs_replay_on_new_inputs(lib, tokens):
    """Two captured graphs replayed in turn and at the same time."""
    a, b = _case(lib, tokens, 1), _case(lib, tokens, 2)
    lib.mlp_int8(*a)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lib.mlp_int8(*c))
        graphs.append(g)
    for n in range(3):
        for c in (a, b):
            c[0].copy_(_values(_rng(16, n), tokens, 520, BF16))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for c, o in zip((a, b), outs):
            want = lib.mlp_int8(*c)
            assert all(torch.equal(x, y) for x, y in zip(o, want))


def test_the_first_call_of_a_process_may_be_captured():
    """No set-up that a capture forbids: in a process of its own."""
    import subprocess
    import sys
    code = """
import torch, post_weight_quantization_13_b200 as g
x = torch.randn(20, 512, device='cuda', dtype=torch.bfloat16)
w = torch.ones(512, device='cuda', dtype=torch.bfloat16)
layer = (torch.randint(-127, 127, (256, 512), dtype=torch.int8, device='cuda'), torch.ones(256, device='cuda'))
down = (torch.randint(-127, 127, (512, 256), dtype=torch.int8, device='cuda'), torch.ones(512, device='cuda'))
run = lambda: g.mlp_int8(x, x, w, layer, layer, down)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(y, run()))
"""
    root = __import__("os").path.dirname(__import__("os").path.dirname(__import__("os").path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_calls_from_several_threads(lib):
    """Host threads on streams of their own: the same bits, and each thread's
    errors its own."""
    import threading
    cases = [_case(lib, t, s) for s, t in enumerate((1, 30, 300, 900))]
    want = [lib.mlp_int8(*c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(c, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    r = lib.mlp_int8(*c)
                    try:
                        lib.linear_int8(c[0][:1].expand(5, c[0].shape[1]), c[3])
                        bad.append("no error")
                    except lib.GptqError as e:
                        if e.status != 1:
                            bad.append(e)
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(r, w)):
                bad.append("bits")
        except Exception as e:      # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=work, args=cw) for cw in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_the_stream_argument_orders_the_work(lib):
    rng = _rng(18)
    layer = R.random_layer(rng, 200, 640)
    dl = R.on_device(lib, layer)
    x = _values(rng, 50, 640, F16)
    q, s = R.quantize(x.float().numpy())
    p = R.product(q, s, layer)
    side = torch.cuda.Stream()
    xd = torch.zeros(50, 640, dtype=F16, device="cuda")
    t = lib.Int8Tokens(torch.empty(50, 640, dtype=torch.int8, device="cuda"), torch.empty(50, device="cuda"),
                       torch.empty(50, dtype=torch.int32, device="cuda"))
    Y = torch.empty(50, 200, dtype=F32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        xd.copy_(x.cuda())
    lib.gptq_quantize_tokens(xd, *t, stream=side)
    lib.gptq_matmul_int8(t, dl, Y, stream=side)
    side.synchronize()
    _within(Y, p, R.linear_tol(p, None, F32))


def test_bound_arguments_are_checked(lib):
    layer = R.on_device(lib, R.random_layer(_rng(19), 32, 64))
    x = torch.ones(4, 64, dtype=BF16, device="cuda")
    with pytest.raises(lib.GptqError) as e:        # a row stride that is no multiple of 16
        t = lib.Int8Tokens(torch.zeros(4, 72, dtype=torch.int8, device="cuda")[:, :64], torch.ones(4, device="cuda"),
                           torch.zeros(4, dtype=torch.int32, device="cuda"))
        lib.linear_int8(t, layer)
    assert e.value.status == 1
    with pytest.raises(lib.GptqError):             # overlapping rows
        lib.linear_int8(x[:1].expand(4, 64), layer)
    with pytest.raises(ValueError):
        lib.linear_int8(x[:, :48], layer)
    with pytest.raises(ValueError):
        lib.linear_int8(x, layer, bias=torch.zeros(32, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        lib.linear_int8(x, layer, bias=torch.zeros(32))
