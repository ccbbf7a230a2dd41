"""The 8-bit serving calls refuse bad arguments on the host, before anything
is launched: through the C ABI with addresses that are never read, and
through the Python functions with tensors that no call accepts."""
import pytest
import torch

INVALID, UNSUPPORTED = 1, 7


@pytest.fixture(scope="module")
def g():
    import __graft_entry__
    __graft_entry__.build()
    import post_weight_quantization_13_b200 as m
    return m


@pytest.fixture(scope="module")
def S(g):
    from post_weight_quantization_13_b200 import serving
    return serving


A = 4096            # an aligned address that is never read


def _tokens(S, **kw):
    return S._Tokens(*{"q": A, "ldq": 64, "scale": A, "sum": A, **kw}.values())


def _layer(S, **kw):
    return S._Layer(*{"w": A, "ldw": 64, "scale": A, "zero": None, **kw}.values())


def _matmul(g, x, w, tokens=4, in_=64, out=32, bias=None, Y=A, yt=1, ldy=32):
    return g.lib.gptq_matmul_int8(x, tokens, in_, w, out, bias, Y, yt, ldy, None)


def _gated(g, x, w, u, tokens=4, in_=64, out=32, act=0, Y=A, yt=1, ldy=32):
    return g.lib.gptq_matmul_int8_gated(x, tokens, in_, w, u, out, act, Y, yt, ldy, None)


@pytest.mark.parametrize("call,status", [
    (dict(tokens=-1), INVALID), (dict(in_=0), INVALID), (dict(out=-1), INVALID),
    (dict(tokens=(1 << 26) + 1), UNSUPPORTED), (dict(in_=32769), UNSUPPORTED), (dict(out=65536), UNSUPPORTED),
    (dict(yt=3), INVALID), (dict(Y=None), INVALID), (dict(Y=A + 1), INVALID), (dict(ldy=31), INVALID),
    (dict(in_=65), INVALID),                                      # ldq, ldw < in
])
def test_products_refuse_sizes_and_outputs(g, S, call, status):
    assert _matmul(g, _tokens(S), _layer(S), **call) == status
    assert g.gptq_last_error()
    assert _gated(g, _tokens(S), _layer(S), _layer(S), **call) == status


@pytest.mark.parametrize("bad", [dict(q=None), dict(q=A + 8), dict(ldq=48), dict(ldq=72), dict(scale=None),
                                 dict(scale=A + 2), dict(sum=None), dict(sum=A + 1)])
def test_products_refuse_tokens(g, S, bad):
    assert _matmul(g, _tokens(S, **bad), _layer(S)) == INVALID
    assert _gated(g, _tokens(S, **bad), _layer(S), _layer(S)) == INVALID
    assert _matmul(g, None, _layer(S)) == INVALID


@pytest.mark.parametrize("bad", [dict(w=None), dict(w=A + 4), dict(ldw=63), dict(ldw=40), dict(scale=None),
                                 dict(scale=A + 1), dict(zero=A + 2)])
def test_products_refuse_layers(g, S, bad):
    assert _matmul(g, _tokens(S), _layer(S, **bad)) == INVALID
    assert _gated(g, _tokens(S), _layer(S, **bad), _layer(S)) == INVALID
    assert _gated(g, _tokens(S), _layer(S), _layer(S, **bad)) == INVALID
    assert _gated(g, _tokens(S), _layer(S), None) == INVALID


def test_other_product_arguments(g, S):
    assert _matmul(g, _tokens(S), _layer(S), bias=A + 2) == INVALID
    assert _gated(g, _tokens(S), _layer(S), _layer(S), act=3) == INVALID
    # no work needs no GPU and no operands
    assert _matmul(g, None, None, tokens=0, Y=None) == 0
    assert _gated(g, None, None, None, out=0, Y=None) == 0


@pytest.mark.parametrize("call,status", [
    (dict(xt=5), INVALID), (dict(tokens=-1), INVALID), (dict(in_=0), INVALID), (dict(in_=40000), UNSUPPORTED),
    (dict(X=None), INVALID), (dict(X=A + 1), INVALID), (dict(ldx=63), INVALID), (dict(q=None), INVALID),
    (dict(q=A + 4), INVALID), (dict(ldq=72), INVALID), (dict(scale=None), INVALID), (dict(sum=None), INVALID),
])
def test_quantize_tokens_refuses(g, call, status):
    a = {"X": A, "xt": 0, "tokens": 4, "in_": 64, "ldx": 64, "q": A, "ldq": 64, "scale": A, "sum": A, **call}
    assert g.lib.gptq_quantize_tokens(*a.values(), None) == status
    assert g.gptq_last_error()


def _norm(S, **kw):
    a = S._Norm(4, 64, 1, 1, 0, 1e-6, 1.0, 1.0, A, 64, A, 64, None, None, None, 0, A, None, A, 64, A, 64, None, 0, None,
                None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(tokens=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769), UNSUPPORTED), (dict(yt=4), INVALID),
    (dict(ht=0), INVALID), (dict(kind=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(h=None), INVALID), (dict(h=A + 1), INVALID), (dict(ldh=63), INVALID), (dict(ldy=1), INVALID),
    (dict(y=None, post_weight=A), INVALID), (dict(y=None, gate=A), INVALID), (dict(post_bias=A), INVALID),
    (dict(gate=A, ldgate=5), INVALID), (dict(gate=A + 1), INVALID), (dict(weight=None), INVALID),
    (dict(weight=None, x=None, bias=A), INVALID), (dict(x=None), INVALID), (dict(x=None, weight=None, h_out=None), INVALID),
    (dict(h_out=A + 1), INVALID), (dict(ldh_out=80), INVALID), (dict(ldx=8), INVALID),
    (dict(q=A, ldq=64, scale=A, sum=None), INVALID), (dict(q=A, ldq=60, scale=A, sum=A), INVALID),
    (dict(q=A + 8, ldq=64, scale=A, sum=A), INVALID),
])
def test_norm_tokens_refuses(g, S, bad, status):
    assert g.lib.gptq_norm_tokens(_norm(S, **bad), None) == status
    assert g.gptq_last_error()


def test_norm_tokens_without_tokens_is_a_no_op(g, S):
    assert g.lib.gptq_norm_tokens(_norm(S, tokens=0, h=None), None) == 0
    assert g.lib.gptq_norm_tokens(None, None) == INVALID


@pytest.mark.parametrize("call,status", [
    (dict(bits=5), INVALID), (dict(in_=0), INVALID), (dict(out=-1), INVALID), (dict(bits=3, in_=36), UNSUPPORTED),
    (dict(qweight=None), INVALID), (dict(zeros=None), INVALID), (dict(w=A + 8), INVALID), (dict(ldw=63), INVALID),
    (dict(ldw=72), INVALID), (dict(zero=A + 1), INVALID), (dict(in_=32769 * 8), UNSUPPORTED),
])
def test_layout_int8_refuses(g, call, status):
    a = {"qweight": A, "zeros": A, "out": 8, "in_": 64, "bits": 8, "w": A, "ldw": 64, "zero": A, **call}
    assert g.lib.gptq_layout_int8(*a.values(), None) == status
    assert g.lib.gptq_layout_int8(None, None, 0, 64, 8, None, 64, None, None) == 0


def _linear(g, w, X=A, xt=1, tokens=40, in_=64, ldx=64, out=32, bias=None, Y=A, yt=1, ldy=32, ws=1 << 20,
            ws_bytes=1 << 20):
    return g.lib.gptq_linear_int8(X, xt, tokens, in_, ldx, w, out, bias, Y, yt, ldy, ws, ws_bytes, None)


def _linear_gated(g, w, u, X=A, xt=1, tokens=40, in_=64, ldx=64, out=32, act=0, Y=A, yt=1, ldy=32, ws=1 << 20,
                  ws_bytes=1 << 20):
    return g.lib.gptq_linear_int8_gated(X, xt, tokens, in_, ldx, w, u, out, act, Y, yt, ldy, ws, ws_bytes, None)


WORKSPACE = 4


@pytest.mark.parametrize("call,status", [
    (dict(tokens=-1), INVALID), (dict(in_=0), INVALID), (dict(out=-1), INVALID), (dict(in_=32769), UNSUPPORTED),
    (dict(xt=3), INVALID), (dict(yt=-1), INVALID), (dict(X=None), INVALID), (dict(X=A + 1), INVALID),
    (dict(ldx=63), INVALID), (dict(Y=None), INVALID), (dict(ldy=31), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=A + 16), WORKSPACE), (dict(ws_bytes=64 * 40), WORKSPACE), (dict(ws_bytes=0), WORKSPACE),
])
def test_linear_int8_refuses(g, S, call, status):
    assert _linear(g, _layer(S), **call) == status
    assert g.gptq_last_error()
    assert _linear_gated(g, _layer(S), _layer(S), **call) == status


def test_linear_int8_other_arguments(g, S):
    assert _linear(g, _layer(S, ldw=72)) == INVALID
    assert _linear(g, _layer(S), bias=A + 1) == INVALID
    assert _linear_gated(g, _layer(S), None) == INVALID
    assert _linear_gated(g, _layer(S), _layer(S), act=-1) == INVALID
    assert _linear(g, None, tokens=0, X=None, Y=None, ws=None, ws_bytes=0) == 0
    assert _linear_gated(g, None, None, out=0, Y=None, ws=None, ws_bytes=0) == 0


def test_linear_int8_workspace_sizes(g):
    """Codes in 16-byte rows, a scale and a sum for each token; none where one
    kernel does both; 0 for sizes no call takes."""
    size = g.gptq_linear_int8_ws_bytes
    assert size(1, 4096) == 0 and size(2, 4096) == 0
    assert size(40, 65) >= 40 * (80 + 4 + 4) and size(3, 4096) >= 3 * (4096 + 8)
    assert size(1 << 26, 32768) >= (1 << 26) * (32768 + 8)
    assert size(-1, 64) == 0 and size(4, 0) == 0 and size(4, 32769) == 0 and size((1 << 26) + 1, 64) == 0
    for t in (1, 3, 100, 5000):
        for d in (1, 15, 4096, 32768):
            assert size(t, d) % 256 == 0


# ------------------------------------------------------------ Python functions
def test_python_calls_refuse_cpu_tensors(g):
    x = torch.ones(4, 64)
    layer = g.Int8Layer(torch.zeros(8, 64, dtype=torch.int8), torch.ones(8))
    with pytest.raises(ValueError, match="CUDA device"):
        g.quantize_tokens(x)
    with pytest.raises(ValueError, match="CUDA device"):
        g.norm_tokens(x, x, torch.ones(64))
    t = g.Int8Tokens(torch.zeros(4, 64, dtype=torch.int8), torch.ones(4), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA device"):
        g.linear_int8(t, layer)
    with pytest.raises(ValueError, match="CUDA device"):
        g.gated_int8(t, layer, layer)


def test_python_calls_check_types_and_shapes(g):
    t = g.Int8Tokens(torch.zeros(4, 64, dtype=torch.int8), torch.ones(4), torch.zeros(4, dtype=torch.int32))
    layer = g.Int8Layer(torch.zeros(8, 64, dtype=torch.int8), torch.ones(8))
    for bad in (t._replace(q=t.q.float()), t._replace(scale=torch.ones(5)), t._replace(sum=torch.zeros(4)),
                t._replace(scale=torch.ones(8)[::2])):
        with pytest.raises(ValueError):
            g.linear_int8(bad, layer)
    for bad in (layer._replace(weight=layer.weight.float()), layer._replace(weight=layer.weight[:, :32]),
                layer._replace(scale=torch.ones(7)), layer._replace(zero=torch.zeros(8)),
                layer._replace(weight=torch.zeros(64, 8, dtype=torch.int8).t())):
        with pytest.raises(ValueError):
            g.linear_int8(t, bad)
        with pytest.raises(ValueError):
            g.gated_int8(t, layer, bad)
    with pytest.raises(ValueError):
        g.gated_int8(t, layer, g.Int8Layer(torch.zeros(9, 64, dtype=torch.int8), torch.ones(9)))
    with pytest.raises(ValueError):
        g.gated_int8(t, layer, layer, act="relu")
    with pytest.raises(TypeError):
        g.linear_int8(t, layer, dtype=torch.float64)
    x = torch.ones(4, 64)
    w = torch.ones(64)
    for kw in (dict(kind="batch"), dict(gate=torch.ones(4)), dict(bias=torch.ones(64, dtype=torch.float16)),
               dict(post_weight=torch.ones(63)), dict(gate=torch.ones(3, 64))):
        with pytest.raises(ValueError):
            g.norm_tokens(x, x, w, **kw)
    with pytest.raises(ValueError):
        g.norm_tokens(x, x)
    with pytest.raises(ValueError):
        g.norm_tokens(x, x.half(), w)


def test_calls_into_given_tensors_check_types_and_shapes(g):
    t = g.Int8Tokens(torch.zeros(4, 64, dtype=torch.int8), torch.ones(4), torch.zeros(4, dtype=torch.int32))
    layer = g.Int8Layer(torch.zeros(8, 64, dtype=torch.int8), torch.ones(8))
    x, Y = torch.ones(4, 64), torch.empty(4, 8)
    for call in (lambda: g.gptq_matmul_int8(t, layer, torch.empty(4, 9)),
                 lambda: g.gptq_matmul_int8(t, layer, Y, bias=torch.ones(9)),
                 lambda: g.gptq_matmul_int8_gated(t, layer, layer, Y, act="no"),
                 lambda: g.gptq_linear_int8(x[:, :63], layer, Y),
                 lambda: g.gptq_linear_int8(x.t().contiguous().t(), layer, Y),
                 lambda: g.gptq_linear_int8_gated(x, layer, layer._replace(scale=torch.ones(3)), Y),
                 lambda: g.gptq_quantize_tokens(x, t.q, torch.ones(3), t.sum),
                 lambda: g.gptq_quantize_tokens(x, t.q.int(), t.scale, t.sum),
                 lambda: g.gptq_norm_tokens(x, x, torch.ones(64), x=torch.empty(4, 63)),
                 lambda: g.gptq_norm_tokens(x, x, torch.ones(64), h_out=x.half()),
                 lambda: g.gptq_norm_tokens(x, x, torch.ones(64), tokens=t._replace(scale=torch.ones(4).half())),
                 lambda: g.gptq_layout_int8(torch.zeros(8, 16, dtype=torch.int32), torch.zeros(7, dtype=torch.int32), 8,
                                            layer.weight),
                 lambda: g.gptq_layout_int8(torch.zeros(8, 16, dtype=torch.int32),
                                            torch.zeros(16, dtype=torch.int32)[::2], 8, layer.weight),
                 lambda: g.gptq_layout_int8(torch.zeros(8, 15, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), 8,
                                            layer.weight)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        g.linear_int8(x, [layer.weight])
    with pytest.raises(TypeError):
        g.linear_int8("x", layer)
    with pytest.raises(TypeError):
        g.linear_int8(x, layer, dtype="float32")
    with pytest.raises(TypeError):
        g.quantize_tokens(x.double())


def test_int8_layer_needs_one_scale_per_channel(g):
    r = {"qweight": torch.zeros(4, 16, dtype=torch.int32), "scales": torch.ones(4, 2), "zeros": torch.zeros(4, 2)}
    with pytest.raises(ValueError, match="group_size=-1"):
        g.int8_layer(r, 8)
    with pytest.raises(ValueError, match="packed codes"):
        g.int8_layer({**r, "qweight": None}, 8)


def test_serving_names_are_public(g):
    for name in ("linear_int8", "gated_int8", "norm_tokens", "quantize_tokens", "mlp_int8", "int8_layer"):
        assert name in g.__all__ and callable(getattr(g, name))
    with pytest.raises(AttributeError):
        g.no_such_call


def test_int8_timeout_selftest_refuses_bad_limits(g):
    for limit in (0, 3 * 10 ** 9):
        assert g.lib.gptq_selftest_int8_timeout(limit, None) == INVALID
        assert "limit_ns" in g.gptq_last_error()


def test_int8_status_is_that_of_the_streams_device(g, S, monkeypatch):
    """A stream of another device than the current one: two devices that answer
    by themselves."""
    import contextlib
    import types
    current, asked = [0], []

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    def status(raw):
        asked.append((current[0], raw))
        return 0

    monkeypatch.setattr(S.torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(S.torch.cuda, "device", device)
    monkeypatch.setattr(S, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(S, "lib", types.SimpleNamespace(gptq_int8_status=status))
    g.gptq_int8_status()
    g.gptq_int8_status(types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=7))
    g.gptq_int8_status(types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=8))
    assert asked == [(0, 100), (1, 7), (0, 8)] and current == [0]


def test_mlp_refuses_before_it_overwrites_the_residual_stream(g, S, monkeypatch):
    def overwritten(*a, **k):
        raise AssertionError("the norm ran")

    monkeypatch.setattr(S, "norm_tokens", overwritten)
    h, w = torch.ones(4, 64), torch.ones(64)

    def layer(out, in_, pad=0):
        return g.Int8Layer(torch.zeros(out, in_ + pad, dtype=torch.int8)[:, :in_], torch.ones(out))

    gate, down = layer(96, 64), layer(64, 96)
    for a in ((gate, gate, down, "relu"), (layer(96, 48), gate, down, "silu"), (gate, layer(80, 64), down, "silu"),
              (gate, gate, layer(64, 80), "silu"), (gate, gate._replace(scale=torch.ones(5)), down, "silu"),
              (gate, gate, down._replace(weight=down.weight.int()), "silu"), (gate, layer(96, 64, 8), down, "gelu"),
              (gate, gate, layer(64, 96)._replace(zero=torch.zeros(64)), "silu"),
              (layer(3, 65536, 0), layer(3, 65536, 0), layer(65536, 3, 13), "silu")):
        with pytest.raises(ValueError):
            g.mlp_int8(h, h, w, *a, inplace=True)
    with pytest.raises(ValueError):
        g.mlp_int8(h, h, w, gate, gate, down, "relu")
    with pytest.raises(AssertionError, match="the norm ran"):
        g.mlp_int8(h, h, w, gate, gate, down, inplace=True)
