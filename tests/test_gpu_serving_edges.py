"""The 8-bit serving calls where sizes, values and callers meet their limits."""
import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _within(got, want, tol):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist(), float((off / tol).max()))


# ------------------------------------------------------------ one or two tokens
def _wide_layer(gen, out, in_, pad):
    """Full-range codes in rows of in_ + pad bytes, on the device."""
    w = torch.randint(-128, 128, (out, (in_ + 15) // 16 * 16 + pad), generator=gen, device="cuda", dtype=torch.int8)
    scale = torch.rand(out, generator=gen, device="cuda") * 1e-4 + 1e-5
    zero = torch.randint(-128, 128, (out,), generator=gen, device="cuda", dtype=torch.int32)
    return w[:, :in_], scale, zero


def _sums(q, layer, rows=4096):
    """The scaled product in float64 (sums of integers below 2^53: exact)."""
    w, scale, zero = layer
    total = torch.cat([q @ w[i:i + rows].double().T for i in range(0, w.shape[0], rows)], 1)
    return (total - q.sum(1, keepdim=True) * zero.double()) * scale.double()


@pytest.mark.parametrize("tokens,in_,out,pad", [
    # the widest rows with the most channels, unpadded and padded: rings that hold just a batch each
    (2, 12288, 40000, 0), (2, 12288, 65535, 0), (2, 12288, 65535, 112), (1, 12288, 65535, 96), (2, 12280, 65535, 0),
    # rings of odd numbers of slots
    (2, 11008, 4096, 0), (1, 11008, 4096, 0), (2, 8208, 5000, 0), (1, 9000, 3001, 16), (2, 4112, 20000, 0),
])
@pytest.mark.parametrize("gated", [False, True])
def test_wide_rows_and_many_channels_of_one_and_two_tokens(lib, tokens, in_, out, pad, gated):
    gen = torch.Generator("cuda").manual_seed(in_ + out + pad)
    x = torch.randn(tokens, in_, generator=gen, device="cuda").to(BF16)
    a, b = _wide_layer(gen, out, in_, pad), _wide_layer(gen, out, in_, pad)
    t = lib.quantize_tokens(x)
    q = t.q.double()
    g, u = (_sums(q, l) * t.scale.double()[:, None] for l in (a, b))
    for _ in range(5):
        if not gated:
            y = lib.linear_int8(t, a, dtype=F32)
            _within(y, g, (5 * R.U32 * g.abs()) * 1.01 + R.FLOOR[F32])
        else:
            y = lib.gated_int8(t, a, b, dtype=F32)
            # silu's relative error: see serving_ref.act_tol
            z = g.abs()
            act = g / (1 + torch.exp(-g))
            off = act.abs() * ((1 + z) * 4 * R.U32 + z * 6 * R.U32 + (6 + 1.173 * z) * 2.0 ** -23) + 2e-36
            _within(y, act * u, (off * u.abs() + 6 * R.U32 * (act * u).abs()) * 1.01 + R.FLOOR[F32])
        # and quantized on the way: the same bits
        assert torch.equal(y, lib.gated_int8(x, a, b, dtype=F32) if gated else lib.linear_int8(x, a, dtype=F32))
    lib.gptq_int8_status()


# ------------------------------------------------------------------ gelu's tail
@pytest.mark.parametrize("tokens", [1, 2, 20, 300])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gelu_keeps_its_relative_accuracy_where_it_vanishes(lib, tokens, dtype):
    """Gate values from -12 (gelu -2e-32) to 3, one product of each."""
    in_, out = 32, 600
    q = torch.zeros(tokens, in_, dtype=torch.int8, device="cuda")
    q[:, 0] = 1
    scale = (1 + torch.arange(tokens, device="cuda") / (4.0 * tokens)).float()
    x = lib.Int8Tokens(q, scale, torch.ones(tokens, dtype=torch.int32, device="cuda"))
    w = torch.zeros(out, in_, dtype=torch.int8, device="cuda")
    w[:, 0] = torch.arange(out, device="cuda") % 160 - 127
    gate = (w, torch.full((out,), 9.6 / 127, device="cuda"))
    one = torch.zeros_like(w)
    one[:, 0] = 1
    up = (one, torch.full((out,), 0.75, device="cuda"))
    y = lib.gated_int8(x, gate, up, act="gelu", dtype=dtype)
    g = scale.double()[:, None] * (w[:, 0].double() * gate[1].double())
    want = 0.5 * g * torch.special.erfc(-g / 2 ** 0.5) * (0.75 * scale.double()[:, None])
    # g is 2 roundings off and erfc's argument 2 more; the condition number of gelu is at most g^2 + 3 below zero
    # (Mills' ratio) and 2 above.  erfcf is within 4 units of 2^-23 (documented); 6 roundings around it.
    tol = want.abs() * ((g ** 2 + 3) * 4 * R.U32 + 4 * 2.0 ** -23 + 6 * R.U32 + R.U[dtype]) * 1.01 + R.FLOOR[dtype]
    _within(y, want, tol)


# ----------------------------------------------- layer norms far from their mean
ROWS = [(1, 4096), (3, 77), (200, 264), (5, 11008), (700, 9000), (650, 9001), (1500, 4096), (700, 4001), (3, 20000)]


@pytest.mark.parametrize("tokens,d", ROWS)
@pytest.mark.parametrize("spread", [0.0, 0.05])
def test_layer_norm_of_rows_with_a_large_common_offset(lib, tokens, d, spread):
    """fp32 rows around +-1000, all equal or 1/20000 of that apart, as h and, with
    a post-norm, as y."""
    rng = np.random.default_rng([23, tokens, d])
    base = 1000.1 * np.where(np.arange(tokens) % 2, -1, 1)[:, None] * (1 + 0.01 * rng.random((tokens, 1)))
    v = (base + spread * rng.standard_normal((tokens, d))).astype(np.float32)
    w, b = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32), rng.standard_normal(d).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    eps = float(np.float32(1e-5))
    a = v.astype(np.float64)
    mean = a.mean(1, keepdims=True)
    c = a - mean
    r = 1 / np.sqrt((c ** 2).mean(1, keepdims=True) + eps)
    x = c * r * w
    # A first mean is off by no more than R.ROUNDINGS roundings of its size, and
    # so are the values without it; their sum takes that out again, but for
    # R.ROUNDINGS roundings of what it sums.
    n = R.ROUNDINGS * R.U32
    size = np.abs(c).mean(1, keepdims=True) + n * np.abs(mean)
    dv = R.U32 * (np.abs(c) + n * np.abs(mean)) + n * size
    # the variance: its own sum's roundings, and those of the squared residue taken from it
    dr = 1.5 * n * r ** 2 * ((c ** 2).mean(1, keepdims=True) + (n * mean) ** 2)
    tol = (dv * r * np.abs(w) + np.abs(x) * (dr + 4 * R.U32) + R.U32 * np.abs(x + b) * 2) * 1.05
    got, out = lib.norm_tokens(dev(v), None, dev(w), bias=dev(b), kind="layer", eps=eps)
    want = torch.from_numpy(x + b).cuda()
    _within(out, want, torch.from_numpy(tol).cuda())
    h1, _ = lib.norm_tokens(torch.zeros_like(got), dev(v), dev(w), bias=dev(b), post_weight=dev(w), post_bias=dev(b),
                            kind="layer", eps=eps)
    _within(h1, want, torch.from_numpy(tol).cuda())
    _, t = lib.norm_tokens(dev(v), None, dev(w), bias=dev(b), kind="layer", eps=eps, quantize=True)
    half = (0.5 + 1e-4) * t.scale.double()[:, None]
    _within(t.q.double() * t.scale.double()[:, None], want, half + torch.from_numpy(tol).cuda())


# ------------------------------------------------------------- other host threads
_STUB = r"""
#include <time.h>
static volatile int other_ran = 0;
void let_go(void) { other_ran = 1; }
void again(void) { other_ran = 0; }
static int wait_for_other(void) {  /* GPTQ_OK once another thread has run, GPTQ_ERR_TIMEOUT after two seconds */
  struct timespec t = {0, 1000000};
  for (int i = 0; i < 2000 && !other_ran; ++i) nanosleep(&t, 0);
  return other_ran ? 0 : 6;
}
int gptq_quantize_tokens() { return wait_for_other(); }
int gptq_norm_tokens() { return wait_for_other(); }
int gptq_matmul_int8() { return wait_for_other(); }
int gptq_matmul_int8_gated() { return wait_for_other(); }
int gptq_linear_int8() { return wait_for_other(); }
int gptq_linear_int8_gated() { return wait_for_other(); }
"""

_THREADS = r"""
import ctypes, sys, threading, time
import torch, post_weight_quantization_13_b200 as g
stub = ctypes.CDLL(sys.argv[1])
x = torch.ones(40, 64, device='cuda', dtype=torch.bfloat16)
w = torch.ones(64, device='cuda', dtype=torch.bfloat16)
layer = g.Int8Layer(torch.ones(64, 64, device='cuda', dtype=torch.int8), torch.ones(64, device='cuda'))
t = g.Int8Tokens(layer.weight, layer.scale, layer.scale.int())
calls = {'quantize': lambda: g.quantize_tokens(x), 'norm': lambda: g.norm_tokens(x, x, w),
         'linear': lambda: g.linear_int8(x, layer), 'gated': lambda: g.gated_int8(x, layer, layer),
         'linear, tokens': lambda: g.linear_int8(t, layer), 'gated, tokens': lambda: g.gated_int8(t, layer, layer)}
stuck = []
for name, call in calls.items():
    stub.again()
    def other():
        time.sleep(0.1)
        stub.let_go()
    th = threading.Thread(target=other)
    th.start()
    try:
        call()
    except g.GptqError as e:
        stuck.append(name)
    th.join()
assert not stuck, stuck
"""


def test_other_threads_run_while_a_call_is_in_the_library(tmp_path):
    """A launch can wait for room in a full queue; a host callback ahead of it may
    need the interpreter.  The library is replaced by calls that wait for another
    Python thread."""
    import os
    import subprocess
    import sys
    (tmp_path / "stub.c").write_text(_STUB)
    stub = str(tmp_path / "stub.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-w", "-o", stub, str(tmp_path / "stub.c")], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _THREADS, stub], cwd=root, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "LD_PRELOAD": stub})
    assert r.returncode == 0, r.stderr[-2000:]


# ------------------------------------------------------------ waits that give up
def _gave_up(lib, stream=None):
    try:
        lib.gptq_int8_status(stream)
    except lib.GptqError as e:
        assert e.status == 6 and "gave up" in str(e)
        return True
    return False


def test_a_wait_that_gives_up_is_reported_once(lib):
    lib.gptq_int8_status()
    lib.gptq_selftest_int8_timeout(200_000)
    assert _gave_up(lib)
    assert not _gave_up(lib)
    rng = np.random.default_rng(31)                 # the device is as usable as before
    layer = R.random_layer(rng, 40, 64)
    x = torch.from_numpy(rng.standard_normal((5, 64)).astype(np.float32))
    q, s = R.quantize(x.numpy())
    p = R.product(q, s, layer)
    _within(lib.linear_int8(x.cuda(), R.on_device(lib, layer)).cpu(), torch.from_numpy(p),
            torch.from_numpy(R.linear_tol(p, None, F32)))
    assert not _gave_up(lib)


def test_reports_from_another_stream_are_not_lost(lib):
    """A wait gives up on one stream while the status is read on another, again
    and again: it is reported by a reading that was under way, or by the next."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    lib.gptq_int8_status()
    done = torch.cuda.Event()
    for i in range(1000):
        lib.gptq_selftest_int8_timeout(1000 + 37 * i, a)
        done.record(a)
        reported = 0
        while not done.query():
            reported += _gave_up(lib, b)
        reported += _gave_up(lib, a)
        assert reported, i


# ------------------------------------------------ a workspace used again and again
@pytest.mark.parametrize("tokens,in_,out", [(700, 256, 520), (3000, 512, 2048), (40, 1024, 300)])
def test_one_workspace_for_many_calls_in_a_row(lib, tokens, in_, out):
    """A product may begin while the quantizer ahead of it still writes the codes,
    scales and sums of its tokens over those of the call before."""
    rng = np.random.default_rng([37, tokens])
    layer = R.on_device(lib, R.random_layer(rng, out, in_, True))
    xs = [torch.from_numpy((10.0 ** (i % 5 - 2) * rng.standard_normal((tokens, in_))).astype(np.float32)).to(BF16).cuda()
          for i in range(8)]
    want = []
    for x in xs:
        t = lib.quantize_tokens(x)
        torch.cuda.synchronize()
        want.append(lib.linear_int8(t, layer, dtype=F32))
    ws = torch.empty(lib.gptq_linear_int8_ws_bytes(tokens, in_), dtype=torch.uint8, device="cuda")
    got = [torch.empty(tokens, out, device="cuda") for _ in xs]
    for _ in range(10):
        for y in got:
            y.fill_(float("nan"))
        for x, y in zip(xs, got):
            lib.gptq_linear_int8(x, layer, y, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------- a reordered layer
@pytest.mark.parametrize("bits", [8, 4])
def test_int8_layer_of_a_layer_solved_in_another_order(lib, bits):
    """desc_act: the codes stand in the weight's own order all the same."""
    rng = np.random.default_rng([29, bits])
    W = torch.from_numpy((0.02 * rng.standard_normal((70, 288))).astype(np.float32)).cuda()
    X = torch.from_numpy((rng.standard_normal((288, 900)) * np.exp(rng.standard_normal((288, 1)))).astype(np.float32))
    r = lib.solve_layer(W, X.to(F16).cuda(), dict(bits=bits, group_size=-1, sym=False, desc_act=True))
    assert not torch.equal(r["perm"].cpu(), torch.arange(288, dtype=r["perm"].dtype))
    layer = lib.int8_layer(r, bits)
    deq = torch.empty(70, 288, device="cuda")
    lib.gptq_dequantize_layer(r["qweight"], r["scales"], r["zeros"], r["g_idx"], bits, deq)
    z = torch.zeros(70, dtype=torch.int32, device="cuda") if layer.zero is None else layer.zero
    assert torch.equal(layer.scale[:, None] * (layer.weight.int() - z[:, None]).float(), deq)


# --------------------------------------------------------------- the most tokens
def test_the_largest_number_of_tokens(lib):
    """2^26 tokens: their rows equal those of small calls."""
    T, d, out = 1 << 26, 32, 3
    gen = torch.Generator("cuda").manual_seed(41)
    x = torch.empty(T, d, dtype=BF16, device="cuda").normal_(generator=gen)
    layer = R.on_device(lib, R.random_layer(np.random.default_rng(43), out, d, True))
    w = torch.rand(d, generator=gen, device="cuda").to(BF16)
    y, z = lib.linear_int8(x, layer), lib.gated_int8(x, layer, layer)
    h, t = lib.norm_tokens(x, x, w, quantize=True)
    for first in (0, T // 2 - 77, T - 300):
        rows = slice(first, first + 300)
        assert torch.equal(y[rows], lib.linear_int8(x[rows], layer))
        assert torch.equal(z[rows], lib.gated_int8(x[rows], layer, layer))
        h1, t1 = lib.norm_tokens(x[rows], x[rows], w, quantize=True)
        assert torch.equal(h[rows], h1) and all(torch.equal(a[rows], b) for a, b in zip(t, t1))
    lib.gptq_int8_status()


# --------------------------------------------------- broadcast gates, shared rows
@pytest.mark.parametrize("tokens,d", [(5, 264), (700, 9000), (3000, 4001)])
def test_a_gate_expanded_over_the_tokens_is_a_gate_for_channels(lib, tokens, d):
    gen = torch.Generator("cuda").manual_seed(47)
    h, y = (torch.randn(tokens, d, generator=gen, device="cuda").to(F16) for _ in range(2))
    w, g = (torch.rand(d, generator=gen, device="cuda").to(F16) for _ in range(2))
    want = lib.norm_tokens(h, y, w, gate=g)
    for gate in (g.expand(tokens, d), g.repeat(tokens, 1)):
        assert all(torch.equal(a, b) for a, b in zip(lib.norm_tokens(h, y, w, gate=gate), want))


@pytest.mark.parametrize("tokens", [1, 2, 3, 40, 700])
def test_slices_of_tokens_and_of_layers_are_tokens_and_layers(lib, tokens):
    rng = np.random.default_rng([53, tokens])
    layer = R.on_device(lib, R.random_layer(rng, 300, 520, True))
    t = lib.quantize_tokens(torch.from_numpy(rng.standard_normal((tokens + 9, 520)).astype(np.float32)).cuda())
    y = lib.linear_int8(t, layer, dtype=F32)
    part = lib.Int8Tokens(*(a[5:5 + tokens] for a in t))
    rows = lib.Int8Layer(*(a[7:290] for a in layer))
    assert torch.equal(lib.linear_int8(part, rows, dtype=F32), y[5:5 + tokens, 7:290])
    assert torch.equal(lib.gated_int8(part, rows, rows, dtype=F32),
                       lib.gated_int8(t, layer, layer, dtype=F32)[5:5 + tokens, 7:290])
