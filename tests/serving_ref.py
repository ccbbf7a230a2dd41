"""Plain float64 forms of the 8-bit serving calls, and how far a kernel that
computes in fp32 and rounds once may be from them."""
import numpy as np
import torch

U32 = 2.0 ** -24
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# half the smallest positive value: what rounding costs below the normal range
FLOOR = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def quantize(x):
    """Codes and scales of float32 rows, with the definition's float32
    roundings (numpy's float32 operations are IEEE)."""
    x = np.asarray(x, np.float32)
    scale = np.abs(x).max(1) * (np.float32(1) / np.float32(127))
    bad = ~np.isfinite(x).all(1)
    with np.errstate(all="ignore"):
        q = np.clip(np.rint(x / scale[:, None]), -127, 127)
    q[(scale == 0) | bad] = 0
    scale[bad] = np.nan
    return q.astype(np.int8), scale


def random_layer(rng, out, in_, zero=False):
    """(weight int8, scale, zero) on the CPU, full code range."""
    w = rng.integers(-128, 128, (out, in_)).astype(np.int8)
    s = (np.abs(rng.standard_normal(out)) * 0.01 + 1e-4).astype(np.float32)
    z = rng.integers(-128, 128, out).astype(np.int32) if zero else None
    return w, s, z


def on_device(g, layer):
    w, s, z = layer
    rows = torch.empty(w.shape[0], (w.shape[1] + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    rows.fill_(77)                      # what lies past the columns must not matter
    rows[:, :w.shape[1]] = torch.from_numpy(w)
    return g.Int8Layer(rows[:, :w.shape[1]], torch.from_numpy(s).cuda(),
                       None if z is None else torch.from_numpy(z).cuda())


def product(q, scale, layer):
    """(sum, y): the integer sums, exact, and the scaled product."""
    w, s, z = layer
    total = q.astype(np.float64) @ w.astype(np.float64).T        # integers below 2^53: exact
    if z is not None:
        total = total - q.sum(1, dtype=np.int64)[:, None] * z.astype(np.float64)[None, :]
    return total * scale.astype(np.float64)[:, None] * s.astype(np.float64)[None, :]


def linear_tol(p, bias, dtype):
    """fp32 conversion of the sum, two products and the bias addition (half a
    step each), then the output's rounding."""
    b = np.zeros(p.shape[1]) if bias is None else bias.astype(np.float64)
    y = p + b
    return 4 * U32 * (np.abs(p) + np.abs(b)) * 1.01 + U[dtype] * np.abs(y) * 1.01 + FLOOR[dtype]


def act(g, kind):
    from math import sqrt, pi
    if kind == "silu":
        return g / (1 + np.exp(-g))
    t = torch.from_numpy(g)
    if kind == "gelu":
        return (0.5 * t * torch.special.erfc(-t / sqrt(2))).numpy()
    return g / (1 + np.exp(-2 * sqrt(2 / pi) * (g + 0.044715 * g ** 3)))   # 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z))


def act_tol(g, kind):
    """The fp32 activation's error.  Its argument is 3 roundings off, which the
    activation's slope (at most 1.13) or, relatively, its condition number
    turns into an error of the result; __expf is 2 + 1.173 |z| units off (a
    unit being 2^-23), __fdividef 2, erff 2 (the documented bounds)."""
    a = np.abs(act(g, kind))
    if kind == "gelu":
        return 1.13 * np.abs(g) * 4 * U32 + 0.5 * np.abs(g) * (2.0 ** -21) + a * 4 * U32
    z = np.abs(g if kind == "silu" else 1.5957691216057308 * (g + 0.044715 * g ** 3))
    cond = 1 + z * (1 if kind == "silu" else 3)
    # z itself: up to 6 roundings, each scaled by |z| in the exponential; a
    # denominator of 2^126 and more gives 0 for a value below 2e-36
    return a * (cond * 4 * U32 + z * 6 * U32 + (2 + 1.173 * z) * 2.0 ** -23 + 4 * 2.0 ** -23) + 2e-36


def gated(q, scale, gate, up, kind, dtype):
    g, u = product(q, scale, gate), product(q, scale, up)
    y = act(g, kind) * u
    tol = act_tol(g, kind) * np.abs(u) + 5 * U32 * np.abs(y) + U[dtype] * np.abs(y) * 1.01 + FLOOR[dtype]
    return y, tol * 1.01


# A row sum of up to 32 terms a thread, 5 + 5 levels of shuffles, and the
# operations around it: no more than 64 roundings on any path.
ROUNDINGS = 64


def _norm(v, dv, weight, bias, kind, eps):
    """norm(v) and its error where v is off by dv and all sums are fp32."""
    spread = np.abs(v).mean(1, keepdims=True)
    if kind == "layer":
        mean = v.mean(1, keepdims=True)
        dv = dv + dv.mean(1, keepdims=True) + ROUNDINGS * U32 * spread + U32 * np.abs(v - mean)
        v = v - mean
    ms = (v ** 2).mean(1, keepdims=True)
    r = 1 / np.sqrt(ms + eps)
    x = v * r * weight
    # r: relative error of the mean square's half, and of v's
    dr = ROUNDINGS * U32 + np.sqrt((dv ** 2).mean(1, keepdims=True)) * r
    dx = dv * r * np.abs(weight) + np.abs(x) * (dr + 4 * U32)
    if bias is not None:
        x = x + bias
        dx = dx + U32 * np.abs(x)
    return x, dx


def norm(h, y, weight, bias, post_weight, post_bias, gate, alpha, beta, kind, eps):
    """(h', its error, x, its error), before the outputs' rounding."""
    u, du = (np.zeros_like(h), 0 * h) if y is None else (y, 0 * y)
    if post_weight is not None:
        u, du = _norm(u, du, post_weight, post_bias, kind, eps)
    if gate is not None:
        u, du = u * gate, du * np.abs(gate) + U32 * np.abs(u * gate)
    # alpha and beta reach the kernel as fp32 values
    alpha, beta = float(np.float32(alpha)), float(np.float32(beta))
    h1 = alpha * h + beta * u
    dh = abs(beta) * du + 3 * U32 * (np.abs(alpha * h) + np.abs(beta * u))
    if weight is None:
        return h1, dh, None, None
    x, dx = _norm(h1, dh, weight, bias, kind, eps)
    return h1, dh, x, dx
