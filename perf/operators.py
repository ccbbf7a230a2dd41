"""The 8-bit serving operators, case by case: what a pass takes in, computes and gives back.

Three operators run a layer that the solver has quantized on 8-bit integer
tensor cores:

  linear  y = s_t s_n (sum_k q_tk w_nk - z_n sum_k q_tk) + b_n, with each
          token quantized to 8 bits on the way in
  gated   act(gate projection) * up projection, both projections as above
  norm    h' = alpha h + beta gate * post(y) and x = pre(h'): the norms after
          and before a block with its gate and residual scale.  With "next"
          the tokens x leave in 8 bits for a linear that reads them, which is
          how they are used.

Where ``own`` is false ``run`` computes them in elementary torch operations,
where it is true through this package's calls.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
ACTS = ("silu", "gelu", "gelu_tanh")


def _linear(name, tokens, in_, out, dtype, zero=False, bias=False):
    return {"name": name, "op": "linear", "tokens": tokens, "in": in_, "out": out, "dtype": dtype, "zero": zero,
            "bias": bias}


def _gated(name, tokens, in_, out, dtype, act="silu", zero=False):
    return {"name": name, "op": "gated", "tokens": tokens, "in": in_, "out": out, "dtype": dtype, "act": act,
            "zero": zero}


def _norm(name, tokens, d, dtype, h_dtype, kind="rms", post=False, gate="none", alpha=1.0, beta=1.0, next_=0):
    return {"name": name, "op": "norm", "tokens": tokens, "in": d, "dtype": dtype, "h_dtype": h_dtype, "kind": kind,
            "post": post, "gate": gate, "alpha": alpha, "beta": beta, "next": next_}


def listed():
    return [
        # one sequence being decoded: an attention projection of a 7B decoder block
        _linear("linear 1 4096>4096", 1, 4096, 4096, "bf16"),
        # a decode batch through the down projection, asymmetric weights
        _linear("linear 24 11008>4096", 24, 11008, 4096, "f16", zero=True),
        # a short prompt of odd length
        _linear("linear 333 4096>4096", 333, 4096, 4096, "bf16", bias=True),
        # odd sizes all round and a 32-bit output: a classifier or a small vocabulary
        _linear("linear 77 1000>2777", 77, 1000, 2777, "f32", zero=True, bias=True),
        # a batch of prompts, or the calibration tokens passed through a solved layer
        _linear("linear 16384 4096>11008", 16384, 4096, 11008, "f16"),
        # the gated projections at decode
        _gated("gated 1 4096>11008", 1, 4096, 11008, "bf16"),
        # odd sizes, a decode batch
        _gated("gated 100 2000>5461", 100, 2000, 5461, "f16", act="gelu_tanh", zero=True),
        # a prompt batch
        _gated("gated 4096 4096>11008", 4096, 4096, 11008, "bf16"),
        # decode: residual add, pre-norm
        _norm("norm 1 4096", 1, 4096, "bf16", "bf16"),
        # a prompt batch with norms on both sides, a gate for each channel and a residual scale
        _norm("norm 8192 4096 post", 8192, 4096, "bf16", "bf16", post=True, gate="channel", beta=0.5),
        # layer norms, a gate for each token, a 32-bit residual stream, an odd count of tokens
        _norm("norm 1001 11008 layer", 1001, 11008, "f16", "f32", kind="layer", post=True, gate="token", alpha=0.7),
        # the tokens leave in 8 bits for the projection that reads them
        _norm("norm 2000 4096 >4096", 2000, 4096, "bf16", "bf16", next_=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "gated", "norm"))
    dtype = rng.choice(("f16", "bf16"))
    tokens = _log(rng, 1, 16384)
    if op == "norm":
        d = _log(rng, 64, 11008)
        tokens = max(1, min(tokens, 8192 * 4096 // d))
        c = _norm("", tokens, d, dtype, rng.choice((dtype, "f32")), rng.choice(("rms", "layer")), rng.random() < 0.5,
                  rng.choice(("none", "channel", "token")), rng.choice((1.0, 0.7)), rng.choice((1.0, 0.5)),
                  rng.choice((0, _log(rng, 64, 4096))))
    else:
        in_, out = _log(rng, 64, 11008), _log(rng, 64, 11008)
        tokens = max(1, min(tokens, 16384 * 4096 * 11008 // (2 * in_ * out)))
        if op == "linear":
            c = _linear("", tokens, in_, out, rng.choice((dtype, dtype, "f32")), rng.random() < 0.5,
                        rng.random() < 0.5)
        else:
            c = _gated("", tokens, in_, out, dtype, rng.choice(ACTS), rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _tokens(gen, tokens, d, dtype):
    """Activations: normal, with lognormal scales of the channels."""
    s = torch.exp(torch.randn(d, generator=gen, device="cuda"))
    return (torch.randn(tokens, d, generator=gen, device="cuda") * s).to(dtype)


def _weight(gen, out, in_, zero):
    """int8 rows (16-byte row stride), a scale for each channel, a zero for
    each channel or none: N(0, 0.02^2) weights rounded to nearest."""
    w = torch.randn(out, in_, generator=gen, device="cuda") * 0.02
    z = None
    if zero:  # the asymmetric grid over [min, max], shifted by 128
        lo, hi = w.amin(1).clamp(max=0), w.amax(1).clamp(min=0)
        scale = (hi - lo) / 255
        z = torch.round(-lo / scale).int() - 128
        q = (torch.round(w / scale[:, None]) + z[:, None]).clamp(-128, 127)
    else:
        scale = w.abs().amax(1) * 2 / 255
        q = torch.round(w / scale[:, None]).clamp(-128, 127)
    rows = torch.zeros(out, (in_ + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    rows[:, :in_] = q
    return rows[:, :in_], scale, z


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    dt, T, I = DTYPES[c["dtype"]], c["tokens"], c["in"]
    s = {"case": c}
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if c["op"] == "linear":
        s["x"] = _tokens(gen, T, I, dt)
        s["layer"] = _weight(gen, c["out"], I, c["zero"])
        s["bias"] = randn(c["out"]) if c["bias"] else None
    elif c["op"] == "gated":
        s["x"] = _tokens(gen, T, I, dt)
        s["gate"] = _weight(gen, c["out"], I, c["zero"])
        s["up"] = _weight(gen, c["out"], I, c["zero"])
    else:
        s["h"] = (2 * randn(T, I)).to(DTYPES[c["h_dtype"]])
        s["y"] = _tokens(gen, T, I, dt)
        layer = c["kind"] == "layer"
        s["post_weight"] = (1 + 0.1 * randn(I)).to(dt) if c["post"] else None
        s["post_bias"] = (0.1 * randn(I)).to(dt) if c["post"] and layer else None
        s["weight"] = (1 + 0.1 * randn(I)).to(dt)
        s["bias"] = (0.1 * randn(I)).to(dt) if layer else None
        shape = {"none": None, "channel": (I,), "token": (T, I)}[c["gate"]]
        s["gate"] = torch.sigmoid(randn(*shape)).to(dt) if shape else None
        s["next"] = _weight(gen, c["next"], I, False) if c["next"] else None
    return s


# ------------------------------------------------------------------ plain form
def _quantize(x):
    scale = x.abs().amax(1, keepdim=True) / 127
    q = torch.round(x / torch.where(scale > 0, scale, 1.0)).clamp(-127, 127)
    return q, scale


def _product(x, layer):
    w, scale, z = layer
    q, s = _quantize(x)
    w = w.float() if z is None else w.float() - z.float()[:, None]
    return (q @ w.T) * s * scale


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _normed(v, kind, weight, bias):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * weight.float()
    return v if bias is None else v + bias.float()


def _run_plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "linear":
        y = _product(s["x"].float(), s["layer"])
        return (y if s["bias"] is None else y + s["bias"]).to(dt)
    if c["op"] == "gated":
        x = s["x"].float()
        return (_act(_product(x, s["gate"]), c["act"]) * _product(x, s["up"])).to(dt)
    u = s["y"].float()
    if c["post"]:
        u = _normed(u, c["kind"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        u = s["gate"].float() * u
    h = c["alpha"] * s["h"].float() + c["beta"] * u
    x = _normed(h, c["kind"], s["weight"], s["bias"])
    if s["next"] is not None:
        x = _product(x, s["next"])
    return h.to(s["h"].dtype), x.to(dt)


def _run_own(s):
    import post_weight_quantization_13_b200 as g
    c = s["case"]
    if c["op"] == "linear":
        return g.linear_int8(s["x"], s["layer"], bias=s["bias"])
    if c["op"] == "gated":
        return g.gated_int8(s["x"], s["gate"], s["up"], act=c["act"])
    h, x = g.norm_tokens(s["h"], s["y"], s["weight"], bias=s["bias"], post_weight=s["post_weight"],
                         post_bias=s["post_bias"], gate=s["gate"], alpha=c["alpha"], beta=c["beta"], kind=c["kind"],
                         eps=EPS, quantize=s["next"] is not None)
    if s["next"] is not None:
        x = g.linear_int8(x, s["next"], dtype=s["y"].dtype)
    return h, x


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ floors
def work(case):
    c = case
    T, I, e = c["tokens"], c["in"], SIZE[c["dtype"]]
    if c["op"] == "norm":
        eh, O = SIZE[c["h_dtype"]], c["next"]
        vectors = 1 + (c["kind"] == "layer")
        b = T * I * (2 * eh + e) + e * I * vectors * (1 + bool(c["post"]))
        b += {"none": 0, "channel": e * I, "token": T * I * e}[c["gate"]]
        b += (I * O + 4 * O + T * O * e) if O else T * I * e
        return {"bytes": b, "flops": 15 * T * I + 2 * T * I * O}
    O, n = c["out"], 2 if c["op"] == "gated" else 1
    b = T * I * e + n * (I * O + 4 * O + 4 * O * bool(c["zero"])) + 4 * O * bool(c.get("bias")) + T * O * e
    return {"bytes": b, "flops": 2 * n * T * I * O}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """The same outputs from the definitions in 64 bits.  A token's scale and
    the quotient that is rounded to a code are 32-bit values by definition;
    both are formed in 64 bits and rounded to 32."""
    s = prepare(case, seed)
    D = torch.float64

    def codes(x):
        scale = (x.abs().max(dim=1).values / 127).float().to(D)
        quotient = torch.zeros_like(x)
        used = scale > 0
        quotient[used] = (x[used] / scale[used].unsqueeze(1)).float().to(D)
        return torch.clamp(torch.round(quotient), -127, 127), scale

    def project(q, scale, layer):
        w, channel, z = layer
        total = torch.mm(q, w.to(D).t())
        if z is not None:
            total = total - torch.outer(q.sum(dim=1), z.to(D))
        return total * torch.outer(scale, channel.to(D))

    def normalise(v, weight, bias):
        n = v.shape[1]
        if case["kind"] == "layer":
            v = v - (v.sum(dim=1) / n).unsqueeze(1)
        root = torch.sqrt((v ** 2).sum(dim=1) / n + EPS)
        v = (v / root.unsqueeze(1)) * weight.to(D)
        return v + bias.to(D) if bias is not None else v

    if case["op"] == "linear":
        y = project(*codes(s["x"].to(D)), s["layer"])
        return y + s["bias"].to(D) if s["bias"] is not None else y
    if case["op"] == "gated":
        q, scale = codes(s["x"].to(D))
        a, b = project(q, scale, s["gate"]), project(q, scale, s["up"])
        if case["act"] == "silu":
            a = a * torch.sigmoid(a)
        elif case["act"] == "gelu":
            a = a * 0.5 * torch.erfc(-a / math.sqrt(2.0))
        else:
            a = a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))
        return a * b
    u = s["y"].to(D)
    if s["post_weight"] is not None:
        u = normalise(u, s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        u = u * s["gate"].to(D)
    h = s["h"].to(D) * case["alpha"] + u * case["beta"]
    x = normalise(h, s["weight"], s["bias"])
    if s["next"] is not None:
        x = project(*codes(x.float().to(D)), s["next"])
    return h, x
