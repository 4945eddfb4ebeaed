"""Cases that time the microscaled 4-bit operators and check them: quantisation, products, a mixture-of-experts layer.

Number formats.  A value is held in 4 bits (sign, two exponent bits, one fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
their negatives).  Each block of consecutive values of a row shares a scale:

* ``mxfp4``: blocks of 32; the scale is a power of two, 2^(byte - 127), with byte = floor(log2(largest |x|)) - 2 + 127.
* ``nvfp4``: blocks of 16; the scale is an 8-bit float (4 exponent bits, 3 fraction bits) times one 32-bit factor g of the
  whole matrix; the block's scale is largest |x| / (6 g), rounded to nearest.

A value is divided by its block's scale and rounded to the nearest of the 16, ties to the even code, at most 6 in magnitude.

``own = False`` computes everything with elementary torch operations in 32 bits; ``own = True`` calls the package.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # Quantise a matrix and read the values back (what a program does that calibrates or checks a checkpoint).
        # A decode step's activations: latency.
        {"name": "quantise 16x4096 mx", "op": "quantise", "rows": 16, "cols": 4096, "pad": 0, "format": "mxfp4", "dtype": "bfloat16"},
        # A slice of a wider matrix with an odd number of columns: rows that start at any address.
        {"name": "quantise 1000x5003 nv", "op": "quantise", "rows": 1000, "cols": 5003, "pad": 6, "format": "nvfp4", "dtype": "float16"},
        # A whole 32-bit weight matrix.
        {"name": "quantise 8192x8192 nv", "op": "quantise", "rows": 8192, "cols": 8192, "pad": 0, "format": "nvfp4", "dtype": "float32"},
        # Products of two quantised matrices, C = A B^T.  Ragged in every direction, small.
        {"name": "product 300x520x200 mx", "op": "product", "m": 300, "n": 520, "k": 200, "format": "mxfp4", "out": "float32"},
        # The repository's headline square size.
        {"name": "product 4096x4096x4096 mx", "op": "product", "m": 4096, "n": 4096, "k": 4096, "format": "mxfp4", "out": "float32"},
        # The largest square size.
        {"name": "product 8192x8192x8192 nv", "op": "product", "m": 8192, "n": 8192, "k": 8192, "format": "nvfp4", "out": "bfloat16"},
        # A linear layer on unquantised activations.  One token of a decode step.
        {"name": "linear 1x4096x4096 nv", "op": "linear", "m": 1, "n": 4096, "k": 4096, "format": "nvfp4", "dtype": "bfloat16"},
        # A decode step over a batch of sequences.
        {"name": "linear 16x8192x8192 mx", "op": "linear", "m": 16, "n": 8192, "k": 8192, "format": "mxfp4", "dtype": "bfloat16"},
        # A prompt, or a training batch's forward pass.
        {"name": "linear 16384x1024x4096 nv", "op": "linear", "m": 16384, "n": 1024, "k": 4096, "format": "nvfp4", "dtype": "float32"},
        # A mixture-of-experts layer for a few tokens.  One token of a decode step.
        {"name": "experts 1 token nv", "op": "experts", "tokens": 1, "d": 2048, "f": 768, "experts": 64, "top": 8, "renorm": True, "format": "nvfp4", "dtype": "bfloat16"},
        # Odd sizes, 32-bit activations, few large experts.
        {"name": "experts 5 tokens mx odd", "op": "experts", "tokens": 5, "d": 1032, "f": 520, "experts": 12, "top": 3, "renorm": False, "format": "mxfp4", "dtype": "float32"},
        # A decode step over a batch: most experts are used by a token or two.
        {"name": "experts 16 tokens nv", "op": "experts", "tokens": 16, "d": 4096, "f": 2048, "experts": 64, "top": 8, "renorm": True, "format": "nvfp4", "dtype": "bfloat16"},
    ]


def _spread(rng, low, high, step=1):
    """A size between low and high, spread over its logarithm; half of them multiples of `step`, the rest any number."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if step > 1 and rng.random() < 0.5:
        n = max(step, n // step * step)
    n = min(high, max(low, n))
    return n if n != 3072 else 3200


def draw(rng):
    op = rng.choice(("quantise", "product", "linear", "experts"))
    c = {"op": op, "format": rng.choice(("mxfp4", "nvfp4"))}
    dtype = rng.choice(("float32", "bfloat16", "float16"))
    if op == "quantise":
        c.update(rows=_spread(rng, 1, 8192), cols=_spread(rng, 16, 8192, 32), pad=rng.choice((0, 0, 8, 3)), dtype=dtype)
    elif op == "product":
        c.update(m=_spread(rng, 16, 8192, 128), n=_spread(rng, 16, 8192, 128), k=_spread(rng, 16, 8192, 32), out=dtype)
    elif op == "linear":
        n, k = _spread(rng, 256, 8192, 128), _spread(rng, 256, 8192, 128)
        c.update(m=_spread(rng, 1, min(16384, 8192**3 // (n * k))), n=n, k=k, dtype=dtype)
    else:
        experts = _spread(rng, 4, 64)
        c.update(tokens=_spread(rng, 1, 16), d=_spread(rng, 256, 4096, 64), f=_spread(rng, 64, 1500, 64), experts=experts,
                 top=rng.randint(1, min(8, experts)), renorm=rng.random() < 0.5, dtype=dtype)
    return c


# --------------------------------------------------------------------------------------------------------------- inputs
def _activations(rows, cols, dtype, gen, pad=0):
    """Normal values in which a few columns are several times larger, as a layer's activations have them."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda")
    large = torch.rand(cols + pad, generator=gen, device="cuda") < 0.01
    return (x * (1.0 + 7.0 * large)).to(DTYPES[dtype])[:, :cols]


def _codes(x, form):
    """A weight matrix as a checkpoint holds it: codes, two to a byte (the even column in the low bits), one scale byte a
    block, and the factor g (None for mxfp4)."""
    g = x.abs().amax().float().reshape(1) / (6.0 * 448.0) if form == "nvfp4" else None
    code, scale = _quantise(x, form, g)
    code = torch.nn.functional.pad(code, (0, code.shape[-1] % 2))
    return code[..., 0::2] | (code[..., 1::2] << 4), scale, g


def _weights(shape, form, gen):
    return _codes(torch.randn(shape, generator=gen, device="cuda") / math.sqrt(shape[-1]), form)


def prepare(case, seed):
    c, form = case, case["format"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": c["op"], "format": form}
    if c["op"] == "quantise":
        s["x"] = _activations(c["rows"], c["cols"], c["dtype"], gen, c["pad"])
        s["g"] = s["x"].abs().amax().float().reshape(1) / (6.0 * 448.0) if form == "nvfp4" else None
        return s
    if c["op"] == "product":
        s["out"], s["k"] = DTYPES[c["out"]], c["k"]
        a = _codes(_activations(c["m"], c["k"], "float32", gen), form)
        b = _weights((c["n"], c["k"]), form, gen)
        s["a"], s["b"] = _handle(a, form, c["k"]), _handle(b, form, c["k"])
        return s
    if c["op"] == "linear":
        s["x"], s["k"] = _activations(c["m"], c["k"], c["dtype"], gen), c["k"]
        s["g"] = s["x"].abs().amax().float().reshape(1) / (6.0 * 448.0) if form == "nvfp4" else None
        s["w"] = _handle(_weights((c["n"], c["k"]), form, gen), form, c["k"])
        return s
    d, f, experts = c["d"], c["f"], c["experts"]
    s.update(top=c["top"], renorm=c["renorm"], d=d, f=f)
    s["x"] = torch.randn(c["tokens"], d, generator=gen, device="cuda").to(DTYPES[c["dtype"]])
    s["router"] = torch.randn(experts, d, generator=gen, device="cuda") * (1.5 / math.sqrt(d))
    gate_up = _weights((experts * 2 * f, d), form, gen)
    down = _weights((experts * d, f), form, gen)
    if own:
        import dense_fp32_gemm_03_gb300 as sg
        s["experts"] = sg.fp4_experts(_handle(gate_up, form, d), _handle(down, form, f), experts)
    else:
        s["gate_up"] = tuple(t.view(experts, 2 * f, -1) for t in gate_up[:2]) + (gate_up[2],)
        s["down"] = tuple(t.view(experts, d, -1) for t in down[:2]) + (down[2],)
    return s


def _handle(parts, form, cols):
    """The weights as a program keeps them: the checkpoint's arrays, or the library's matrix made from them once."""
    if not own:
        return parts
    import dense_fp32_gemm_03_gb300 as sg
    return sg.fp4_matrix(parts[0], parts[1], form, cols=cols, scale=parts[2])


# ---------------------------------------------------------------------------------------------------------- plain forms
def _blocks(x, form):
    n = BLOCK[form]
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % n)).unflatten(-1, (-1, n))


def _quantise(x, form, g):
    """(codes, one to a byte; scale bytes) of the rows of x, in 32 bits."""
    b = _blocks(x.float(), form)
    top = b.abs().amax(-1)
    if form == "mxfp4":
        e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
        scale, unit = (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(top), e)
    else:
        s = (top / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale, unit = s.view(torch.uint8), s.float() * g
    v = torch.where(unit[..., None] > 0, b / unit[..., None], 0.0)
    m = v.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    return code.flatten(-2)[..., : x.shape[-1]], scale


def _units(scale, form, g):
    """The blocks' scales in 32 bits."""
    if form == "mxfp4":
        return torch.ldexp(torch.ones(scale.shape, device=scale.device), scale.int() - 127)
    return scale.view(torch.float8_e4m3fn).float() * g


def _values(packed, scale, g, form, cols):
    """The values that two-to-a-byte codes and their scales stand for, in 32 bits."""
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=packed.device)
    pair = torch.stack((level.repeat(16), level.repeat_interleave(16)), -1)
    v = _blocks(pair[packed.int()].flatten(-2)[..., :cols], form)
    return (v * _units(scale, form, g)[..., None]).flatten(-2)[..., :cols]


def _round(x, form, g):
    """x quantised and read back, in 32 bits."""
    code, scale = _quantise(x, form, g)
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=x.device)
    v = _blocks(level[code.int()], form) * _units(scale, form, g)[..., None]
    return v.flatten(-2)[..., : x.shape[-1]]


def _plain_experts(s):
    x, form = s["x"].float(), s["format"]
    logits = x @ s["router"].t()
    ids = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, : s["top"]]
    e = torch.exp(logits - logits.amax(-1, keepdim=True))
    w = (e / e.sum(-1, keepdim=True)).gather(-1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    pick, tokens = ids.flatten(), x.shape[0]
    codes, scale, g = s["gate_up"]
    rows = x.repeat_interleave(s["top"], 0)[:, :, None]
    gate, up = (_values(codes[pick], scale[pick], g, form, s["d"]) @ rows).squeeze(-1).split(s["f"], -1)
    h = gate / (1.0 + torch.exp(-gate)) * up
    codes, scale, g = s["down"]
    y = (_values(codes[pick], scale[pick], g, form, s["f"]) @ h[:, :, None]).view(tokens, s["top"], -1)
    return {"out": (y * w[:, :, None]).sum(1).to(s["x"].dtype), "ids": ids.int(), "weights": w}


def run(s):
    if own:
        import dense_fp32_gemm_03_gb300 as sg
        if s["op"] == "quantise":
            return sg.fp4_dequantize(sg.fp4_quantize(s["x"], s["format"], scale=s["g"]), dtype=s["x"].dtype)
        if s["op"] == "product":
            return sg.fp4_gemm(s["a"], s["b"], out_dtype=s["out"])
        if s["op"] == "linear":
            return sg.fp4_linear(s["x"], s["w"], x_scale=s["g"])
        out, ids, weights = sg.fp4_moe(s["x"], s["router"], s["experts"], s["top"], renormalize=s["renorm"], return_routing=True)
        return {"out": out, "ids": ids, "weights": weights}
    if s["op"] == "quantise":
        return _round(s["x"], s["format"], s["g"]).to(s["x"].dtype)
    if s["op"] == "product":
        a, b = (_values(*s[k], s["format"], s["k"]) for k in ("a", "b"))
        return (a @ b.t()).to(s["out"])
    if s["op"] == "linear":
        a = _round(s["x"], s["format"], s["g"])
        return (a @ _values(*s["w"], s["format"], s["k"]).t()).to(s["x"].dtype)
    return _plain_experts(s)


def work(case):
    """Each input read once, each output written once; two operations a product term."""
    c, bits = case, 4 + 8 / BLOCK[case["format"]]
    size = {"float32": 4, "bfloat16": 2, "float16": 2}[c.get("dtype", c.get("out"))]
    if c["op"] == "quantise":
        return {"bytes": 2 * c["rows"] * c["cols"] * size, "flops": 2 * c["rows"] * c["cols"]}
    if c["op"] in ("product", "linear"):
        m, n, k = c["m"], c["n"], c["k"]
        a = m * k * bits / 8 if c["op"] == "product" else m * k * size
        return {"bytes": a + n * k * bits / 8 + m * n * size, "flops": 2 * m * n * k}
    t, d, f, e, top = c["tokens"], c["d"], c["f"], c["experts"], c["top"]
    used = e * (1.0 - (1.0 - top / e) ** t)  # experts that some token goes to, on average
    return {"bytes": used * 3 * d * f * bits / 8 + e * d * 4 + 2 * t * d * size + 8 * t * top, "flops": 2 * t * d * e + 6 * t * top * d * f}


# -------------------------------------------------------------------------------------------------------- in 64 bits
def _round_level(v):
    """The nearest 4-bit value, ties to the even code: the spacing is 1/2 below 2, 1 below 4, 2 above."""
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(v.dtype)
    return (torch.round(v / step) * step).clamp(-6, 6)


def _exponent(v):
    """The largest e with 2^e <= v (taken from the number's bits: a logarithm may be an ulp short at a power of two)."""
    return torch.where(v > 0, ((v.view(torch.int64) >> 52) - 1023).double(), -1023.0)


def _round_scale(v):
    """The nearest number with 4 exponent bits and 3 fraction bits, at most 448."""
    step = torch.exp2(_exponent(v.clamp(min=2.0**-6)) - 3)
    return (torch.round(v / step) * step).clamp(max=448)


def _round64(x, form, g):
    n, cols = BLOCK[form], x.shape[-1]
    x = torch.cat((x.double(), x.new_zeros(*x.shape[:-1], -cols % n, dtype=torch.float64)), -1)
    x = x.reshape(*x.shape[:-1], -1, n)
    top = x.abs().max(-1, keepdim=True)[0]
    if form == "mxfp4":
        unit = torch.exp2((_exponent(top) - 2).clamp(-127, 127))
    else:
        unit = _round_scale(top / (6.0 * g.double())) * g.double()
    v = torch.where(unit > 0, _round_level(x / unit), 0.0) * unit
    return v.reshape(*v.shape[:-2], -1)[..., :cols]


def _values64(packed, scale, g, form, cols):
    level = torch.tensor(LEVELS, dtype=torch.float64, device=packed.device)
    v = packed.new_empty(*packed.shape, 2, dtype=torch.float64)
    for half, bits in ((0, packed & 15), (1, packed >> 4)):
        v[..., half] = level[(bits & 7).int()] * torch.where(bits > 7, -1.0, 1.0)
    v = v.reshape(*packed.shape[:-1], -1)[..., :cols]
    if form == "mxfp4":
        unit = torch.exp2(scale.double() - 127)
    else:
        e, m = (scale >> 3).double(), (scale & 7).double()
        unit = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), m * 2.0**-9) * g.double()
    return v * unit.repeat_interleave(BLOCK[form], -1)[..., :cols]


def exact(case, seed):
    s, form = _exact_state(case, seed), case["format"]
    if s["op"] == "quantise":
        return _round64(s["x"], form, s["g"])
    if s["op"] == "product":
        return _values64(*s["a"], form, s["k"]) @ _values64(*s["b"], form, s["k"]).t()
    if s["op"] == "linear":
        return _round64(s["x"], form, s["g"]) @ _values64(*s["w"], form, s["k"]).t()
    x = s["x"].double()
    logits = x @ s["router"].double().t()
    ids = torch.argsort(-logits, dim=-1, stable=True)[:, : s["top"]]
    p = torch.softmax(logits, -1).gather(-1, ids)
    if s["renorm"]:
        p = p / p.sum(-1, keepdim=True)
    out = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(s["top"]):
            i = int(ids[t, j])
            gu = _values64(s["gate_up"][0][i], s["gate_up"][1][i], s["gate_up"][2], form, s["d"]) @ x[t]
            h = gu[: s["f"]] * torch.sigmoid(gu[: s["f"]]) * gu[s["f"] :]
            out[t] += p[t, j] * (_values64(s["down"][0][i], s["down"][1][i], s["down"][2], form, s["f"]) @ h)
    return {"out": out, "ids": ids.int(), "weights": p}


def _exact_state(case, seed):
    """The same inputs in the checkpoint's form, whatever `own` says."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was
