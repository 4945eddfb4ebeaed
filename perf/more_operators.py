"""Cases that time the 8-bit integer operators and check them: products with scales for each token and channel, linear layers
on such weights, activation checkpoints in 8 bits and the gradients that are taken from them.

Two ways of holding numbers in 8-bit integers q from -127 to 127:

* rows (weights, and activations on their way into a product): each row has a 32-bit scale s = max(largest |x| / 127, 2^-126);
  q is the integer nearest to x / s, ties to even.  A product of two such matrices is an integer sum, then multiplied by the
  scales of its row and of its column.
* checkpoints: each block of 32 consecutive channels of a token has a unit u = 2^e, e = floor(log2 of the largest |x|) - 6 (at
  least -126, for 16-bit floats of five exponent bits -24); q is the integer nearest to x / u, ties to even, at most 127 in
  magnitude.  The value q u that is read back has at most seven bits, so 16-bit floats hold it exactly.

``own = False`` computes everything with elementary torch operations; ``own = True`` calls the package.
"""
import math

import torch

own = False

DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
BLOCK = 32


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # Products of two quantised matrices, C = A B^T.  Ragged in every direction, small.
        {"name": "product 300x520x200", "op": "product", "m": 300, "n": 520, "k": 200, "out": "float32"},
        # The repository's headline square size.
        {"name": "product 4096x4096x4096", "op": "product", "m": 4096, "n": 4096, "k": 4096, "out": "bfloat16"},
        # The largest square size.
        {"name": "product 8192x8192x8192", "op": "product", "m": 8192, "n": 8192, "k": 8192, "out": "bfloat16"},
        # A linear layer on unquantised activations.  One token of a decode step.
        {"name": "linear 1x4096x4096", "op": "linear", "m": 1, "n": 4096, "k": 4096, "dtype": "bfloat16"},
        # A decode step over a batch of sequences.
        {"name": "linear 16x8192x8192", "op": "linear", "m": 16, "n": 8192, "k": 8192, "dtype": "bfloat16"},
        # A prompt: many tokens, 32-bit activations.
        {"name": "linear 16384x1024x4096", "op": "linear", "m": 16384, "n": 1024, "k": 4096, "dtype": "float32"},
        # A linear layer's input kept in 8 bits and its weight gradient.  Odd sizes, a short sequence.
        {"name": "gradient 333x520x1001", "op": "gradient", "m": 333, "n": 520, "k": 1001, "pad": 3, "dtype": "float16"},
        # A small layer trained in 32 bits.
        {"name": "gradient 4096x1024x1024", "op": "gradient", "m": 4096, "n": 1024, "k": 1024, "pad": 0, "dtype": "float32"},
        # A wide layer over a micro-batch.
        {"name": "gradient 4096x4096x1024", "op": "gradient", "m": 4096, "n": 4096, "k": 1024, "pad": 0, "dtype": "bfloat16"},
        # The same over a whole batch.
        {"name": "gradient 16384x4096x4096", "op": "gradient", "m": 16384, "n": 4096, "k": 4096, "pad": 0, "dtype": "bfloat16"},
        # A gated activation forward and backward, its two inputs kept in 8 bits.  A short odd sequence.
        {"name": "swiglu 33x1001", "op": "swiglu", "m": 33, "f": 1001, "dtype": "float32"},
        # A training batch.
        {"name": "swiglu 8192x8192", "op": "swiglu", "m": 8192, "f": 8192, "dtype": "bfloat16"},
    ]


def _spread(rng, low, high, step=1):
    """A size between low and high, spread over its logarithm; half of them multiples of `step`, the rest any number."""
    high = max(low, high)
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if step > 1 and rng.random() < 0.5:
        n = max(step, n // step * step)
    return min(high, max(low, n))


def draw(rng):
    op = rng.choice(("product", "linear", "gradient", "swiglu"))
    dtype = rng.choice(("float32", "bfloat16", "float16"))
    c = {"op": op}
    if op == "product":
        c.update(m=_spread(rng, 1, 8192, 128), n=_spread(rng, 16, 8192, 128), k=_spread(rng, 16, 8192, 32), out=dtype)
    elif op == "linear":
        n, k = _spread(rng, 256, 8192, 128), _spread(rng, 256, 8192, 128)
        c.update(m=_spread(rng, 1, min(16384, 8192**3 // (n * k))), n=n, k=k, dtype=dtype)
    elif op == "gradient":
        n, k = _spread(rng, 64, 4096, 64), _spread(rng, 64, 4096, 64)
        c.update(m=_spread(rng, 16, 16384, 64), n=n, k=k, pad=rng.choice((0, 0, 8, 3)), dtype=dtype)
    else:
        f = _spread(rng, 64, 8192, 32)
        c.update(m=_spread(rng, 1, min(16384, 8192 * 4096 // f)), f=f, dtype=dtype)
    return c


# --------------------------------------------------------------------------------------------------------------- inputs
def _activations(rows, cols, dtype, gen, pad=0):
    """Normal values in which a few columns are several times larger, as a layer's activations have them."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda")
    large = torch.rand(cols + pad, generator=gen, device="cuda") < 0.01
    return (x * (1.0 + 7.0 * large)).to(DTYPES[dtype])[:, :cols]


def _weights(n, k, gen):
    """A weight matrix as a checkpoint holds it: 8-bit integers and a scale for each channel."""
    return _quantise(torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": c["op"]}
    if c["op"] == "product":
        s["out"] = DTYPES[c["out"]]
        s["a"] = _handle(_quantise(_activations(c["m"], c["k"], "float32", gen)))
        s["b"] = _handle(_weights(c["n"], c["k"], gen))
    elif c["op"] == "linear":
        s["x"] = _activations(c["m"], c["k"], c["dtype"], gen)
        s["w"] = _handle(_weights(c["n"], c["k"], gen))
    elif c["op"] == "gradient":
        s["x"] = _activations(c["m"], c["k"], c["dtype"], gen, c["pad"])
        s["dy"] = (torch.randn(c["m"], c["n"] + c["pad"], generator=gen, device="cuda") * 0.1).to(DTYPES[c["dtype"]])[:, : c["n"]]
    else:
        both = _activations(c["m"], 2 * c["f"], c["dtype"], gen)  # what one projection to gate and up gives
        s["gate"], s["up"] = both[:, : c["f"]], both[:, c["f"] :]
        s["dh"] = (torch.randn(c["m"], c["f"], generator=gen, device="cuda") * 0.1).to(DTYPES[c["dtype"]])
    return s


def _handle(parts):
    """The matrix as a program keeps it: the checkpoint's arrays, or the library's matrix made from them once."""
    if not own:
        return parts
    import dense_fp32_gemm_03_gb300 as sg
    return sg.int8_matrix(*parts)


# ---------------------------------------------------------------------------------------------------------- plain forms
def _quantise(x):
    """(integers, scales) of the rows of x.  The quotient is taken in 64 bits, where no rounding leads across a tie."""
    s = (x.float().abs().amax(-1) / 127.0).clamp(min=2.0**-126)
    return torch.round(x.double() / s.double()[:, None]).to(torch.int8), s


def _keep(x):
    """(integers, units) of the blocks of the rows of x: tokens x blocks x 32 and tokens x blocks x 1."""
    b = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 7, -126).clamp(min=-24 if x.dtype == torch.float16 else -126)
    u = torch.ldexp(torch.ones_like(top), e)
    return torch.round(b / u).clamp(-127, 127).to(torch.int8), u


def _kept(q, u, cols):
    """The values that a checkpoint's integers stand for, in 32 bits (exact)."""
    return (q.float() * u).flatten(-2)[..., :cols]


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def run(s):
    if own:
        import dense_fp32_gemm_03_gb300 as sg
        if s["op"] == "product":
            return sg.int8_gemm(s["a"], s["b"], out_dtype=s["out"])
        if s["op"] == "linear":
            return sg.int8_linear(s["x"], s["w"])
        if s["op"] == "gradient":
            return sg.int8_weight_grad(s["dy"], sg.int8_checkpoint(s["x"]))
        h, kept = sg.int8_swiglu(s["gate"], s["up"])
        dgate, dup = sg.int8_swiglu_backward(s["dh"], kept)
        return {"h": h, "dgate": dgate, "dup": dup}
    if s["op"] == "product":
        (a, sa), (b, sb) = s["a"], s["b"]
        return ((a.float() @ b.float().t()) * sa[:, None] * sb).to(s["out"])
    if s["op"] == "linear":
        (a, sa), (b, sb) = _quantise(s["x"]), s["w"]
        return ((a.float() @ b.float().t()) * sa[:, None] * sb).to(s["x"].dtype)
    if s["op"] == "gradient":
        return (s["dy"].float().t() @ _kept(*_keep(s["x"]), s["x"].shape[1])).to(s["dy"].dtype)
    dtype, cols = s["gate"].dtype, s["gate"].shape[1]
    g, u = s["gate"].float(), s["up"].float()
    h = g * _sigmoid(g) * u
    g, u, d = _kept(*_keep(s["gate"]), cols), _kept(*_keep(s["up"]), cols), s["dh"].float()
    p = _sigmoid(g)
    return {"h": h.to(dtype), "dgate": (d * u * p * (1.0 + g * (1.0 - p))).to(dtype), "dup": (d * g * p).to(dtype)}


def work(case):
    """Each input read once, each output written once; two operations a product term.  A checkpoint is written and read: an
    integer a value, and 16 bits a block of 32."""
    c = case
    size = {"float32": 4, "bfloat16": 2, "float16": 2}[c.get("dtype", c.get("out"))]
    kept = 1 + 2 / BLOCK
    if c["op"] in ("product", "linear"):
        m, n, k = c["m"], c["n"], c["k"]
        a = m * k + 4 * m if c["op"] == "product" else m * k * size
        return {"bytes": a + n * k + 4 * n + m * n * size, "flops": 2 * m * n * k}
    if c["op"] == "gradient":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": m * k * size + 2 * kept * m * k + m * n * size + n * k * size, "flops": 2 * m * n * k}
    m, f = c["m"], c["f"]
    return {"bytes": 6 * m * f * size + 4 * kept * m * f, "flops": 20 * m * f}


# -------------------------------------------------------------------------------------------------------- in 64 bits
def _nearest(v):
    """The nearest integer, ties to even."""
    low = torch.floor(v)
    gap = v - low
    return torch.where((gap > 0.5) | ((gap == 0.5) & (low % 2 != 0)), low + 1, low)


def _integers64(x):
    """(integers, scales) of rows; the scale is the 32-bit number that the definition has."""
    s = torch.clamp((x.abs().max(-1, keepdim=True)[0].float() / 127).double(), min=2.0**-126)
    return _nearest(x.double() / s), s


def _exponent(v):
    """The largest e with 2^e <= v (taken from the number's bits: a logarithm may be an ulp short at a power of two)."""
    return torch.where(v > 0, ((v.view(torch.int64) >> 52) - 1023).double(), -1023.0)


def _kept64(x):
    low, cols = (-24.0 if x.dtype == torch.float16 else -126.0), x.shape[-1]
    x = torch.cat((x.double(), x.new_zeros(x.shape[0], -cols % BLOCK, dtype=torch.float64)), -1)
    x = x.reshape(x.shape[0], -1, BLOCK)
    unit = torch.exp2(torch.clamp(_exponent(x.abs().max(-1, keepdim=True)[0]) - 6, min=low))
    return (_nearest(x / unit).clamp(-127, 127) * unit).reshape(x.shape[0], -1)[:, :cols]


def exact(case, seed):
    s = _exact_state(case, seed)
    if s["op"] == "product":
        (a, sa), (b, sb) = s["a"], s["b"]
        return torch.einsum("mk,nk->mn", a.double(), b.double()) * sa.double()[:, None] * sb.double()[None, :]
    if s["op"] == "linear":
        (a, sa), (b, sb) = _integers64(s["x"]), s["w"]
        return torch.einsum("mk,nk->mn", a, b.double()) * sa * sb.double()[None, :]
    if s["op"] == "gradient":
        return torch.einsum("mn,mk->nk", s["dy"].double(), _kept64(s["x"]))
    g, u, d = s["gate"].double(), s["up"].double(), s["dh"].double()
    out = {"h": g * torch.sigmoid(g) * u}
    g, u = _kept64(s["gate"]), _kept64(s["up"])
    p = torch.sigmoid(g)
    out["dgate"] = d * u * (p + g * p * torch.sigmoid(-g))
    out["dup"] = d * g * p
    return out


def _exact_state(case, seed):
    """The same inputs in the checkpoint's form, whatever `own` says."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was
