"""GPU tests of the 4-bit operators where their arithmetic is hardest: values far from usual, non-finite weights, streams.

Tolerances, derived from the definitions in ``include/fp4.h``:

* the experts' layer keeps x and h to 2^-25 (32 bits), 2^-19 (float16) or 2^-16 (bfloat16) of a block's largest value in the
  mean; a block's largest value is about twice its root mean square, and x enters twice, h once, so y is within 2e-7,
  1e-5 or 8e-5 in the 2-norm, and below that where the blocks' largest values are the usual ones.  Its 32-bit sums are
  off by a few 2^-24 of their partial sums, which a pre-activation g away from zero turns into a relative error of h of a
  few |g| 2^-24: 3e-6 at |g| = 16.  So 5e-6 in 32 bits; with a 16-bit output the half unit of the type decides, at most
  2^-9 or 2^-12 of a value in the mean, and 2^-8 or 2^-10 leaves room;
* two results whose inner values differ by 3e-5 (2^-16 in the mean, three times) round to different bfloat16 numbers where a
  rounding boundary lies between them: for 3e-5 / 2^-8 = 0.8 % of the outputs, and a few times that counting the small ones.
  3 % is the limit.
"""
import numpy as np
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg

import fp4_ref as ref
from test_fp4_gpu import DTYPES, FORMATS, _built, _status, check_product, gen, host_factor   # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def stored(x, fmt):
    """(library matrix, 64-bit values) of a float32 tensor quantised by the plain implementation."""
    g = (x.abs().amax() / 2688).reshape(1) if fmt == "nvfp4" else None
    codes, scales = ref.quantize(x.cpu().numpy(), fmt, host_factor(g))
    q = sg.fp4_matrix(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales.astype(np.uint8)).cuda(),
                      fmt, cols=x.shape[1], scale=g)
    return q, ref.values(codes, scales, fmt, host_factor(g))


# ----------------------------------------------------- precision of the layer
E, D, F, TOP = 4, 2048, 192, 2


def layer_inputs(kind, tokens):
    """x, router, gate-and-up and down weights whose h lies far from what the norms of x and of the weights suggest."""
    x = torch.randn(tokens, D, generator=gen(1), device="cuda")
    up = torch.randn(E, 2 * F, D, generator=gen(2), device="cuda") / D ** 0.5
    down = torch.randn(E, D, F, generator=gen(3), device="cuda") / F ** 0.5
    router = torch.randn(E, D, generator=gen(4), device="cuda") / D ** 0.5
    if kind == "one large row":          # of an expert: its h is large, or next to zero where the gate is negative
        up[:, 5] *= 30
        up[:, F + 5] *= 30
        x[:, :] += 0.5
        up[:, 5] -= up[:, 5].mean(-1, keepdim=True) + 30 * 0.5 / D ** 0.5
    elif kind.startswith("gates"):       # pre-activations around a negative number
        x += 1
        up[:, :F] -= (up[:, :F].sum(-1, keepdim=True) + float(kind.split()[1])) / D
    elif kind == "ignored channels":     # large channels that the weights do not look at
        x[:, 64:96] *= 1000
        up[:, :, 64:96] = 0
        router[:, 64:96] = 0
    elif kind == "aligned":              # x along a row of the weights: h as large as the norms allow
        x[0] = up[0, 3] * 40
        up[:, F + 3] = up[:, 3]
    elif kind == "small":
        x *= 1e-4
    elif kind == "tokens apart":         # one token's h says nothing about another's
        x *= torch.logspace(-6, 1, tokens, device="cuda")[:, None]
    return x, router, up.reshape(E * 2 * F, D), down.reshape(E * D, F)


KINDS = ("normal", "one large row", "gates 6", "gates 12", "gates 16", "ignored channels", "aligned", "small", "tokens apart")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
def test_layer_precision(kind, dtype, fmt):
    x, router, up, down = layer_inputs(kind, 3)
    x = x.to(dtype)
    (qu, uv), (qd, dv) = stored(up, fmt), stored(down, fmt)
    y, ids, p = sg.fp4_moe(x, router, sg.fp4_experts(qu, qd, E), TOP, return_routing=True)
    wy, wids, wp = ref.moe(ref.as_numpy(x), ref.as_numpy(router), uv.reshape(E, 2 * F, D), dv.reshape(E, D, F), TOP, True)
    assert np.array_equal(ids.cpu().numpy(), wids)
    limit = {torch.float32: 5e-6, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}[dtype]
    got = ref.as_numpy(y)
    scale = np.linalg.norm(wy, axis=1)
    if dtype == torch.float16:           # its subnormal numbers are 2^-24 apart
        scale = np.maximum(scale, 2.0 ** -24 * D ** 0.5 / limit)
    off = np.linalg.norm(got - wy, axis=1) / scale
    assert off.max() <= limit, f"{kind}: relative errors {off}"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ("normal", "gates 12"))
def test_layer_16_bit_activations_lose_their_output_rounding_only(kind, fmt):
    """The same bfloat16 values as bfloat16 and as float32: the outputs differ where a rounding boundary lies between."""
    x, router, up, down = layer_inputs(kind, 16)
    x = x.bfloat16()
    w = sg.fp4_experts(stored(up, fmt)[0], stored(down, fmt)[0], E)
    y, wide = sg.fp4_moe(x, router, w, TOP), sg.fp4_moe(x.float(), router, w, TOP)
    assert float((y != wide.bfloat16()).float().mean()) <= 0.03


def test_layer_zero_tokens_beside_others():
    """Tokens without any h (x of zeros: padding) leave the others' precision alone."""
    x, router, up, down = layer_inputs("gates 12", 5)
    x[1] = x[4] = 0
    (qu, uv), (qd, dv) = stored(up, "nvfp4"), stored(down, "nvfp4")
    y = sg.fp4_moe(x, router, sg.fp4_experts(qu, qd, E), TOP)
    wy, _, _ = ref.moe(ref.as_numpy(x), ref.as_numpy(router), uv.reshape(E, 2 * F, D), dv.reshape(E, D, F), TOP, True)
    assert bool((y[1] == 0).all()) and bool((y[4] == 0).all())
    keep = [0, 2, 3]
    off = np.linalg.norm(ref.as_numpy(y)[keep] - wy[keep], axis=1) / np.linalg.norm(wy[keep], axis=1)
    assert off.max() <= 5e-6


# ---------------------------------------------------------------- quantisation
def huge_beside_small():
    """Finite blocks with both signs from 1 to the largest numbers of 32 bits."""
    x = torch.randn(9, 96, generator=gen(11), device="cuda")
    for i, s in enumerate((1.0, 1e10, 1e20, 1e30, 1e37, 5e37, 5e37, 1e25, 1e5)):
        x[i, 16:64] *= s
    x[5, 70], x[5, 71] = 3.4e38, -3.4e38
    x[6] = 3.4e38 * torch.sign(x[6])
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [0.01, 1.0, 1e-12, 2.0 ** -90, 2.0 ** -101, 1e-35, 1e30])
def test_values_far_above_the_factor_saturate(g, dtype):
    """a / (6 g) beyond 32 bits: the largest scale, and codes of 6 with the values' signs."""
    x = huge_beside_small().clamp(-3.3e38, 3.3e38).to(dtype)
    g = torch.tensor([g], device="cuda")
    codes, scales, _ = ref.read_codes(sg.fp4_quantize(x, "nvfp4", scale=g))
    want_codes, want_scales = ref.quantize(ref.as_numpy(x), "nvfp4", g.item())
    assert want_scales.max() <= 126
    assert np.array_equal(scales, want_scales) and np.array_equal(codes, want_codes)


@pytest.mark.parametrize("m", [2, 100])
def test_linear_of_values_far_above_the_factor(m):
    w, wv = stored(torch.randn(70, 96, generator=gen(12), device="cuda"), "nvfp4")
    x = huge_beside_small()[3:5].repeat(m // 2, 1)
    g = torch.tensor([2.0 ** -90], device="cuda")
    codes, scales = ref.quantize(ref.as_numpy(x), "nvfp4", g.item())
    check_product(sg.fp4_linear(x, w, x_scale=g), ref.values(codes, scales, "nvfp4", g.item()), wv, f"saturated {m}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_zeros_keep_their_sign(dtype, fmt):
    """-0, and negative values that round to zero, have the code of -0 beside values of any size."""
    x = torch.randn(6, 64, generator=gen(13), device="cuda")
    x[:, ::3] = -0.0
    x[:, 1::6] = 0.0
    x[0, 5], x[0, 6] = -1e-7, 1e-7
    x[1, 5] = -1e-40
    x[2] *= 1e4
    x[3] *= 1e-4
    x = x.to(dtype)
    g = (x.abs().amax().float() / 2688).reshape(1) if fmt == "nvfp4" else None
    q = sg.fp4_quantize(x, fmt, scale=g)
    codes, scales, _ = ref.read_codes(q)
    want_codes, want_scales = ref.quantize(ref.as_numpy(x), fmt, host_factor(g))
    assert np.array_equal(scales, want_scales) and np.array_equal(codes, want_codes)
    # (A block whose unit is 0 has zero codes by definition.)
    assert np.array_equal(torch.signbit(q.dequantize()).cpu().numpy(), want_codes > 7)


# -------------------------------------------------------- non-finite weights
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("where", ("down", "gate and up"))
def test_nan_weights_reach_the_tokens_of_their_expert_only(where, dtype, fmt):
    """Token 0 goes to experts 0 and 1, token 1 to 1 and 2, token 2 to 2 and 3; NaN blocks are in experts 0 and 3."""
    experts, d, f = 5, 200, 300
    up = torch.randn(experts, 2 * f, d, generator=gen(21), device="cuda") / d ** 0.5
    down = torch.randn(experts, d, f, generator=gen(22), device="cuda") / f ** 0.5
    if where == "down":
        down[0, 5, 0] = down[0, 130, 299] = down[3, 199, 256] = float("nan")
        down[1, 7, 16:64] = -0.0            # blocks of -0 with the scale 0 are not NaN
        down[2, :, :] *= torch.where(torch.arange(f, device="cuda") < 32, -0.0, 1.0)
    else:
        up[0, 17, 3] = up[3, f + 299, 199] = float("nan")
    (qu, uv), (qd, dv) = stored(up.reshape(-1, d).nan_to_num(7.0), fmt), stored(down.reshape(-1, f).nan_to_num(7.0), fmt)
    for q, v, t in ((qu, uv, up.reshape(-1, d)), (qd, dv, down.reshape(-1, f))):   # a NaN scale for the marked blocks
        n = ref.BLOCK[fmt]
        codes, scales, _ = ref.read_codes(q)
        for r, c in torch.isnan(t).nonzero().tolist():
            scales[r, c // n] = 255 if fmt == "mxfp4" else 127
            v[r, c // n * n: c // n * n + n] = np.nan
        if bool(torch.isnan(t).any()):
            fresh = sg.fp4_matrix(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales.astype(np.uint8)).cuda(),
                                  fmt, cols=t.shape[1], scale=q.scale)
            if t.shape[1] == d:
                qu = fresh
            else:
                qd = fresh
    x = torch.randn(4, d, generator=gen(23), device="cuda").to(dtype)
    router = torch.zeros(experts, d, device="cuda")
    basis = torch.linalg.pinv(x.float())                        # logits of the tokens as wanted
    wanted = torch.tensor([[5, 4, 1, 0, -1], [0, 4, 5, 1, -1], [0, 1, 4, 5, -1], [-1, 4, 0, 1, 5]], device="cuda")
    router[:] = (basis @ wanted.float()).t()
    y, ids, p = sg.fp4_moe(x, router, sg.fp4_experts(qu, qd, experts), 2, return_routing=True)
    with np.errstate(invalid="ignore"):
        wy, wids, _ = ref.moe(ref.as_numpy(x), ref.as_numpy(router), uv.reshape(experts, 2 * f, d),
                              dv.reshape(experts, d, f), 2, True)
    got = ref.as_numpy(y)
    assert wids.tolist() == [[0, 1], [2, 1], [3, 2], [4, 1]] and np.array_equal(ids.cpu().numpy(), wids)
    assert np.isnan(wy[0]).any() and np.isnan(wy[2]).any() and np.isfinite(wy[[1, 3]]).all()
    assert np.array_equal(np.isnan(got), np.isnan(wy))
    limit = {torch.float32: 5e-6, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}[dtype]
    good = np.isfinite(wy)
    for t in range(4):
        if good[t].any():
            assert np.linalg.norm((got - wy)[t][good[t]]) <= limit * np.linalg.norm(wy[t][good[t]])


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("experts", [6, 100, 200, 300])
def test_nan_router_row_spoils_the_weights(experts, renorm):
    """A NaN among a token's logits makes its softmax NaN, whichever experts are chosen; NaN comes after every number."""
    d, f = 64, 16
    up = torch.randn(experts * 2 * f, d, generator=gen(31), device="cuda")
    down = torch.randn(experts * d, f, generator=gen(32), device="cuda")
    w = sg.fp4_experts(sg.fp4_quantize(up, "mxfp4"), sg.fp4_quantize(down, "mxfp4"), experts)
    router = torch.randn(experts, d, generator=gen(33), device="cuda")
    x = torch.randn(3, d, generator=gen(34), device="cuda")
    x[:, 5] = torch.tensor([0.0, 1.0, 2.0], device="cuda")
    router[4, 5] = float("inf")          # times 0: NaN; times a positive number: infinity
    y, ids, p = sg.fp4_moe(x, router, w, 2, renormalize=renorm, return_routing=True)
    assert bool(torch.isnan(p).all()) and bool(torch.isnan(y).all())
    assert 4 not in ids[0].tolist() and ids[1, 0] == 4 and ids[2, 0] == 4
    router[4, 5] = -float("inf")         # no weight where it is a number
    y, ids, p = sg.fp4_moe(x, router, w, 2, renormalize=renorm, return_routing=True)
    assert bool(torch.isnan(p[0]).all()) and bool(torch.isnan(y[0]).all())
    assert bool(torch.isfinite(p[1:]).all()) and bool(torch.isfinite(y[1:]).all()) and 4 not in ids[1:].flatten().tolist()


# ------------------------------------------------------------------- streams
def test_inputs_may_be_dropped_behind_a_call_on_another_stream():
    """Memory that a call on another stream still reads is not given out again: everything is dropped and overwritten
    while that stream is held up."""
    experts, d, f = 4, 256, 128
    s = torch.cuda.Stream()

    def inputs():
        up, down = (torch.randn(r, c, generator=gen(41 + c), device="cuda") for r, c in ((experts * 2 * f, d), (experts * d, f)))
        x, router = torch.randn(40, d, generator=gen(42), device="cuda"), torch.randn(experts, d, generator=gen(43), device="cuda")
        codes = torch.randint(0, 256, (300, d // 2), generator=gen(44), device="cuda", dtype=torch.uint8)
        scales = torch.randint(30, 90, (300, d // 16), generator=gen(45), device="cuda", dtype=torch.uint8)
        q = [sg.fp4_quantize(t, "nvfp4", scale=torch.full((1,), 0.01, device="cuda")) for t in (up, down)]
        return [x, router, codes, scales, torch.full((1,), 0.02, device="cuda"), *q]

    def calls(stream, x, router, codes, scales, factor, up, down):
        w = sg.fp4_experts(up, down, experts, stream=stream)
        m = sg.fp4_matrix(codes, scales, "nvfp4", scale=factor, stream=stream)
        xq = sg.fp4_quantize(x, "nvfp4", scale=factor, stream=stream)
        return [w.gate_up, w.down, sg.fp4_dequantize(m, stream=stream), sg.fp4_linear(x, m, x_scale=factor, stream=stream),
                sg.fp4_gemm(xq, m, stream=stream), sg.fp4_dequantize(up, stream=stream),
                sg.fp4_moe(x[:5], router, w, 2, stream=stream)]

    for _ in range(2):   # the second time every workspace is there
        args = inputs()
        torch.cuda.synchronize()
        want = calls(None, *args)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000_000)   # about a tenth of a second
        got = calls(s, *args)
        sizes = [t.untyped_storage().nbytes() for t in args[:5]] + [q._memory.untyped_storage().nbytes() for q in args[5:]]
        del args
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del junk


def test_tensors_that_the_library_has_addresses_of_stay():
    """Assigning another factor would leave the library with the address of the first, whose memory may be gone."""
    one, two = torch.ones(1, device="cuda"), torch.full((1,), 2.0, device="cuda")
    q = sg.fp4_quantize(torch.randn(64, 64, generator=gen(51), device="cuda"), "nvfp4", scale=one)
    before = q.dequantize()
    with pytest.raises(AttributeError):
        q.scale = two
    w = sg.fp4_experts(q, sg.fp4_quantize(torch.randn(64, 32, generator=gen(52), device="cuda"), "nvfp4", scale=one), 1)
    for name in ("gate_up", "down", "gate_up_scale", "down_scale"):
        with pytest.raises(AttributeError):
            setattr(w, name, two)
    assert q.scale is one and w.gate_up_scale is one
    one.fill_(2)                      # a write into the factor counts
    assert torch.equal(q.dequantize(), 2 * before)


# ------------------------------------------------------------------- factors
@pytest.mark.parametrize("ga,gb", [(1e-30, 1e35), (1e35, 1e-30), (1e-37, 1e-3), (1e-20, 1e-20), (1e34, 1e34), (0.0, 1e35)])
@pytest.mark.parametrize("m,n,k", [(1, 200, 600), (9, 300, 5000), (40, 130, 256), (200, 300, 256), (2100, 2500, 128)])
def test_factors_far_apart(m, n, k, ga, gb):
    """Sums are multiplied by both factors without leaving the range of 32 bits on the way."""
    rng = np.random.default_rng(m)

    def side(rows, g):
        codes, scales = rng.integers(0, 16, (rows, k)), rng.integers(40, 70, (rows, -(-k // 16)))
        t = torch.tensor([g], device="cuda")
        q = sg.fp4_matrix(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales.astype(np.uint8)).cuda(), "nvfp4",
                          cols=k, scale=t)
        return q, ref.values(codes, scales, "nvfp4", t.item())
    (a, av), (b, bv) = side(m, ga), side(n, gb)
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    got = ref.as_numpy(sg.fp4_gemm(a, b))
    fits = size < 3e38                       # beyond, the result is infinite or not, as the sums fall
    bound = (k + 4) * 2.0 ** -23 * size + 2.0 ** -149
    assert np.all(np.abs(got - want)[fits] <= bound[fits])
    # The linear layer: x holds exactly what its codes stand for at this factor.
    if ga and np.abs(av).max() < 3e38 and np.abs(av)[av != 0].min() > 2.0 ** -120:
        x = torch.from_numpy(av).float().cuda()
        codes, scales = ref.quantize(x.cpu().numpy(), "nvfp4", ga)
        xv = ref.values(codes, scales, "nvfp4", a.scale.item())
        want, size = xv @ bv.T, np.abs(xv) @ np.abs(bv).T
        fits = size < 3e38
        got = ref.as_numpy(sg.fp4_linear(x, b, x_scale=a.scale))
        assert np.all(np.abs(got - want)[fits] <= ((k + 4) * 2.0 ** -23 * size + 2.0 ** -149)[fits])


# --------------------------------------------- paths of the kernels beyond one tile
def random_matrix(rows, cols, fmt, seed):
    """(library matrix, 64-bit values on the GPU) of random codes and scales."""
    n = ref.BLOCK[fmt]
    codes = torch.randint(0, 16, (rows, cols + cols % 2), generator=gen(seed), device="cuda", dtype=torch.uint8)
    if cols % 2:
        codes[:, -1] = 0
    low, high = (122, 130) if fmt == "mxfp4" else (40, 70)
    scales = torch.randint(low, high, (rows, -(-cols // n)), generator=gen(seed + 1), device="cuda", dtype=torch.uint8)
    q = sg.fp4_matrix(codes[:, 0::2] | codes[:, 1::2] << 4, scales, fmt, cols=cols)
    table = torch.from_numpy(np.concatenate((ref.LEVELS, -ref.LEVELS))).cuda()
    unit = torch.exp2(scales.double() - 127) if fmt == "mxfp4" else torch.from_numpy(ref.E4M3).cuda()[scales.long()]
    return q, table[codes[:, :cols].long()] * unit.repeat_interleave(n, 1)[:, :cols]


def check_sums(got, a, b, what):
    """As check_product, on the GPU."""
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    unit = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[got.dtype]
    bound = (a.shape[1] + 4) * 2.0 ** -23 * size + unit * want.abs() + (2.0 ** -24 if got.dtype == torch.float16 else 0)
    assert bool(((got.double() - want).abs() <= bound).all()), what


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [
    (16, 5120, 8192),     # clusters of 8 CTAs, three tiles each, the ring of stages goes round
    (5, 40001, 4096),     # of 4, nine tiles
    (7, 77947, 510),      # of 2, nine tiles
    (3, 160001, 200),     # single CTAs, nine tiles
    (1, 20000, 1300)])    # a part of K that some CTAs of a cluster do not have
def test_linear_of_few_tokens_over_many_tiles(m, n, k, dtype, fmt):
    w, wv = random_matrix(n, k, fmt, 61)
    x = torch.randn(m, k, generator=gen(62), device="cuda").to(dtype) / 64
    codes, scales = ref.quantize(ref.as_numpy(x), fmt)
    xv = torch.from_numpy(ref.values(codes, scales, fmt)).cuda()
    got = [sg.fp4_linear(x, w) for _ in range(10)]
    check_sums(got[0], xv, wv, f"{(m, n, k)} {fmt} {dtype}")
    assert all(torch.equal(g, got[0]) for g in got[1:])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(17, 20000, 1000), (20, 8192, 8192), (33, 40000, 520), (64, 300, 30000), (50, 4096, 4096)])
def test_linear_of_some_tokens(m, n, k, fmt):
    """Swapped tiles: more than one wave of them, and tiles that are cut over K."""
    w, wv = random_matrix(n, k, fmt, 63)
    x = torch.randn(m, k, generator=gen(64), device="cuda").bfloat16() / 64
    codes, scales = ref.quantize(ref.as_numpy(x), fmt)
    xv = torch.from_numpy(ref.values(codes, scales, fmt)).cuda()
    got = [sg.fp4_linear(x, w) for _ in range(5)]
    check_sums(got[0], xv, wv, f"{(m, n, k)} {fmt}")
    assert all(torch.equal(g, got[0]) for g in got[1:])


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("experts,top", [(64, 3), (65, 5), (100, 32), (128, 1), (129, 7), (200, 20), (256, 4)])
def test_selection_among_many_experts(experts, top, renorm):
    d, f = 96, 16
    up = torch.randn(experts * 2 * f, d, generator=gen(71), device="cuda")
    down = torch.randn(experts * d, f, generator=gen(72), device="cuda")
    (qu, uv), (qd, dv) = stored(up, "mxfp4"), stored(down, "mxfp4")
    router = torch.randint(-1, 2, (experts, d), generator=gen(73), device="cuda").float()   # equal logits, exact sums
    router[experts - 1] = router[experts // 3]
    x = torch.randint(-2, 3, (5, d), generator=gen(74), device="cuda").float() / 8
    y, ids, p = sg.fp4_moe(x, router, sg.fp4_experts(qu, qd, experts), top, renormalize=renorm, return_routing=True)
    wy, wids, wp = ref.moe(ref.as_numpy(x), ref.as_numpy(router), uv.reshape(experts, 2 * f, d), dv.reshape(experts, d, f),
                           top, renorm)
    assert np.array_equal(ids.cpu().numpy(), wids)
    assert np.allclose(ref.as_numpy(p), wp, rtol=2e-5, atol=0)
    assert (np.linalg.norm(ref.as_numpy(y) - wy, axis=1) <= 1e-5 * np.linalg.norm(wy, axis=1)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols,pad", [(37, 290, 1), (37, 290, 3), (5, 1025, 2), (3, 40, 5)])
def test_values_read_back_into_rows_at_any_address(rows, cols, pad, fmt, dtype):
    q, _ = random_matrix(rows, cols, fmt, 81)
    if fmt == "nvfp4":
        g = torch.tensor([0.0371], device="cuda")
        codes, scales, _ = ref.read_codes(q)
        q = sg.fp4_matrix(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales.astype(np.uint8)).cuda(), fmt,
                          cols=cols, scale=g)
    codes, scales, _ = ref.read_codes(q)
    unit = ref.values(np.full((rows, cols), 2), scales, fmt).astype(np.float32)
    if fmt == "nvfp4":
        unit = unit * np.float32(0.0371)
    level = (ref.LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)).astype(np.float32)
    out = torch.full((rows, cols + 7), 5.0, device="cuda", dtype=dtype)
    sg.fp4_dequantize(q, out=out[:, pad:pad + cols])
    assert torch.equal(out[:, pad:pad + cols].cpu(), torch.from_numpy(level * unit).to(dtype))
    assert bool((out[:, :pad] == 5).all()) and bool((out[:, pad + cols:] == 5).all())
