"""GPU tests of the microscaled 4-bit operators against a plain 64-bit implementation (``fp4_ref``).

Tolerances, derived from the definitions:

* quantisation has none: codes and scale bytes are equal, and values read back
  in 32 bits are one rounding of code * unit;
* a product with 32-bit sums of K terms in any order, each addition off by at
  most one unit in the last place, is within K 2^-23 sum |a b| (+ two roundings
  by the factors); sums of small integers are exact; a 16-bit output adds half
  a unit, at most 2^-8 (bfloat16) or 2^-11 (float16) of the value;
* the experts' layer: its dot products are within (K 2^-23 + 2^-21) sum |a b| for
  32-bit activations, so about 1e-6 in the 2-norm and 1e-5 with room; with
  16-bit activations h carries 2^-12 and the output half a unit, at most 2^-8 or
  2^-11 of a value and about half of that in the 2-norm, so that one is within
  2^-8 (bfloat16) or 2^-10 (float16).
"""
import numpy as np
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg

import fp4_ref as ref

pytestmark = pytest.mark.gpu

FORMATS = ("mxfp4", "nvfp4")
DTYPES = (torch.float32, torch.bfloat16, torch.float16)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(autouse=True)
def _status():
    yield
    torch.cuda.synchronize()
    assert sg.query_device_status() == (0, 0)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(rows, cols, seed, dtype=torch.float32, spread=True):
    x = torch.randn(rows, cols, generator=gen(seed), device="cuda")
    if spread:   # blocks of very different magnitudes
        x = x * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=gen(seed + 1), device="cuda").float())
    return x.to(dtype)


def factor_of(x, fmt):
    return (x.abs().amax().float() / 2688).reshape(1) if fmt == "nvfp4" else None


def host_factor(g):
    return 1.0 if g is None else g.item()


def made(rows, cols, fmt, seed):
    """(library matrix, 64-bit values): normal weights quantised by the plain implementation."""
    x = torch.randn(rows, cols, generator=gen(seed), device="cuda") if rows and cols else torch.zeros(rows, cols)
    g = factor_of(x, fmt).cuda() if fmt == "nvfp4" and x.numel() else None
    codes, scales = ref.quantize(x.cpu().numpy(), fmt, host_factor(g))
    q = sg.fp4_matrix(torch.from_numpy(ref.packed(codes)).cuda(), torch.from_numpy(scales.astype(np.uint8)).cuda(),
                      fmt, cols=cols, scale=g)
    return q, ref.values(codes, scales, fmt, host_factor(g))


# ------------------------------------------------------------- quantisation
SHAPES = [(1, 1), (1, 32), (3, 31), (2, 33), (130, 257), (16, 4096), (257, 100), (5, 5003), (129, 16)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_and_scales_are_exact(rows, cols, dtype, fmt):
    x = normal(rows, cols, rows * 7 + cols, dtype)
    g = factor_of(x, fmt)
    q = sg.fp4_quantize(x, fmt, scale=g)
    codes, scales, clean = ref.read_codes(q)
    want_codes, want_scales = ref.quantize(ref.as_numpy(x), fmt, host_factor(g))
    assert np.array_equal(scales, want_scales)
    assert np.array_equal(codes, want_codes)
    assert clean, "padding is not zero"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_strided_rows(pad, dtype, fmt):
    wide = normal(37, 300 + pad, 5, dtype)
    x = wide[:, pad:pad + 290]
    g = factor_of(x, fmt)
    codes, scales, _ = ref.read_codes(sg.fp4_quantize(x, fmt, scale=g))
    want_codes, want_scales = ref.quantize(ref.as_numpy(x), fmt, host_factor(g))
    assert np.array_equal(codes, want_codes) and np.array_equal(scales, want_scales)
    out = torch.full((37, 300 + pad), 7.0, device="cuda", dtype=dtype)
    sg.fp4_dequantize(sg.fp4_quantize(x, fmt, scale=g), out=out[:, pad:pad + 290])
    want = torch.from_numpy(ref.values(want_codes, want_scales, fmt, host_factor(g))).float().to(dtype)
    if fmt == "mxfp4" or dtype != torch.float32:
        assert torch.equal(out[:, pad:pad + 290].cpu(), want)
    assert bool((out[:, :pad] == 7).all()) and bool((out[:, pad + 290:] == 7).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_ties_and_saturation(fmt):
    """Every midpoint between two levels, and values above the largest, at units that are powers of two."""
    base = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 0.5, 5.5, 7, 7.9, 0.2, 0.3, 0, 1], dtype=np.float32)
    base = np.concatenate((base, -base))
    rows = [base * np.float32(2.0 ** s) for s in (-20, -3, 0, 5)]
    if fmt == "nvfp4":   # a factor of one: the scale is largest / 6 in eight bits
        rows = [np.minimum(np.abs(r), 6 * 2.0 ** s).astype(np.float32) * np.sign(r)
                for r, s in zip(rows, (-20, -3, 0, 5))]
    x = np.stack(rows).astype(np.float32)
    codes, scales, _ = ref.read_codes(sg.fp4_quantize(torch.from_numpy(x).cuda(), fmt))
    want = ref.quantize(x, fmt)
    assert np.array_equal(scales, want[1]) and np.array_equal(codes, want[0])


@pytest.mark.parametrize("fmt", FORMATS)
def test_extremes(fmt):
    """Zeros, subnormals, the largest values; NaN and infinities spoil their block alone."""
    x = torch.zeros(8, 96)
    x[1] = 1e-42
    x[2] = 3.0e38
    x[3, 40] = float("nan")
    x[4, 0] = float("inf")
    x[5, 95] = -float("inf")
    x[3:6, 50] = 2.0
    x[6, ::2] = -0.0
    x[7] = torch.linspace(-3e-39, 3e-39, 96)
    q = sg.fp4_quantize(x.cuda(), fmt)
    codes, scales, _ = ref.read_codes(q)
    want = ref.quantize(x.numpy(), fmt)
    n = ref.BLOCK[fmt]
    assert np.array_equal(scales, want[1])
    fine = np.repeat(np.isfinite(x.numpy()).reshape(8, -1, n).all(-1), n, axis=1)
    assert np.array_equal(codes[fine], want[0][fine])
    y = q.dequantize().cpu().numpy()
    assert np.isnan(y[~fine]).all() and np.isfinite(y[fine]).all()


def test_zero_factor_gives_zeros():
    x = torch.zeros(2, 64, device="cuda")
    q = sg.fp4_quantize(x, "nvfp4", scale=torch.zeros(1, device="cuda"))
    assert bool((q.dequantize() == 0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 333), (130, 512)])
def test_checkpoint_arrays_and_values(rows, cols, dtype, fmt):
    q, v = made(rows, cols, fmt, 11)
    codes, scales, clean = ref.read_codes(q)
    assert clean
    # The definition's operations in 32 bits (the unit, the value), then one rounding to the output type.
    g = host_factor(q.scale)
    unit = ref.values(np.full((rows, cols), 2), scales, fmt, 1.0).astype(np.float32)
    if fmt == "nvfp4":
        unit = unit * np.float32(g)
    level = (ref.LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)).astype(np.float32)
    want = torch.from_numpy(level * unit)
    assert torch.equal(sg.fp4_dequantize(q, dtype).cpu(), want.to(dtype))
    assert np.all(np.abs(want.double().numpy() - v) <= 2.0 ** -23 * np.abs(v))


def test_strided_checkpoint_arrays():
    codes = np.random.default_rng(1).integers(0, 16, (50, 75))
    scales = np.random.default_rng(2).integers(100, 140, (50, 3))
    a = torch.zeros(50, 41, dtype=torch.uint8, device="cuda")
    a[:, 2:40] = torch.from_numpy(ref.packed(codes)).cuda()
    a[:, 39] |= 0xf0   # the unused half of the last byte
    s = torch.zeros(50, 8, dtype=torch.uint8, device="cuda")
    s[:, 1:4] = torch.from_numpy(scales.astype(np.uint8)).cuda()
    q = sg.fp4_matrix(a[:, 2:40], s[:, 1:4], "mxfp4", cols=75)
    got = ref.read_codes(q)
    assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales) and got[2]


@pytest.mark.parametrize("rows,cols", [(0, 5), (5, 0), (0, 0)])
def test_empty_matrices(rows, cols):
    x = torch.zeros(rows, cols, device="cuda")
    assert tuple(sg.fp4_quantize(x, "mxfp4").dequantize().shape) == (rows, cols)


# ------------------------------------------------------------------ products
def check_product(got, a, b, what, exact=False):
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    err = np.abs(ref.as_numpy(got) - want)
    unit = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[got.dtype]
    bound = (0 if exact else (a.shape[1] + 4) * 2.0 ** -23) * size + unit * np.abs(want) + (2.0 ** -24 if got.dtype == torch.float16 else 0)
    assert np.isfinite(ref.as_numpy(got)).all(), f"{what}: not finite"
    assert np.all(err <= bound), f"{what}: off by {(err - bound).max():.3g} more than the bound"


PRODUCTS = [(1, 1, 1), (1, 8, 32), (2, 130, 64), (17, 33, 65), (128, 256, 256), (129, 257, 300), (300, 520, 200),
            (256, 256, 512), (33, 4096, 1024), (700, 40, 2049), (512, 768, 1536), (1, 1000, 5000), (16, 640, 4096),
            (2048, 300, 96), (100, 128, 40000), (3, 200, 60000), (2600, 2100, 300)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k, fmt):
    (a, av), (b, bv) = made(m, k, fmt, 3), made(n, k, fmt, 4)
    for dtype in DTYPES:
        check_product(sg.fp4_gemm(a, b, out_dtype=dtype), av, bv, f"{(m, n, k)} {fmt} {dtype}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(2000, 2504, 4000), (4100, 3801, 4000), (1400, 3500, 3100), (2500, 3501, 100),
                                   (2561, 3500, 64)])
def test_product_of_many_tiles(m, n, k, fmt):
    """Pairs of CTAs with 128 and with 256 columns a tile, rows that TMA stores and rows that it does not."""
    (a, av), (b, bv) = made(m, k, fmt, 3), made(n, k, fmt, 4)
    for dtype in DTYPES:
        check_product(sg.fp4_gemm(a, b, out_dtype=dtype), av, bv, f"{(m, n, k)} {fmt} {dtype}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(128, 256, 256), (130, 300, 700), (5, 260, 4096), (1024, 512, 1024)])
def test_integer_products_are_exact(m, n, k, fmt):
    """Codes that stand for integers times powers of two, every block with a scale of its own."""
    rng = np.random.default_rng(m + n + k)
    n_blk = -(-k // ref.BLOCK[fmt])

    def side(rows):
        codes = rng.choice([0, 2, 4, 5, 6, 7, 10, 12, 13, 14, 15], (rows, k))
        low = 127 if fmt == "mxfp4" else 56
        step = 1 if fmt == "mxfp4" else 8
        scales = low + step * rng.integers(0, 3, (rows, n_blk))
        q = sg.fp4_matrix(torch.from_numpy(ref.packed(codes)).cuda(),
                          torch.from_numpy(scales.astype(np.uint8)).cuda(), fmt, cols=k)
        return q, ref.values(codes, scales, fmt)
    (a, av), (b, bv) = side(m), side(n)
    assert (np.abs(av) @ np.abs(bv).T).max() < 2 ** 24
    check_product(sg.fp4_gemm(a, b), av, bv, f"integers {(m, n, k)} {fmt}", exact=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [3, 40, 200])
def test_product_into_strided_output(m, fmt):
    (a, av), (b, bv) = made(m, 160, fmt, 5), made(77, 160, fmt, 6)
    for dtype in DTYPES:
        wide = torch.full((m, 90), 3.0, device="cuda", dtype=dtype)
        sg.fp4_gemm(a, b, out=wide[:, 5:82])
        check_product(wide[:, 5:82], av, bv, f"strided {dtype}")
        assert bool((wide[:, :5] == 3).all()) and bool((wide[:, 82:] == 3).all())


@pytest.mark.parametrize("m,n,k", [(0, 5, 64), (5, 0, 64), (4, 6, 0)])
def test_empty_products(m, n, k):
    a, b = (sg.fp4_quantize(torch.zeros(r, k, device="cuda"), "mxfp4") for r in (m, n))
    out = torch.full((m, n), 9.0, device="cuda")
    sg.fp4_gemm(a, b, out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_scale_reaches_its_row_only(fmt):
    x = torch.randn(140, 300, generator=gen(1), device="cuda")
    x[130, 299] = float("nan")
    a, b = sg.fp4_quantize(x, fmt), sg.fp4_quantize(torch.randn(50, 300, generator=gen(2), device="cuda"), fmt)
    c = sg.fp4_gemm(a, b)
    assert bool(torch.isnan(c[130]).all()) and bool(torch.isfinite(c[:130]).all()) and bool(torch.isfinite(c[131:]).all())
    c = sg.fp4_gemm(b, a)
    assert bool(torch.isnan(c[:, 130]).all()) and bool(torch.isfinite(c[:, :130]).all())


# -------------------------------------------------------------- linear layer
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 128, 256), (1, 4096, 1024), (2, 33, 70), (5, 200, 1000), (8, 300, 513),
                                   (16, 256, 4096), (17, 300, 256), (64, 500, 640), (100, 1000, 100), (257, 129, 2048)])
def test_linear_is_quantise_and_product(m, n, k, dtype, fmt):
    w, wv = made(n, k, fmt, 8)
    x = normal(m, k, 9, dtype, spread=False)
    g = factor_of(x, fmt)
    codes, scales = ref.quantize(ref.as_numpy(x), fmt, host_factor(g))
    xv = ref.values(codes, scales, fmt, host_factor(g))
    check_product(sg.fp4_linear(x, w, x_scale=g), xv, wv, f"linear {(m, n, k)} {fmt} {dtype}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [1, 7, 130])
def test_linear_strided(m, fmt):
    w, wv = made(100, 250, fmt, 8)
    wide = normal(m, 263, 9, torch.bfloat16, spread=False)
    x = wide[:, 3:253]
    codes, scales = ref.quantize(ref.as_numpy(x), fmt)
    out = torch.full((m, 111), 5.0, device="cuda", dtype=torch.bfloat16)
    sg.fp4_linear(x, w, out=out[:, 1:101])
    check_product(out[:, 1:101], ref.values(codes, scales, fmt), wv, "strided linear")
    assert bool((out[:, :1] == 5).all()) and bool((out[:, 101:] == 5).all())


@pytest.mark.parametrize("m", [1, 100])
def test_linear_non_finite_row(m):
    w, _ = made(64, 256, "mxfp4", 8)
    x = torch.randn(m, 256, generator=gen(3), device="cuda")
    x[0, 7] = float("inf")
    y = sg.fp4_linear(x, w)
    assert bool(torch.isnan(y[0]).all()) and bool(torch.isfinite(y[1:]).all())


@pytest.mark.parametrize("m", [1, 16])
def test_linear_longer_than_a_cluster_holds(m):
    """K beyond what one kernel keeps of x in shared memory: quantised first, then multiplied."""
    w, wv = made(130, 90000, "mxfp4", 8)
    x = normal(m, 90000, 9, torch.bfloat16, spread=False)
    codes, scales = ref.quantize(ref.as_numpy(x), "mxfp4")
    check_product(sg.fp4_linear(x, w), ref.values(codes, scales, "mxfp4"), wv, f"long {m}")


def test_no_columns_gives_zeros():
    w = sg.fp4_quantize(torch.zeros(6, 0, device="cuda"), "mxfp4")
    assert bool((sg.fp4_linear(torch.zeros(3, 0, device="cuda"), w) == 0).all())


# ----------------------------------------------------------- mixture of experts
def layer(experts, d, f, fmt, seed):
    (up, upv), (down, downv) = made(experts * 2 * f, d, fmt, seed), made(experts * d, f, fmt, seed + 1)
    router = torch.randn(experts, d, generator=gen(seed + 2), device="cuda") / d ** 0.5
    return (sg.fp4_experts(up, down, experts), router, upv.reshape(experts, 2 * f, d), downv.reshape(experts, d, f))


def check_layer(x, router, w, upv, downv, top, renorm, what):
    y, ids, p = sg.fp4_moe(x, router, w, top, renormalize=renorm, return_routing=True)
    wy, wids, wp = ref.moe(ref.as_numpy(x), ref.as_numpy(router), upv, downv, top, renorm)
    assert np.array_equal(ids.cpu().numpy(), wids), what
    assert np.allclose(ref.as_numpy(p), wp, rtol=2e-5, atol=0), what
    limit = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}[x.dtype]
    off = np.linalg.norm(ref.as_numpy(y) - wy, axis=1) / np.linalg.norm(wy, axis=1)
    assert off.max() <= limit, f"{what}: relative error {off.max():.3g}"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,experts,d,f,top,renorm", [
    (1, 4, 128, 64, 1, True), (1, 16, 256, 128, 4, True), (3, 8, 200, 72, 2, False), (5, 12, 1032, 520, 3, False),
    (8, 4, 130, 33, 4, True), (9, 64, 384, 96, 8, True), (16, 40, 512, 160, 6, False), (16, 2, 64, 8, 1, True),
    (21, 8, 256, 64, 2, True), (2, 300, 64, 16, 32, True), (4, 1, 40, 7, 1, False)])
def test_layer(tokens, experts, d, f, top, renorm, dtype, fmt):
    w, router, upv, downv = layer(experts, d, f, fmt, 20)
    x = normal(tokens, d, 30, dtype, spread=False)
    check_layer(x, router, w, upv, downv, top, renorm, f"{tokens} tokens, {experts} experts {d} x {f}")


def test_layer_scales_of_tokens_differ():
    w, router, upv, downv = layer(8, 256, 64, "nvfp4", 40)
    x = normal(6, 256, 41, spread=False) * torch.tensor([1e-6, 1e-3, 1, 30, 1e-12, 5.0], device="cuda")[:, None]
    check_layer(x, router / 30, w, upv, downv, 2, True, "scales")


def test_layer_equal_logits_take_the_lowest_index():
    w, router, upv, downv = layer(10, 64, 16, "mxfp4", 50)
    router = torch.zeros_like(router)
    router[7] = router[3] = torch.randn(64, generator=gen(1), device="cuda")
    x = normal(4, 64, 51, spread=False)
    ids = sg.fp4_moe(x, router, w, 3, return_routing=True)[1].cpu().numpy()
    logits = (ref.as_numpy(x) @ ref.as_numpy(router).T)
    want = np.array([[3, 7, 0] if l[3] > 0 else [0, 1, 2] for l in logits])
    assert np.array_equal(ids, want)


def test_layer_zero_and_non_finite_tokens():
    w, router, upv, downv = layer(6, 128, 32, "nvfp4", 60)
    x = normal(5, 128, 61, spread=False)
    x[1] = 0
    x[3, 5] = float("nan")
    y, ids, p = sg.fp4_moe(x, router, w, 2, return_routing=True)
    assert bool((y[1] == 0).all()) and ids[1].tolist() == [0, 1]
    assert bool(torch.isnan(y[3]).all()) and bool(((ids >= 0) & (ids < 6)).all())
    keep = [0, 2, 4]
    wy, _, _ = ref.moe(ref.as_numpy(x)[keep], ref.as_numpy(router), upv, downv, 2, True)
    assert np.allclose(ref.as_numpy(y)[keep], wy, rtol=0, atol=1e-5 * np.abs(wy).max())


def test_layer_strided():
    w, router, upv, downv = layer(6, 100, 32, "mxfp4", 70)
    wide = normal(4, 111, 71, spread=False)
    out = torch.full((4, 107), 2.0, device="cuda")
    big = torch.zeros(6, 105, device="cuda")
    big[:, 2:102] = router
    sg.fp4_moe(wide[:, 5:105], big[:, 2:102], w, 2, out=out[:, 3:103])
    wy, _, _ = ref.moe(ref.as_numpy(wide[:, 5:105]), ref.as_numpy(router), upv, downv, 2, True)
    assert np.allclose(ref.as_numpy(out[:, 3:103]), wy, rtol=0, atol=1e-5 * np.abs(wy).max())
    assert bool((out[:, :3] == 2).all()) and bool((out[:, 103:] == 2).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_norms_beyond_32_bits(fmt):
    """Tokens whose squares leave the range of 32 bits (their norm is bounded otherwise) keep their precision."""
    w, router, upv, downv = layer(6, 128, 64, fmt, 75)
    x = normal(4, 128, 76, spread=False) * torch.tensor([1e-17, 1e-12, 1.0, 1e16], device="cuda")[:, None]
    check_layer(x, router * 1e-17, w, upv, downv, 2, True, "norms")


def test_matrix_sizes_are_the_librarys():
    import ctypes
    from dense_fp32_gemm_03_gb300 import fp4
    for fmt, number in fp4.FORMATS.items():
        for rows, cols in ((1, 1), (128, 256), (129, 257), (1000, 5003), (0, 64)):
            q = sg.Fp4Matrix(rows, cols, fmt)
            ld, codes, scales = (ctypes.c_int64() for _ in range(3))
            assert fp4.load().fp4_layout(number, rows, cols, *map(ctypes.byref, (ld, codes, scales))) == 0
            assert q.codes.shape == (rows, ld.value) and q.codes.numel() == codes.value and q.scales.numel() == scales.value


def test_workspaces_may_be_released_between_calls():
    w, router, _, _ = layer(8, 128, 64, "nvfp4", 77)
    b, _ = made(300, 512, "nvfp4", 78)
    x, xm = normal(100, 512, 79, torch.bfloat16, spread=False), normal(3, 128, 80, spread=False)
    want = sg.fp4_linear(x, b), sg.fp4_moe(xm, router, w, 2)
    sg.release_workspaces()
    got = sg.fp4_linear(x, b), sg.fp4_moe(xm, router, w, 2)
    assert all(torch.equal(g, t) for g, t in zip(got, want))


# -------------------------------------------------------- streams and repeats
def test_results_repeat_and_streams_do_not_mix():
    """Two streams at once, many calls each: every result equals the first one bit for bit."""
    a, _ = made(300, 1000, "nvfp4", 80)
    b, _ = made(520, 1000, "nvfp4", 81)
    w, router, _, _ = layer(16, 256, 96, "mxfp4", 82)
    xs = [normal(m, 1000, 83 + m, torch.bfloat16, spread=False) for m in (1, 12, 90)]
    xm = normal(7, 256, 90, spread=False)

    def calls(stream=None):
        return [sg.fp4_gemm(a, b, stream=stream), *(sg.fp4_linear(x, b, stream=stream) for x in xs),
                sg.fp4_moe(xm, router, w, 3, stream=stream)]
    want = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [calls(streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(g, want))


def test_graph_capture():
    a, _ = made(64, 512, "mxfp4", 84)
    b, _ = made(200, 512, "mxfp4", 85)
    w, router, _, _ = layer(8, 128, 64, "mxfp4", 86)
    x, xm = normal(4, 512, 87, torch.bfloat16, spread=False), normal(3, 128, 88, torch.bfloat16, spread=False)
    s = torch.cuda.Stream()

    def calls():
        return [sg.fp4_gemm(a, b), sg.fp4_linear(x, b), sg.fp4_moe(xm, router, w, 2)]
    with torch.cuda.stream(s):
        want = [t.clone() for t in calls()]
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = calls()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, t) for g, t in zip(got, want))


# ------------------------------------------------------------------- refusals
def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    q, n = sg.fp4_quantize(x, "mxfp4"), sg.fp4_quantize(x, "nvfp4")
    one = torch.ones(1, device="cuda")
    bad = [
        (ValueError, lambda: sg.fp4_quantize(x.cpu(), "mxfp4")),
        (ValueError, lambda: sg.fp4_quantize(x.double(), "mxfp4")),
        (ValueError, lambda: sg.fp4_quantize(x, "fp4")),
        (ValueError, lambda: sg.fp4_quantize(x.t(), "mxfp4")),
        (ValueError, lambda: sg.fp4_quantize(x[0], "mxfp4")),
        (ValueError, lambda: sg.fp4_quantize(x[:1].expand(4, 64), "mxfp4")),
        (ValueError, lambda: sg.fp4_quantize(x, "mxfp4", scale=one)),
        (ValueError, lambda: sg.fp4_quantize(x, "nvfp4", scale=one.cpu())),
        (ValueError, lambda: sg.fp4_quantize(x, "nvfp4", scale=torch.ones(2, device="cuda"))),
        (ValueError, lambda: sg.fp4_quantize(x, "nvfp4", out=q)),
        (TypeError, lambda: sg.fp4_quantize("x", "mxfp4")),
        (TypeError, lambda: sg.fp4_dequantize(x)),
        (ValueError, lambda: sg.fp4_dequantize(q, torch.int32)),
        (ValueError, lambda: sg.fp4_dequantize(q, out=torch.zeros(4, 63, device="cuda"))),
        (ValueError, lambda: sg.fp4_gemm(q, n)),
        (ValueError, lambda: sg.fp4_gemm(q, sg.fp4_quantize(x[:, :32], "mxfp4"))),
        (ValueError, lambda: sg.fp4_gemm(q, q, out_dtype=torch.int8)),
        (TypeError, lambda: sg.fp4_gemm(x, q)),
        (ValueError, lambda: sg.fp4_linear(x[:, :32], q)),
        (ValueError, lambda: sg.fp4_linear(x, q, x_scale=one)),
        (ValueError, lambda: sg.fp4_linear(x, q, out=torch.zeros(4, 4, device="cuda", dtype=torch.float16))),
        (ValueError, lambda: sg.fp4_matrix(torch.zeros(4, 32, device="cuda", dtype=torch.uint8),
                                           torch.zeros(4, 1, device="cuda", dtype=torch.uint8))),
        (ValueError, lambda: sg.fp4_matrix(torch.zeros(4, 32, device="cuda"), torch.zeros(4, 2, device="cuda"))),
        (ValueError, lambda: sg.fp4_experts(q, q, 3)),
        (sg.SgemmError, lambda: sg.fp4_linear(x, q, out=x[:, :4])),   # the output overlaps x
    ]
    w, router, _, _ = layer(4, 64, 16, "mxfp4", 1)
    bad += [
        (ValueError, lambda: sg.fp4_moe(x, router, w, 0)),
        (ValueError, lambda: sg.fp4_moe(x, router, w, 5)),
        (ValueError, lambda: sg.fp4_moe(x, router[:3], w, 2)),
        (ValueError, lambda: sg.fp4_moe(x, router.half(), w, 2)),
        (ValueError, lambda: sg.fp4_moe(x[:, :32], router, w, 2)),
        (TypeError, lambda: sg.fp4_moe(x, router, q, 2)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_calls_in_a_row_share_scratch(fmt):
    """Calls of several sizes one after another on one stream: a product reads only its own call's codes of x."""
    w, _ = made(700, 1000, fmt, 21)
    xs = [torch.randn(m, 1000, generator=gen(60 + m), device="cuda") for m in (17, 300, 64, 1500, 40, 300, 129)]
    g = torch.full((1,), 2.0 ** -8, device="cuda") if fmt == "nvfp4" else None
    want = []
    for x in xs:
        want.append(sg.fp4_gemm(sg.fp4_quantize(x, fmt, scale=g), w))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [sg.fp4_linear(x, w, x_scale=g) for x in xs]
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_start_after_what_they_read():
    """Calls that may start early read what kernels, copies and other streams wrote just before, eager and in a graph."""
    w = sg.fp4_quantize(torch.randn(256, 512, generator=gen(1), device="cuda"), "mxfp4")
    src = [torch.randn(m, 512, generator=gen(m), device="cuda") for m in (4, 40, 300)]
    x = [torch.zeros_like(t) for t in src]
    other = torch.cuda.Stream()

    def chain(k):
        main = torch.cuda.current_stream()
        res = []
        for a, s in zip(x, src):
            big = torch.full((1 << 22,), float(k), device="cuda")          # keeps the GPU busy before the copy
            a.copy_(s * k + 0 * big[0])
            q = sg.fp4_quantize(a, "mxfp4")
            other.wait_stream(main)
            with torch.cuda.stream(other):
                r = sg.fp4_gemm(q, w)
                a.mul_(2)
            main.wait_stream(other)
            r.record_stream(main)
            res += [r, sg.fp4_linear(a, w), sg.fp4_dequantize(q, torch.float32)]
        return res

    def want(k):
        res = []
        for s in src:
            a = s * k
            q = sg.fp4_quantize(a, "mxfp4")
            torch.cuda.synchronize()
            r, v = sg.fp4_gemm(q, w), sg.fp4_dequantize(q, torch.float32)
            torch.cuda.synchronize()
            b = a * 2
            torch.cuda.synchronize()
            res += [r, sg.fp4_linear(b, w), v]
            torch.cuda.synchronize()
        return res
    for k in (1, 2, 3):
        for a, b in zip(chain(k), want(k)):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        res = chain(5)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(res, want(5)):
            assert torch.equal(a, b)
