"""The 8-bit integer operators against a plain implementation in 64 bits (GPU)."""
import numpy as np
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg

import int8_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def values(rows, cols, dtype, seed=0, pad=0, scale=1.0):
    """Normal values with a few large columns, `pad` columns of a wider matrix left out on the right."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=gen) * scale
    x[:, ::37] *= 8
    return x.to(dtype).cuda()[:, :cols]


def same(got, want):
    """Bit for bit, NaN for NaN."""
    got, want = got.cpu(), want.cpu()
    assert got.dtype == want.dtype and got.shape == want.shape
    torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True)


def finish():
    torch.cuda.synchronize()
    assert sg.query_device_status() == (0, 0)


# ------------------------------------------------------------------------- rows
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 7, 0), (5, 16, 3), (33, 1000, 1), (17, 1024, 8), (2, 1025, 0),
                                           (9, 8192, 0), (2, 8200, 1), (1, 40003, 0)])
def test_rows_are_quantised_bit_for_bit(dtype, rows, cols, pad):
    x = values(rows, cols, dtype, rows + cols, pad)
    q = sg.int8_quantize(x)
    codes, scales = ref.quantize(ref.array(x))
    same(q.codes, torch.from_numpy(codes))
    same(q.scales, torch.from_numpy(scales))
    for out in TYPES:
        want = codes.astype(np.float32) * scales[:, None]
        same(sg.int8_dequantize(q, out), ref.round_to(want, out))
    finish()


def test_quotients_next_to_a_tie():
    """Rows whose scale is a number of 24 bits and whose values lie on both sides of (n + 1/2) scales."""
    gen = np.random.default_rng(5)
    top = gen.uniform(1, 2, (64, 1)).astype(np.float32)
    s = top * (np.float32(1) / np.float32(127))
    n = gen.integers(-126, 126, (64, 500)) + 0.5
    x = (n * s).astype(np.float32)
    x = np.concatenate([x, np.nextafter(x, np.float32(4)), np.nextafter(x, np.float32(-4)), top], 1)
    q = sg.int8_quantize(torch.from_numpy(x).cuda())
    codes, scales = ref.quantize(x)
    same(q.codes, torch.from_numpy(codes))
    same(q.scales, torch.from_numpy(scales))


def test_exact_ties_go_to_even():
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]]).cuda()
    assert sg.int8_quantize(x).codes.tolist() == [[127, 0, 2, 2, 0, -2, -2, 126]]


def test_rows_at_the_ends_of_the_range():
    rows = [[0.0] * 5, [3.4e38, -3.4e38, 1e38, 1.0, 0.0], [1e-38, 2e-39, -1e-45, 0, 5e-39], [2.0 ** -120, 2.0 ** -126, -2.0 ** -127, 1e-45, 0],
            [float("nan"), 1, 2, 3, 4], [float("inf"), 1, 2, 3, 4], [1, 2, -float("inf"), 3, 4], [-127.0, 1, 2, 3, 4]]
    x = torch.tensor(rows)
    q = sg.int8_quantize(x.cuda())
    codes, scales = ref.quantize(x.numpy())
    same(q.codes, torch.from_numpy(codes))
    same(q.scales, torch.from_numpy(scales))
    back = q.dequantize().cpu()
    assert back[4:7].isnan().all() and back[[0, 1, 2, 3, 7]].isfinite().all()


def test_empty_matrices():
    for rows, cols in ((0, 5), (5, 0), (0, 0)):
        x = torch.empty(rows, cols, device="cuda")
        q = sg.int8_quantize(x)
        assert q.dequantize().shape == (rows, cols)
        w = sg.int8_quantize(torch.ones(3, cols, device="cuda"))
        assert sg.int8_gemm(q, w).tolist() == [[0.0] * 3] * rows
        assert sg.int8_linear(x, w).tolist() == [[0.0] * 3] * rows
        assert sg.int8_checkpoint(x).restore().shape == (rows, cols)
        h, kept = sg.int8_swiglu(x, x)
        assert h.shape == (rows, cols) and sg.int8_swiglu_backward(h, kept)[1].shape == (rows, cols)
    finish()


def test_a_checkpoints_arrays_in_place_or_copied():
    codes = torch.randint(-128, 128, (20, 64), dtype=torch.int8, device="cuda")
    scales = torch.rand(20, device="cuda")
    want = (codes.float() * scales[:, None])
    assert sg.int8_matrix(codes, scales).codes.data_ptr() == codes.data_ptr()
    for c in (codes, codes[:, :50], codes[:, 3:40], codes[1:, 16:33], codes[::2, :48], codes.t().contiguous().t(), codes[19:, 17:]):
        rows = want[:c.shape[0]] if c.shape[0] == 20 else None
        q = sg.int8_matrix(c, scales[:c.shape[0]])
        same(q.codes, c)
        same(q.dequantize(), c.float() * scales[:c.shape[0], None])
    finish()


# --------------------------------------------------------------------- products
def integers(rows, cols, seed, low=-127, high=128):
    gen = np.random.default_rng(seed)
    q = gen.integers(low, high, (rows, cols)).astype(np.int8)
    s = np.exp(gen.normal(size=rows)).astype(np.float32)
    return q, s


def matrix(q, s):
    return sg.int8_matrix(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())


SHAPES = [(1, 1, 1), (1, 16, 16), (2, 300, 33), (7, 128, 1000), (8, 129, 1024), (9, 257, 1025), (15, 40, 4096), (16, 4096, 512),
          (17, 100, 129), (31, 1000, 200), (32, 256, 2048), (33, 255, 64), (63, 520, 128), (64, 130, 3000), (65, 384, 127),
          (100, 1, 500), (127, 513, 1), (128, 128, 128), (129, 777, 1030), (256, 256, 4100), (300, 520, 200), (500, 1024, 96), (1000, 40, 2050)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products_are_exact(m, n, k):
    """Full-range integers: a sum that lost one unit anywhere would show."""
    (a, sa), (b, sb) = integers(m, k, 1), integers(n, k, 2, -128)
    for dtype in TYPES:
        same(sg.int8_gemm(matrix(a, sa), matrix(b, sb), out_dtype=dtype), ref.product(a, sa, b, sb, dtype))
    finish()


@pytest.mark.parametrize("m,n,k", [(1, 256, 131071), (40, 300, 20000), (300, 300, 20001)])
def test_sums_beyond_24_bits(m, n, k):
    """Equal signs: sums far beyond what 32-bit floats count, with neighbours one apart."""
    a, b = np.full((m, k), 127, np.int8), np.full((n, k), -128, np.int8)
    a[:, -1] = np.arange(m) % 120
    b[:, 0] = np.arange(n) % 100
    one = np.ones(max(m, n), np.float32)
    got = sg.int8_gemm(matrix(a, one[:m]), matrix(b, one[:n]))
    same(got, ref.product(a, one[:m], b, one[:n], F32))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,pad", [(1, 256, 300, 0), (2, 1000, 4096, 3), (5, 70, 1031, 0), (8, 512, 8192, 0), (16, 300, 2048, 1),
                                       (17, 256, 512, 0), (40, 129, 777, 3), (200, 300, 1024, 0), (260, 70, 4097, 1)])
def test_linear_is_quantise_and_product(dtype, m, n, k, pad):
    x = values(m, k, dtype, m + n, pad)
    b, sb = integers(n, k, n)
    w = matrix(b, sb)
    codes, scales = ref.quantize(ref.array(x))
    got = sg.int8_linear(x, w)
    same(got, ref.product(codes, scales, b, sb, dtype))
    same(got, sg.int8_gemm(sg.int8_quantize(x), w, out_dtype=dtype))
    finish()


@pytest.mark.parametrize("m", [1, 4, 20, 150])
def test_rows_that_are_not_finite_stay_apart(m):
    x = values(m + 3, 200, F32)
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    b, sb = integers(90, 200, 3)
    sb[7] = np.nan
    y = sg.int8_linear(x, matrix(b, sb)).cpu()
    assert y[1:3].isnan().all() and y[:, 7].isnan().all()
    rest = [i for i in range(m + 3) if i not in (1, 2)]
    assert y[rest][:, [j for j in range(90) if j != 7]].isfinite().all()


@pytest.mark.parametrize("m", [3, 70])
def test_scales_far_apart(m):
    (a, _), (b, _) = integers(m, 60, 4), integers(50, 60, 5)
    sa, sb = np.full(m, 1e33, np.float32), np.full(50, 1e-36, np.float32)
    sa[1], sb[3], sb[4] = 3e-38, -1e30, 0
    same(sg.int8_gemm(matrix(a, sa), matrix(b, sb)), ref.product(a, sa, b, sb, F32))


@pytest.mark.parametrize("m,n,k", [(3, 100, 64), (50, 200, 300), (257, 385, 130)])
@pytest.mark.parametrize("dtype", TYPES)
def test_strided_outputs_leave_their_surroundings(m, n, k, dtype):
    (a, sa), (b, sb) = integers(m, k, 6), integers(n, k, 7)
    around = torch.full((m + 2, n + 5), 7.0, dtype=dtype, device="cuda")
    out = around[1:-1, 3:-2]
    sg.int8_gemm(matrix(a, sa), matrix(b, sb), out=out)
    same(out, ref.product(a, sa, b, sb, dtype))
    around[1:-1, 3:-2] = 7.0
    assert (around == 7.0).all()
    x = values(m, k, dtype)
    around[:] = 7.0
    sg.int8_linear(x, matrix(b, sb), out=out)
    same(out, sg.int8_linear(x, matrix(b, sb)))
    around[1:-1, 3:-2] = 7.0
    assert (around == 7.0).all()


# ------------------------------------------------------------------ checkpoints
CHECKPOINTS = [(1, 1, 0), (1, 32, 0), (3, 31, 1), (16, 33, 0), (17, 128, 3), (127, 129, 0), (128, 128, 8), (130, 500, 0), (300, 64, 1)]


def check_layout(c, q, u):
    """Integers, units and their padding where int8.h has them."""
    rows, cols = c.shape
    blocks = u.shape[1]
    codes, units = c.codes.cpu(), c.units.cpu().double()
    q = torch.from_numpy(q.reshape(rows, -1)[:, :cols]).to(torch.int8)
    u = torch.from_numpy(u)
    if c.order == "channels":
        q, u = q.t(), u.t()
    assert codes.shape[1] % 16 == 0 and units.shape[1] % 8 == 0
    same(codes[:, :q.shape[1]], q.contiguous())
    assert codes.shape[0] == q.shape[0] and (codes[:, q.shape[1]:] == 0).all()
    same(units[:, :u.shape[1]], u.contiguous())
    assert units.shape[0] == u.shape[0] and (units[:, u.shape[1]:] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", CHECKPOINTS)
def test_checkpoints_bit_for_bit(dtype, rows, cols, pad):
    x = values(rows, cols, dtype, rows * cols, pad)
    c = sg.int8_checkpoint(x)
    q, u = ref.keep(ref.array(x), dtype == F16)
    check_layout(c, q, u)
    want = torch.from_numpy(ref.kept(ref.array(x), dtype == F16))
    assert (c.restore().double().cpu() == want).all()     # the type holds them exactly
    for out in TYPES:
        same(c.restore(out), want.float().to(out))
    finish()


def test_checkpoints_at_the_ends_of_the_range():
    x = torch.zeros(9, 96)
    x[1, 0], x[1, 1] = 3.4e38, -1.7e38
    x[2, 40], x[2, 41], x[2, 42] = 1e-38, -3e-39, 2.0 ** -126
    x[3, 64], x[4, 70], x[5, 95] = float("nan"), float("inf"), -float("inf")
    x[6, :] = torch.linspace(-1, 1, 96) * 127.4
    x[7, 0], x[7, 1], x[7, 2] = 127.5, 2.5, 3.5
    x[8, 1] = 2.0 ** -120
    c = sg.int8_checkpoint(x.cuda())
    q, u = ref.keep(x.numpy(), False)
    check_layout(c, q, u)
    back = c.restore().cpu()
    assert back[3:6, 64:].isnan().all() and back[3:6, :64].isfinite().all() and back[[0, 1, 2, 6, 7, 8]].isfinite().all()
    x = torch.zeros(3, 32, dtype=F16)
    x[0, 0], x[0, 1], x[1, 0], x[1, 1], x[2, 3] = 65504, -513, 2.0 ** -24, -2.0 ** -23, 2.0 ** -13
    c = sg.int8_checkpoint(x.cuda())
    check_layout(c, *ref.keep(x.double().numpy(), True))
    same(c.restore(), torch.from_numpy(ref.kept(x.double().numpy(), True)).to(F16))


# ------------------------------------------------------------- weight gradients
def check_gradient(dw, dy, x, half, before=None):
    """|error| <= tokens * 2^-23 * sum |dy x| (32-bit sums in any order, cut or rounded) and the last rounding."""
    d, k = ref.array(dy), ref.kept(ref.array(x), half)
    want, size = d.T @ k, np.abs(d).T @ np.abs(k)
    if before is not None:
        want, size = want + ref.array(before), size + np.abs(ref.array(before))
    bound = (d.shape[0] + 2) * 2.0 ** -23 * size
    bound = bound + ref.half_step(dw.dtype) * (np.abs(want) + bound) + (2.0 ** -25 if dw.dtype == F16 else 0)
    err = np.abs(ref.array(dw) - want)
    assert (err <= bound).all(), f"largest excess {(err - bound).max()}"


GRADIENTS = [(1, 1, 1, 0), (1, 33, 40, 3), (5, 70, 32, 0), (16, 128, 129, 1), (63, 8, 200, 0), (64, 256, 256, 0), (100, 520, 392, 8), (129, 65, 33, 1),
             (333, 130, 257, 3), (500, 257, 64, 0), (1024, 100, 300, 0), (1100, 384, 130, 1), (2500, 72, 96, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k,pad", GRADIENTS)
def test_weight_gradients(dtype, m, n, k, pad):
    x, dy = values(m, k, dtype, 1, pad), values(m, n, dtype, 2, pad, 0.1)
    c = sg.int8_checkpoint(x)
    check_gradient(sg.int8_weight_grad(dy, c), dy, x, dtype == F16)
    dw = sg.int8_weight_grad(dy, c, out_dtype=F32)
    assert dw.dtype == F32
    check_gradient(dw, dy, x, dtype == F16)
    finish()


@pytest.mark.parametrize("dtype", TYPES)
def test_every_bit_of_a_gradient_counts(dtype):
    """Tokens that each hold one 1: the gradient's rows are dy's, all 24 bits of them."""
    x = torch.eye(40, 64, dtype=dtype, device="cuda")
    dy = values(40, 90, dtype, 3)
    dw = sg.int8_weight_grad(dy, sg.int8_checkpoint(x))
    same(dw, torch.cat([dy.t(), torch.zeros(90, 24, dtype=dtype, device="cuda")], 1))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", ["own", "float32"])
def test_gradients_are_added_up(dtype, out):
    m, n, k = 200, 150, 70
    x, dy = values(m, k, dtype, 4), values(m, n, dtype, 5)
    kind = dtype if out == "own" else F32
    around = values(n + 2, k + 9, kind, 6)
    before = around.clone()
    dw = around[1:-1, 4:-5]
    got = sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out=dw, accumulate=True)
    assert got is dw
    check_gradient(dw, dy, x, dtype == F16, before[1:-1, 4:-5])
    around[1:-1, 4:-5] = before[1:-1, 4:-5]
    same(around, before)
    sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out=dw)          # not added: what was there is not read
    check_gradient(dw, dy, x, dtype == F16)
    none = sg.int8_checkpoint(x[:0])
    kept = dw.clone()
    same(sg.int8_weight_grad(dy[:0], none, out=dw, accumulate=True), kept)
    assert (sg.int8_weight_grad(dy[:0], none, out=dw) == 0).all()


def test_outputs_are_not_read():
    x, dy = values(50, 70, BF16), values(50, 33, BF16, 1)
    dw = torch.full((33, 70), float("nan"), dtype=BF16, device="cuda")
    assert sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out=dw).isfinite().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_of_values_that_are_not_finite(dtype):
    """A block that is NaN reaches its channels, a gradient that is not finite its row; nothing else."""
    x, dy = values(70, 100, dtype), values(70, 60, dtype, 1)
    x[:, 10] = 1.0
    x[5, 40], dy[8, 3], dy[9, 4] = float("nan"), float("nan"), float("inf")
    dw = sg.int8_weight_grad(dy, sg.int8_checkpoint(x)).cpu()
    assert dw[:, 32:64].isnan().all() and dw[3].isnan().all()
    assert dw[4, 10] == float("inf")
    rest = dw[[i for i in range(60) if i not in (3, 4)]]
    assert rest[:, :32].isfinite().all() and rest[:, 64:].isfinite().all()


def test_a_gradient_is_a_difference_quotient():
    """Of L(W) = sum dy * (x W^T), linear in W: two evaluations in 64 bits give the gradient exactly."""
    x, dy = values(30, 40, F32), values(30, 20, F32, 1)
    c = sg.int8_checkpoint(x)
    dw = ref.array(sg.int8_weight_grad(dy, c))
    k, d, w = ref.array(c.restore()), ref.array(dy), np.random.default_rng(0).normal(size=(20, 40))
    loss = lambda w: float((d * (k @ w.T)).sum())  # noqa: E731
    for i, j in ((0, 0), (19, 39), (7, 21)):
        up, down = w.copy(), w.copy()
        up[i, j] += 1
        down[i, j] -= 1
        size = np.abs(d[:, i]) @ np.abs(k[:, j])
        assert abs(dw[i, j] - (loss(up) - loss(down)) / 2) <= 32 * 2.0 ** -23 * size + 1e-9 * np.abs(d).sum()


def test_results_repeat_bit_for_bit():
    x, dy = values(3000, 200, BF16), values(3000, 100, BF16, 1)
    c = sg.int8_checkpoint(x)
    first = sg.int8_weight_grad(dy, c, out_dtype=F32)
    for _ in range(3):
        same(sg.int8_weight_grad(dy, c, out_dtype=F32), first)


# ------------------------------------------------------------- gated activation
def swiglu_bounds(d, g, u, dtype):
    """Errors of 32-bit arithmetic: e^-g within 2 ulp (2^-22), a sum, a reciprocal, and each product 2^-24: the sigmoid within
    2^-22 + 2^-23 of itself, whatever follows another 2^-22; 1 - s loses |g| of that beside 1 + g (1 - s).  For 16-bit types the
    exponential is 2^(-g log2 e) with the product rounded: |g| log2(e) 2^-24 ln 2 = |g| 2^-24 for it and as much for the constant,
    2^-22 for the power, and the reciprocal another 2^-23, so (|g| + 4) 2^-22 covers the sigmoid."""
    s = ref.sigmoid(g)
    rel = 2.0 ** -20 * np.ones_like(g) if dtype == F32 else 2.0 ** -20 + (np.abs(g) + 4) * 2.0 ** -22
    forward = rel * np.abs(g * s * u)
    dgate = rel * np.abs(d * u * s) * (1 + np.abs(g) * (1 + (1 - s)))
    return forward, dgate, rel * np.abs(d * g * s)


def near(got, want, bound, dtype):
    """Within `bound`, the last rounding, and what the type cannot hold near zero."""
    tiny = {F32: 2.0 ** -125, BF16: 2.0 ** -125, F16: 2.0 ** -25}[dtype]
    err = np.abs(ref.array(got) - want)
    assert (err <= bound + ref.half_step(dtype) * (np.abs(want) + bound) + tiny).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (2, 31, 1), (1, 64, 0), (5, 100, 3), (33, 1001, 0), (40, 256, 8), (300, 40, 0)])
def test_swiglu_and_its_gradients(dtype, rows, cols, pad):
    both = values(rows, 2 * cols, dtype, 7, pad, 2.0)
    gate, up = both[:, :cols], both[:, cols:]
    dh = values(rows, cols, dtype, 8, pad)
    h, kept = sg.int8_swiglu(gate, up)
    g, u, d = ref.array(gate), ref.array(up), ref.array(dh)
    near(h, ref.swiglu(g, u), swiglu_bounds(d, g, u, dtype)[0], dtype)
    for c, v in zip(kept, (g, u)):
        check_layout(c, *ref.keep(v, dtype == F16))
        assert (c.restore().double().cpu().numpy() == ref.kept(v, dtype == F16)).all()
    dgate, dup = sg.int8_swiglu_backward(dh, kept)
    g, u = ref.kept(g, dtype == F16), ref.kept(u, dtype == F16)
    want, bounds = ref.swiglu_backward(d, g, u), swiglu_bounds(d, g, u, dtype)
    near(dgate, want[0], bounds[1], dtype)
    near(dup, want[1], bounds[2], dtype)
    step = 1e-5                                            # and against differences
    numeric = d * (ref.swiglu(g + step, u) - ref.swiglu(g - step, u)) / (2 * step)
    assert np.allclose(want[0], numeric, rtol=1e-5, atol=1e-7 * (1 + np.abs(d * u)).max())
    finish()


@pytest.mark.parametrize("dtype", (BF16, F16))
@pytest.mark.parametrize("rows,cols,pad", [(700, 912, 16), (39000, 16, 0), (1, 655376, 0)])
def test_swiglu_of_many_values(dtype, rows, cols, pad):
    """Sizes where a thread takes 16 values: blocks of 16 at the end of a row, a block that is not finite."""
    both = values(rows, 2 * cols, dtype, 17, pad, 2.0)
    gate, up = both[:, :cols], both[:, cols:]
    both[rows // 2, 3], both[rows // 2, cols + 11] = float("nan"), float("inf")
    h, kept = sg.int8_swiglu(gate, up)
    g, u = ref.array(gate), ref.array(up)
    bad = ~np.isfinite(g * u)
    got = h.double().cpu().numpy()
    assert bad.sum() == 2 and np.isnan(got[rows // 2, 3]) and np.isinf(got[rows // 2, 11])
    for c, v in zip(kept, (g, u)):
        check_layout(c, *ref.keep(v, dtype == F16))
    h[torch.tensor(bad)] = 0
    g[bad] = u[bad] = 0
    near(h, ref.swiglu(g, u), swiglu_bounds(g, g, u, dtype)[0], dtype)
    finish()


def test_swiglu_far_from_zero():
    g = torch.tensor([[0.0, 100.0, -100.0, 88.0, -88.0, 1e30, -1e30, -60.0, float("inf"), 20.0, -0.0, 3.4e38]]).cuda()
    u = torch.full_like(g, 2.0)
    h, kept = sg.int8_swiglu(g, u)
    want = [0, 200, 0, 176, None, 2e30, 0, None, float("inf"), 40, 0, float("inf")]
    for i, w in enumerate(want):
        if w is not None:
            assert h[0, i].item() == pytest.approx(w, rel=1e-6, abs=1e-35), i
    g[0, 8], g[0, 11] = 5.0, -5.0
    _, kept = sg.int8_swiglu(g[:, :1].contiguous(), u[:, :1].contiguous())
    dg, du = sg.int8_swiglu_backward(torch.ones(1, 1, device="cuda"), kept)
    assert dg.item() == 1.0 and du.item() == 0.0
    big = torch.tensor([[60.0, -60.0, 64.0, -64.0]]).cuda()
    _, kept = sg.int8_swiglu(big, big)
    dg, du = sg.int8_swiglu_backward(torch.ones(1, 4, device="cuda"), kept)
    assert dg.isfinite().all() and du[0, 0] == 60.0 and abs(du[0, 1].item()) < 1e-20


def test_swiglu_writes_halves_of_one_tensor_and_nothing_else():
    rows, f = 21, 70
    both, dh = values(rows, 2 * f, BF16, 1), values(rows, f, BF16, 2)
    _, kept = sg.int8_swiglu(both[:, :f], both[:, f:])
    want = sg.int8_swiglu_backward(dh, kept)
    around = torch.full((rows + 2, 2 * f + 3), 5.0, dtype=BF16, device="cuda")
    out = around[1:-1, 1:f + 1], around[1:-1, f + 1:2 * f + 1]
    got = sg.int8_swiglu_backward(dh, kept, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    same(out[0], want[0])
    same(out[1], want[1])
    around[1:-1, 1:2 * f + 1] = 5.0
    assert (around == 5.0).all()
    h = torch.full((rows + 1, f + 1), 5.0, dtype=BF16, device="cuda")
    sg.int8_swiglu(both[:, :f], both[:, f:], out=h[:-1, :-1])
    assert (h[-1] == 5.0).all() and (h[:, -1] == 5.0).all()


# ---------------------------------------------------------- streams and graphs
def test_a_passed_stream_is_used():
    s = torch.cuda.Stream()
    x, dy = values(100, 300, BF16), values(100, 50, BF16, 1)
    w = sg.int8_quantize(values(80, 300, F32))
    torch.cuda.synchronize()
    y = sg.int8_linear(x, w, stream=s)
    c = sg.int8_checkpoint(x, stream=s)
    dw = sg.int8_weight_grad(dy, c, stream=s)
    h, kept = sg.int8_swiglu(x, x, stream=s)
    dg = sg.int8_swiglu_backward(h, kept, stream=s)
    back = sg.int8_restore(c, stream=s)
    q = sg.int8_matrix(w.codes[:, 1:], w.scales, stream=s)
    s.synchronize()
    same(y, sg.int8_linear(x, w))
    same(dw, sg.int8_weight_grad(dy, sg.int8_checkpoint(x)))
    same(dg[0], sg.int8_swiglu_backward(h, sg.int8_swiglu(x, x)[1])[0])
    same(back, c.restore())
    same(q.codes, w.codes[:, 1:])


def test_captured_and_replayed():
    x, dy = values(70, 256, BF16), values(70, 128, BF16, 1)
    w = sg.int8_quantize(values(128, 256, F32))

    def step():
        y = sg.int8_linear(x, w)
        c = sg.int8_checkpoint(x)
        h, kept = sg.int8_swiglu(y, y)
        dgate, dup = sg.int8_swiglu_backward(dy, kept)
        return y, sg.int8_weight_grad(dgate, c), h, dup, sg.int8_gemm(sg.int8_quantize(y), sg.int8_quantize(h)), sg.int8_linear(x[:5], w)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for seed in (3, 4):
        x.copy_(values(70, 256, BF16, seed))
        dy.copy_(values(70, 128, BF16, seed + 10))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            same(a, b)
    finish()


def test_two_streams_at_once():
    """Each stream has a workspace of its own."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    w = [sg.int8_quantize(values(300, 512, F32, i)) for i in range(2)]
    x = [values(200, 512, BF16, i + 5) for i in range(2)]
    dy = [values(200, 100, F32, i + 8) for i in range(2)]
    c = [sg.int8_checkpoint(x[i].float()) for i in range(2)]
    want = [(sg.int8_linear(x[i], w[i]), sg.int8_weight_grad(dy[i], c[i])) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((sg.int8_linear(x[i], w[i]), sg.int8_weight_grad(dy[i], c[i])))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same(a[0], b[0])
            same(a[1], b[1])


def test_a_call_after_the_call_that_made_its_input():
    """Kernels that start beside the end of the one before wait for what it writes."""
    x = values(16, 4096, BF16)
    for m in (1, 16, 150):
        base = values(m, 4096, BF16, m)
        for i in range(4):
            weights = sg.int8_quantize(values(256, 4096, F32, i))
            y = sg.int8_linear(base, weights)
            z = sg.int8_linear(y.contiguous(), sg.int8_quantize(weights.dequantize()[:, :256].contiguous()))
            torch.cuda.synchronize()
            again = sg.int8_linear(base, weights)
            torch.cuda.synchronize()
            same(y, again)
            w2 = sg.int8_quantize(weights.dequantize()[:, :256].contiguous())
            torch.cuda.synchronize()
            same(z, sg.int8_linear(y, w2))


# --------------------------------------------------------------------- refusals
def test_refusals():
    x, w = values(4, 64, BF16), sg.int8_quantize(values(8, 64, F32))
    c = sg.int8_checkpoint(x)
    h, kept = sg.int8_swiglu(x, x)
    for call, error in [
            (lambda: sg.int8_quantize(x.cpu()), ValueError), (lambda: sg.int8_quantize(x.int()), ValueError),
            (lambda: sg.int8_quantize(x.t()), ValueError), (lambda: sg.int8_quantize("x"), TypeError),
            (lambda: sg.int8_quantize(x, out=w), ValueError), (lambda: sg.int8_quantize(x[0]), ValueError),
            (lambda: sg.int8_matrix(w.codes.int(), w.scales), ValueError), (lambda: sg.int8_matrix(w.codes, w.scales[:3]), ValueError),
            (lambda: sg.int8_matrix(w.codes, w.scales.double()), ValueError), (lambda: sg.int8_matrix([1], w.scales), TypeError),
            (lambda: sg.int8_linear(x[:, :63], w), ValueError), (lambda: sg.int8_linear(x, x), TypeError),
            (lambda: sg.int8_linear(x, w, out=torch.empty(4, 8, device="cuda")), ValueError),
            (lambda: sg.int8_gemm(w, sg.int8_quantize(x[:, :60])), ValueError), (lambda: sg.int8_gemm(w, w, out_dtype=torch.int32), ValueError),
            (lambda: sg.int8_weight_grad(x.float(), c), ValueError), (lambda: sg.int8_weight_grad(x[:3], c), ValueError),
            (lambda: sg.int8_weight_grad(x, kept[0]), ValueError), (lambda: sg.int8_weight_grad(x, c, accumulate=True), ValueError),
            (lambda: sg.int8_weight_grad(x, c, out_dtype=F16), ValueError), (lambda: sg.int8_weight_grad(x, w), TypeError),
            (lambda: sg.int8_checkpoint(x, out=kept[0]), ValueError), (lambda: sg.int8_restore(w), TypeError),
            (lambda: sg.int8_swiglu(x, x[:, :32]), ValueError), (lambda: sg.int8_swiglu(x, x.float()), ValueError),
            (lambda: sg.int8_swiglu_backward(h, kept[0]), TypeError), (lambda: sg.int8_swiglu_backward(h, (c, c)), ValueError),
            (lambda: sg.int8_swiglu_backward(h.float(), kept), ValueError), (lambda: sg.int8_swiglu_backward(h, kept, out=h), TypeError),
            (lambda: sg.int8_swiglu_backward(h, kept, out=(h, h)), sg.SgemmError), (lambda: sg.int8_swiglu(x, x, out=x), sg.SgemmError),
            (lambda: sg.int8_linear(x, sg.int8_quantize(x.repeat(16, 1)), out=x), sg.SgemmError),
            (lambda: sg.int8_dequantize(w, torch.int8), ValueError), (lambda: sg.Int8Matrix(2, 2, device="cpu"), ValueError),
            (lambda: sg.Int8Checkpoint(2, 2, F32, "rows"), ValueError)]:
        with pytest.raises(error):
            call()
    finish()


def test_sums_that_integers_cannot_hold_are_refused():
    q = sg.Int8Matrix(1, 131072)
    with pytest.raises(sg.SgemmError):
        sg.int8_gemm(q, q)
