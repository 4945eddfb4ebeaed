"""The 8-bit integer operators at the ends of what their calls allow (GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg
from dense_fp32_gemm_03_gb300 import binding, int8

import int8_ref as ref
from test_int8_gpu import BF16, F16, F32, check_gradient, integers, matrix, same, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


# ------------------------------------------------------------ sizes and offsets
# Elements beyond 2^31 of a matrix: rows from all over it are compared.
BIG = 66000, 33000


def some_rows(n):
    return torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")


def test_rows_beyond_32_bit_offsets():
    rows, cols = BIG
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    at = some_rows(rows)
    for r in at.tolist():
        x[r] = values(1, cols, BF16, r)[0]
    q = sg.int8_quantize(x)
    codes, scales = ref.quantize(ref.array(x[at]))
    same(q.codes[at], torch.from_numpy(codes))
    same(q.scales[at], torch.from_numpy(scales))
    y = sg.int8_dequantize(q, BF16)
    same(y[at], ref.round_to(codes.astype(np.float32) * scales[:, None], BF16))


@pytest.mark.parametrize("m", [1, 7, 20])
def test_weights_beyond_32_bit_offsets(m):
    n, k = BIG
    w = torch.empty(n, k + 8, dtype=torch.int8, device="cuda")     # 33008 bytes a row: a multiple of 16
    at = some_rows(n)
    for r in at.tolist():
        w[r] = torch.from_numpy(integers(1, k + 8, r)[0][0]).cuda()
    scales = torch.rand(n, device="cuda")
    q = sg.int8_matrix(w[:, :k], scales)
    assert q.codes.data_ptr() == w.data_ptr()
    x = values(m, k, F16, 3)
    y = sg.int8_linear(x, q)
    a, sa = ref.quantize(ref.array(x))
    same(y[:, at], ref.product(a, sa, w[at, :k].cpu().numpy(), scales[at].cpu().numpy(), F16))


def test_checkpoints_beyond_32_bit_offsets():
    rows, cols = 70000, 31000
    x = torch.zeros(rows, cols, dtype=F16, device="cuda")
    at = some_rows(rows)
    for r in at.tolist():
        x[r] = values(1, cols, F16, r)[0]
    c = sg.int8_checkpoint(x)
    want = torch.from_numpy(ref.kept(ref.array(x[at]), True)).to(F16)
    same(sg.int8_restore(c)[at], want)
    dy = torch.zeros(rows, 8, dtype=F16, device="cuda")
    dy[at] = values(len(at), 8, F16, 5)
    check_gradient(sg.int8_weight_grad(dy, c), dy[at], x[at], True)      # the other tokens are zero


def test_swiglu_beyond_32_bit_offsets():
    rows, cols = 70000, 31000
    both = torch.zeros(rows, 2 * cols, dtype=F16, device="cuda")
    at = some_rows(rows)
    for r in at.tolist():
        both[r] = values(1, 2 * cols, F16, r)[0]
    gate, up = both[:, :cols], both[:, cols:]
    h, kept = sg.int8_swiglu(gate, up)
    small_h, small = sg.int8_swiglu(gate[at], up[at])
    same(h[at], small_h)
    same(kept[0].restore()[at], small[0].restore())
    dg, du = sg.int8_swiglu_backward(h, kept)
    want = sg.int8_swiglu_backward(small_h, small)
    same(dg[at], want[0])
    same(du[at], want[1])


def test_rows_far_apart():
    """Row strides beyond 2^31 elements."""
    stride = (1 << 31) + 8
    memory = torch.empty(2 * stride + 400, dtype=BF16, device="cuda")
    x = memory.as_strided((3, 200), (stride, 1))
    x.copy_(values(3, 200, BF16))
    near = x.contiguous()
    w = sg.int8_quantize(values(64, 200, F32, 1))
    same(sg.int8_linear(x, w), sg.int8_linear(near, w))
    same(sg.int8_quantize(x).codes, sg.int8_quantize(near).codes)
    c = sg.int8_checkpoint(x)
    same(c.restore(), sg.int8_checkpoint(near).restore())
    same(sg.int8_weight_grad(x, c), sg.int8_weight_grad(near, c))
    out = memory.as_strided((3, 64), (stride, 1), 256)
    sg.int8_linear(near, w, out=out)
    same(out, sg.int8_linear(near, w))


@pytest.mark.parametrize("m,n,k", [(20, 4, 70000), (300, 1, 17), (1, 1, 131071), (9, 5000, 1), (2, 70000, 5), (70000, 3, 20), (513, 130, 640)])
def test_lopsided_products(m, n, k):
    (a, sa), (b, sb) = integers(m, k, 1, -128), integers(n, k, 2, -128)
    same(sg.int8_gemm(matrix(a, sa), matrix(b, sb), out_dtype=BF16), ref.product(a, sa, b, sb, BF16))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("m,n,k", [(20000, 5, 40), (7, 3000, 8), (3, 9, 5000), (129, 300, 1000), (16, 16, 16), (2049, 1, 1)])
def test_lopsided_gradients(dtype, m, n, k):
    x, dy = values(m, k, dtype, 1), values(m, n, dtype, 2, 0, 0.1)
    check_gradient(sg.int8_weight_grad(dy, sg.int8_checkpoint(x)), dy, x, dtype == F16)


@pytest.mark.parametrize("m,n,k", [(9, 8192, 1000), (16, 4096, 4096), (20, 1024, 8200), (32, 300, 3000), (33, 8192, 1024), (64, 1000, 9000),
                                   (128, 500, 20000), (200, 256, 5000)])
def test_sums_cut_over_k(m, n, k):
    """Shapes whose sums are cut into shares, joined in a cluster or by a kernel."""
    (a, sa), (b, sb) = integers(m, k, 1, -128), integers(n, k, 2, -128)
    x, w = matrix(a, sa), matrix(b, sb)
    want = ref.product(a, sa, b, sb, F32)
    for _ in range(2):
        same(sg.int8_gemm(x, w), want)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("m,n,k", [(9, 17, 33), (16, 40, 15), (17, 6401, 16), (65, 100, 1), (23, 33, 127), (40000, 3, 20), (120, 300, 777), (8, 6401, 130),
                                   (700, 1001, 1031), (1030, 2047, 513), (300, 3001, 2100)])
def test_products_by_eight_tokens_and_in_tiles(m, n, k, dtype):
    (a, sa), (b, sb) = integers(m, k, 7, -128), integers(n, k, 8, -128)
    w = matrix(b, sb)
    around = torch.full((m + 2, n + 5), 5.0, dtype=dtype, device="cuda")
    out = around[1:-1, 1:n + 1]
    sg.int8_gemm(matrix(a, sa), w, out=out)
    same(out.contiguous(), ref.product(a, sa, b, sb, dtype))
    x = values(m, k, dtype, 9, 3)
    sg.int8_linear(x, w, out=out)
    same(out.contiguous(), ref.product(*ref.quantize(ref.array(x)), b, sb, dtype))
    out.fill_(5.0)
    assert (around == 5.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("m,n,k,pad", [(1, 6401, 300, 0), (1, 7000, 4096, 0), (1, 12011, 1001, 1), (2, 6500, 1000, 3), (8, 12000, 200, 0), (5, 6400, 2064, 0)])
def test_few_tokens_of_many_channels(dtype, m, n, k, pad):
    (b, sb), x = integers(n, k, 11, -128), values(m, k, dtype, 12, pad)
    w = matrix(b, sb)
    want = ref.product(*ref.quantize(ref.array(x)), b, sb, dtype)
    for _ in range(2):
        same(sg.int8_linear(x, w), want)
    same(sg.int8_gemm(sg.int8_quantize(x), w, out_dtype=dtype), want)


@pytest.mark.parametrize("m", [3, 40])
def test_codes_behind_both_rows_are_not_used(m):
    """Integers behind the columns of either operand, in the 16 bytes that the kernels read."""
    n, k = 50, 100
    (a, sa), (b, sb) = integers(m, k, 1, -128), integers(n, k, 2, -128)
    want = ref.product(a, sa, b, sb, F32)
    held = []
    for q, s in ((a, sa), (b, sb)):
        memory = torch.full((len(q), 112), 77, dtype=torch.int8, device="cuda")
        memory[:, :k] = torch.from_numpy(q).cuda()
        held.append(sg.int8_matrix(memory[:, :k], torch.from_numpy(s).cuda()))
        assert held[-1].codes.data_ptr() == memory.data_ptr()
    same(sg.int8_gemm(*held), want)


@pytest.mark.parametrize("m,n,k", [(120, 250, 1600), (260, 1000, 2100), (128, 1000, 4000), (100, 2500, 3000), (130, 4100, 3000), (700, 512, 4001)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_products_whose_shares_meet(m, n, k, dtype):
    """Two and four shares of k for each width of tile, in a part of a larger output."""
    (a, sa), (b, sb) = integers(m, k, 3, -128), integers(n, k, 4, -128)
    around = torch.full((m + 2, n + 9), 5.0, dtype=dtype, device="cuda")
    x, w = matrix(a, sa), matrix(b, sb)
    for _ in range(2):
        sg.int8_gemm(x, w, out=around[1:-1, 1:n + 1])
    same(around[1:-1, 1:n + 1].contiguous(), ref.product(a, sa, b, sb, dtype))
    around[1:-1, 1:n + 1] = 5.0
    assert (around == 5.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("m,n,k", [(1000, 100, 200), (1300, 1001, 1024), (2600, 200, 519), (1200, 520, 700), (2049, 130, 300)])
def test_gradients_whose_shares_meet(dtype, own, m, n, k):
    x, dy = values(m, k, dtype, 5), values(m, n, dtype, 6, 3, 0.1)
    c, kind = sg.int8_checkpoint(x), dtype if own else F32
    around = torch.full((n + 2, k + 9), 5.0, dtype=kind, device="cuda")
    out = around[1:-1, 1:k + 1]
    sg.int8_weight_grad(dy, c, out=out)
    check_gradient(out, dy, x, dtype == F16)
    first = out.clone()
    sg.int8_weight_grad(dy, c, out=out)
    same(out.contiguous(), first)
    sg.int8_weight_grad(dy, c, out=out, accumulate=True)
    check_gradient(out, dy, x, dtype == F16, first)
    out.fill_(5.0)
    assert (around == 5.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (5, 70, 33), (64, 256, 256), (65, 33, 32), (200, 40, 65), (700, 31, 96), (333, 520, 1001), (333, 2050, 1501), (129, 4001, 1031)])
def test_gradients_of_few_tokens(dtype, own, m, n, k):
    """Small ones, and ones in tiles; dy with rows of 16 bytes and others."""
    x, dy = values(m, k, dtype, 5), values(m, n, dtype, 6, 3 if m % 2 else 0, 0.1)
    c, kind = sg.int8_checkpoint(x), dtype if own else F32
    around = torch.full((n + 2, k + 9), 5.0, dtype=kind, device="cuda")
    out = around[1:-1, 1:k + 1]
    sg.int8_weight_grad(dy, c, out=out)
    check_gradient(out, dy, x, dtype == F16)
    first = out.clone()
    sg.int8_weight_grad(dy, c, out=out)
    same(out.contiguous(), first)
    sg.int8_weight_grad(dy, c, out=out, accumulate=True)
    check_gradient(out, dy, x, dtype == F16, first)
    out.fill_(5.0)
    assert (around == 5.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_small_gradients_beside_nan(dtype):
    """What is not finite in dy or in x reaches the sums that it is part of, and no others."""
    m, n, k = 130, 50, 100
    x, dy = values(m, k, dtype, 1), values(m, n, dtype, 2, 1, 0.1)
    clean = sg.int8_weight_grad(dy, sg.int8_checkpoint(x))
    x[7, 40], dy[129, 3], dy[0, 9] = float("nan"), float("inf"), float("nan")
    got = sg.int8_weight_grad(dy, sg.int8_checkpoint(x))
    bad = torch.zeros(n, k, dtype=torch.bool, device="cuda")
    bad[:, 32:64] = bad[9] = True
    assert got[bad].isnan().all()
    assert not got[3].isfinite().any()
    bad[3] = True
    same(got[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("scale", [2.0 ** -14, 2.0 ** -20, 2.0 ** -24, 2.0 ** 8, 2.0 ** -100, 2.0 ** 100])
def test_gradients_far_from_one(dtype, scale):
    """Units and gradients at the ends of their types: tokens of one value each, so that dW is dY times it, exactly."""
    if dtype == F16 and not 2.0 ** -24 <= scale <= 2.0 ** 8:
        pytest.skip("beyond 16-bit floats of five exponent bits")
    x = torch.eye(40, 64, dtype=F32, device="cuda") * scale
    x[:, 40:] = 0
    dy = values(40, 90, dtype, 3, 0, 1.0 / 64)
    factor = 2.0 ** 10 if scale < 1 else 2.0 ** -6           # and the product far from the type's ends
    dy = (dy.float() * factor).to(dtype)
    dw = sg.int8_weight_grad(dy, sg.int8_checkpoint(x.to(dtype)), out_dtype=F32)
    same(dw[:, :40], (dy.float() * scale).t())
    if dtype != F16:
        # Large times small.  The last of a 32-bit gradient's terms ends where bfloat16 does, at 2^-133: what a gradient has
        # below that is cut off, less than 2^-133 of it, which the one product multiplies by the kept value.
        tiny = (dy.float() / scale * 2.0 ** -4).to(dtype)
        dw = sg.int8_weight_grad(tiny, sg.int8_checkpoint(x.to(dtype)), out_dtype=F32)[:, :40]
        assert ((dw.double() - tiny.double().t() * scale).abs() <= (2.0 ** -133 * scale if dtype == F32 else 0.0)).all()


def test_subnormal_gradients():
    x = torch.eye(20, 32, dtype=F16, device="cuda") * 512
    dy = (torch.arange(20 * 16, device="cuda").view(20, 16) - 150).half() * 2.0 ** -24
    same(sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out_dtype=F32)[:, :20], dy.float().t() * 512)


# ------------------------------------------------------- what lies beside a call
def test_codes_behind_a_row_are_not_used():
    """Rows of 33 bytes in 48: the other 15 hold anything."""
    for m in (1, 5, 40):
        for n in (3, 300):
            wide_a = torch.randint(-128, 128, (m, 48), dtype=torch.int8, device="cuda")
            wide_b = torch.randint(-128, 128, (n, 48), dtype=torch.int8, device="cuda")
            a, b = sg.int8_matrix(wide_a[:, :33], torch.ones(m, device="cuda")), sg.int8_matrix(wide_b[:, :33], torch.ones(n, device="cuda"))
            assert a.codes.data_ptr() == wide_a.data_ptr()
            same(sg.int8_gemm(a, b), (wide_a[:, :33].double() @ wide_b[:, :33].double().t()).float())
            x = wide_a[:, :33].float().clamp(-127, 127)
            x[:, 0] = 127                                                     # scales of 1
            same(sg.int8_linear(x, b), (x.double() @ wide_b[:, :33].double().t()).float())


def test_gradients_beside_nan():
    """dY between columns of NaN, read where it is: aligned, 16-bit, and not a multiple of eight columns."""
    around = torch.full((70, 64), float("nan"), dtype=BF16, device="cuda")
    dy = around[:, 8:45]
    dy.copy_(values(70, 37, BF16))
    x = values(70, 50, BF16, 1)
    check_gradient(sg.int8_weight_grad(dy, sg.int8_checkpoint(x)), dy, x, False)


def test_a_call_leaves_other_streams_scratch_alone():
    """A workspace grows while a graph that uses the old one lives."""
    s = torch.cuda.Stream()
    w = sg.int8_quantize(values(300, 400, F32))
    x = values(40, 400, BF16)
    with torch.cuda.stream(s):
        want = sg.int8_linear(x, w)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = sg.int8_linear(x, w)
    big = values(5000, 400, BF16)
    with torch.cuda.stream(s):
        sg.int8_linear(big, w)
        y.zero_()
        graph.replay()
    s.synchronize()
    same(y, want)


def test_the_same_inputs_twice_in_one_call():
    q = sg.int8_quantize(values(200, 300, F32))
    a = q.codes.cpu().numpy()
    sa = q.scales.cpu().numpy()
    same(sg.int8_gemm(q, q), ref.product(a, sa, a, sa, F32))
    x = values(60, 64, BF16)
    check_gradient(sg.int8_weight_grad(x, sg.int8_checkpoint(x)), x, x, False)
    h, kept = sg.int8_swiglu(x, x)
    same(kept[0].codes, kept[1].codes)


def test_outputs_of_earlier_calls_are_filled_again():
    x, other = values(50, 100, BF16), values(50, 100, BF16, 1)
    q, c = sg.int8_quantize(x), sg.int8_checkpoint(x)
    assert sg.int8_quantize(other, out=q) is q and sg.int8_checkpoint(other, out=c) is c
    same(q.codes, sg.int8_quantize(other).codes)
    same(c.restore(), sg.int8_checkpoint(other).restore())
    y = torch.empty(50, 100, dtype=F32, device="cuda")
    assert sg.int8_restore(c, out=y) is y and sg.int8_dequantize(q, out=y) is y
    arrays = sg.int8_matrix(torch.zeros(50, 112, dtype=torch.int8, device="cuda")[:, :100], torch.ones(50, device="cuda"))
    with pytest.raises(ValueError):
        sg.int8_quantize(x, out=arrays)


# -------------------------------------------------------------------- the C ABI
def test_through_the_c_abi():
    lib = int8.load()
    stream = torch.cuda.current_stream().cuda_stream
    x = values(33, 70, BF16)
    codes, scales = torch.zeros(33, 96, dtype=torch.int8, device="cuda"), torch.zeros(33, device="cuda")
    q = int8._Matrix(33, 70, codes.data_ptr(), 96, scales.data_ptr())
    assert lib.int8_quantize(1, x.data_ptr(), 70, ctypes.addressof(q), stream) == binding.OK
    want, s = ref.quantize(ref.array(x))
    same(codes[:, :70], torch.from_numpy(want))
    same(scales, torch.from_numpy(s))
    ld, ldu, cb, ub = (ctypes.c_int64() for _ in range(4))
    assert lib.int8_checkpoint_layout(0, 33, 70, *map(ctypes.byref, (ld, ldu, cb, ub))) == binding.OK
    a, b = torch.empty(cb.value, dtype=torch.int8, device="cuda"), torch.empty(ub.value // 2, dtype=BF16, device="cuda")
    c = int8._Checkpoint(1, 0, 33, 70, a.data_ptr(), ld.value, b.data_ptr(), ldu.value)
    assert lib.int8_checkpoint(x.data_ptr(), 70, ctypes.addressof(c), stream) == binding.OK
    dw = torch.empty(20, 70, device="cuda")
    dy = values(33, 20, BF16, 1)
    assert lib.int8_weight_grad(dy.data_ptr(), 20, 20, ctypes.addressof(c), 0, 0, dw.data_ptr(), 70, stream) == binding.OK
    check_gradient(dw, dy, x, False)
