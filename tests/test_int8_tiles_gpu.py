"""The tiled kernel of the 8-bit integer operators where it can go wrong (GPU).

Every size is one that the library's own plan gives to the tiles, and to the form and the shares of the sums that the case means;
``int8_plans`` asks the plan, so that a change of the estimates cannot move a case to another kernel unseen.
"""
import numpy as np
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg

import int8_plans
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


# Tokens, channels, columns; quantised tokens or not; columns of a tile, shares, whether they meet in a cluster.
PRODUCTS = [((200, 1500, 130), False, (32, 1, 0)), ((513, 512, 700), True, (32, 2, 1)), ((200, 512, 1500), False, (32, 4, 1)),
            ((200, 200, 8200), False, (32, 10, 0)), ((2050, 333, 130), True, (64, 1, 0)), ((700, 333, 1500), False, (64, 2, 1)),
            ((700, 130, 3000), False, (64, 4, 1)), ((300, 200, 8200), True, (64, 15, 0)), ((1000, 1030, 130), True, (128, 1, 0)),
            ((1000, 520, 2048), False, (128, 2, 1)), ((700, 333, 4100), True, (128, 4, 1))]
# Tokens, columns of dY, channels, dY's row pitch; type kept and of the gradient; columns of a tile, stages of a run, shares, in a cluster.
GRADIENTS = [((130, 1500, 520, 1504), BF16, BF16, (128, 0, 1, 0)), ((700, 130, 1500, 136), F16, F16, (128, 0, 2, 1)),
             ((1030, 130, 130, 136), BF16, BF16, (128, 0, 4, 1)), ((4100, 130, 130, 136), BF16, BF16, (128, 0, 8, 0)),
             ((130, 2048, 1030, 2048), BF16, BF16, (256, 0, 1, 0)), ((8200, 130, 1500, 136), F16, F16, (128, 4, 4, 1)),
             ((9000, 2001, 1056, 2008), F16, F16, (256, 16, 1, 0)), ((1030, 130, 130, 136), F16, F32, (128, 4, 4, 1)), ((2050, 520, 512, 521), BF16, F32, (128, 4, 4, 1)),
             ((130, 3000, 333, 3000), F32, F32, (128, 4, 1, 0)), ((300, 130, 700, 133), F32, F32, (128, 4, 2, 1)),
             ((513, 130, 130, 130), F32, F32, (128, 4, 4, 1)), ((4100, 130, 130, 130), F32, F32, (128, 4, 8, 0))]


def planned_product(size, quantised, want):
    p = int8_plans.product(*size, quantised)
    assert not p.small and (p.cols, p.splits, p.join) == want, (size, p)


def planned_gradient(size, dtype, out, want=None):
    m, n, k, ld = size
    p = int8_plans.gradient(m, n, k, dtype, out, aligned=ld % 8 == 0)
    assert not p.small and (want is None or (p.cols, p.run, p.splits, p.join) == want), (size, p)


def gradient_inputs(size, dtype, seed=1):
    """(x, dy): dy's rows `ld` values apart."""
    m, n, k, ld = size
    return values(m, k, dtype, seed), values(m, n, dtype, seed + 1, ld - n, 0.1)


product_cases = pytest.mark.parametrize("size,quantised,want", PRODUCTS)
gradient_cases = pytest.mark.parametrize("size,dtype,out,want", GRADIENTS)


# ------------------------------------------------------------- calls after one another
@product_cases
def test_a_product_after_the_calls_that_made_its_operands(size, quantised, want):
    """The product starts beside the end of the kernel that prepares its tokens, and reads weights that a call just before that made."""
    planned_product(size, quantised, want)
    m, n, k = size
    xs, ws = [values(m, k, BF16, s) for s in range(3)], [values(n, k, F32, 10 + s) for s in range(3)]
    expected = [ref.product(*ref.quantize(ref.array(x)), *ref.quantize(ref.array(w)), BF16) for x, w in zip(xs, ws)]
    w8, x8 = sg.int8_quantize(ws[0]), sg.int8_quantize(xs[0])
    out = torch.empty(m, n, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for x, w in zip(xs, ws):
            sg.int8_quantize(w, out=w8)                   # over weights that the product before reads
            if quantised:
                sg.int8_gemm(sg.int8_quantize(x, out=x8), w8, out=out)
            else:
                sg.int8_linear(x, w8, out=out)
            got.append(out.clone())
    for i, y in enumerate(got):
        same(y, expected[i % 3])


@gradient_cases
def test_a_gradient_after_the_calls_that_made_its_operands(size, dtype, out, want):
    planned_gradient(size, dtype, out, want)
    made = [gradient_inputs(size, dtype, s) for s in (1, 4, 7)]
    c = [sg.int8_checkpoint(x) for x, _ in made]
    torch.cuda.synchronize()
    expected = []
    for (_, dy), kept in zip(made, c):
        expected.append(sg.int8_weight_grad(dy, kept, out_dtype=out))
        torch.cuda.synchronize()
    check_gradient(expected[0], made[0][1], made[0][0], dtype == F16)
    one, dw, dy = c[0], torch.empty_like(expected[0]), torch.empty_strided(made[0][1].shape, made[0][1].stride(), dtype=dtype, device="cuda")
    for _ in range(3):
        for (x, d), e in zip(made, expected):
            sg.int8_checkpoint(x, out=one)
            dy.copy_(d)
            sg.int8_weight_grad(dy, one, out=dw)
            same(dw, e)


# ------------------------------------------------------------------- graphs and streams
def test_captured_and_replayed_in_tiles():
    linear, gemm = [(s, w) for s, q, w in PRODUCTS if not q], [(s, w) for s, q, w in PRODUCTS if q]
    xs = {s: values(s[0], s[2], BF16, 1) for s, _ in linear + gemm}
    ws = {s: sg.int8_quantize(values(s[1], s[2], F32, 2)) for s, _ in linear + gemm}
    grads = {g[:3]: gradient_inputs(g[0], g[1]) for g in GRADIENTS}

    def step():
        got = [sg.int8_linear(xs[s], ws[s]) for s, _ in linear] + [sg.int8_gemm(sg.int8_quantize(xs[s]), ws[s]) for s, _ in gemm]
        return got + [sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out_dtype=out) for (_, _, out), (x, dy) in grads.items()]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for seed in (3, 4):
        for size, x in xs.items():
            x.copy_(values(size[0], size[2], BF16, seed))
        for (size, dtype, _), (x, dy) in grads.items():
            new = gradient_inputs(size, dtype, 10 * seed)
            x.copy_(new[0])
            dy.copy_(new[1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            same(a, b)
    assert sg.query_device_status() == (0, 0)


def test_two_streams_at_once_in_tiles():
    """Each stream's scratch (tokens in 16 bits, terms of dY, shares of sums) is its own."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = []
    for i in range(2):
        for size, quantised, _ in PRODUCTS:
            x, w = values(size[0], size[2], BF16, 5 + i), sg.int8_quantize(values(size[1], size[2], F32, 7 + i))
            q = sg.int8_quantize(x)
            cases.append((i, (lambda q=q, w=w: sg.int8_gemm(q, w)) if quantised else (lambda x=x, w=w: sg.int8_linear(x, w))))
        for size, dtype, out, _ in GRADIENTS:
            x, dy = gradient_inputs(size, dtype, 20 + i)
            cases.append((i, lambda dy=dy, c=sg.int8_checkpoint(x), out=out: sg.int8_weight_grad(dy, c, out_dtype=out)))
    want = [call() for _, call in cases]
    torch.cuda.synchronize()
    half = len(cases) // 2
    for _ in range(4):
        got = [None] * len(cases)
        for j in range(half):
            for at in (j, half + (j + 5) % half):            # other calls of the other stream beside it
                with torch.cuda.stream(streams[cases[at][0]]):
                    got[at] = cases[at][1]()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same(a, b)
    assert sg.query_device_status() == (0, 0)


def test_a_passed_stream_is_used_in_tiles():
    s = torch.cuda.Stream()
    for size, quantised, _ in PRODUCTS[:4]:
        x, w = values(size[0], size[2], BF16), sg.int8_quantize(values(size[1], size[2], F32, 1))
        torch.cuda.synchronize()
        y = sg.int8_gemm(sg.int8_quantize(x, stream=s), w, stream=s) if quantised else sg.int8_linear(x, w, stream=s)
        s.synchronize()
        same(y, sg.int8_gemm(sg.int8_quantize(x), w) if quantised else sg.int8_linear(x, w))
    for size, dtype, out, _ in GRADIENTS:
        x, dy = gradient_inputs(size, dtype)
        torch.cuda.synchronize()
        dw = sg.int8_weight_grad(dy, sg.int8_checkpoint(x, stream=s), out_dtype=out, stream=s)
        s.synchronize()
        same(dw, sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out_dtype=out))


def test_scratch_grows_while_a_graph_of_tiles_lives():
    s = torch.cuda.Stream()
    size, _, want = PRODUCTS[2]
    planned_product(size, False, want)
    m, n, k = size
    w, x = sg.int8_quantize(values(n, k, F32)), values(m, k, BF16)
    grad, dtype, out, want = GRADIENTS[-1]
    planned_gradient(grad, dtype, out, want)
    gx, dy = gradient_inputs(grad, dtype)
    c = sg.int8_checkpoint(gx)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        wanted = sg.int8_linear(x, w), sg.int8_weight_grad(dy, c)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = sg.int8_linear(x, w), sg.int8_weight_grad(dy, c)
    big, wide = values(20000, k, BF16), values(20000, 2000, F32, 3)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        sg.int8_linear(big, w)
        sg.int8_weight_grad(wide, sg.int8_checkpoint(wide[:, :300]))
        for g in got:
            g.zero_()
        graph.replay()
    s.synchronize()
    for a, b in zip(got, wanted):
        same(a, b)


# ------------------------------------------------------------------------ values
@product_cases
def test_products_of_tokens_and_weights_that_are_not_finite(size, quantised, want):
    planned_product(size, quantised, want)
    m, n, k = size
    x = values(m, k, F32)
    x[1, 5], x[m - 1, k - 1] = float("nan"), float("inf")
    b, sb = integers(n, k, 3)
    sb[7], sb[n - 1] = np.nan, np.inf
    w = matrix(b, sb)
    y = (sg.int8_gemm(sg.int8_quantize(x), w) if quantised else sg.int8_linear(x, w))
    a, sa = ref.quantize(ref.array(x))
    same(y, ref.product(a, sa, b, sb, F32))
    assert y[1].isnan().all() and y[m - 1].isnan().all() and y[:, 7].isnan().all()


@product_cases
def test_scales_far_apart_in_tiles(size, quantised, want):
    if not quantised:
        pytest.skip("scales of unquantised tokens are those of their values")
    planned_product(size, quantised, want)
    m, n, k = size
    (a, _), (b, _) = integers(m, k, 4, -128), integers(n, k, 5, -128)
    sa, sb = np.full(m, 1e33, np.float32), np.full(n, 1e-36, np.float32)
    sa[1], sb[3], sb[4], sa[m - 1] = 3e-38, -1e30, 0, 1e-30
    same(sg.int8_gemm(matrix(a, sa), matrix(b, sb)), ref.product(a, sa, b, sb, F32))


def test_codes_behind_rows_are_not_used_in_tiles():
    """Columns that end within 16 bytes, and others' integers behind them in both operands."""
    for (m, n, k), quantised, want in PRODUCTS:
        if k % 16 == 0 or not quantised:
            continue
        planned_product((m, n, k), quantised, want)
        (a, sa), (b, sb) = integers(m, k, 1, -128), integers(n, k, 2, -128)
        held, pitch = [], (k + 15) // 16 * 16
        for q, s in ((a, sa), (b, sb)):
            memory = torch.full((len(q), pitch), 77, dtype=torch.int8, device="cuda")
            memory[:, :k] = torch.from_numpy(q).cuda()
            held.append(sg.int8_matrix(memory[:, :k], torch.from_numpy(s).cuda()))
            assert held[-1].codes.data_ptr() == memory.data_ptr()
        same(sg.int8_gemm(*held), ref.product(a, sa, b, sb, F32))


def eye(m, k, dtype, value=1.0):
    return torch.eye(m, k, dtype=F32, device="cuda").mul_(value).to(dtype)


@gradient_cases
def test_every_bit_of_a_gradient_counts_in_tiles(size, dtype, out, want):
    """Tokens that each hold one 1: the gradient's rows are dy's, all 24 bits of them."""
    planned_gradient(size, dtype, out, want)
    m, n, k, _ = size
    _, dy = gradient_inputs(size, dtype)
    for last in (False, True):                                 # the first tokens, or the last (which end within a stage)
        x, t = torch.zeros(m, k, dtype=dtype, device="cuda"), min(m, k)
        first = m - t if last else 0
        x[first:first + t] = eye(t, k, dtype)
        dw = sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out_dtype=out)
        same(dw[:, :t].contiguous(), dy[first:first + t].t().to(out).contiguous())
        assert (dw[:, t:] == 0).all()


@gradient_cases
@pytest.mark.parametrize("scale", [2.0 ** -14, 2.0 ** -20, 2.0 ** -24, 2.0 ** 8, 2.0 ** -100, 2.0 ** 100])
def test_gradients_far_from_one_in_tiles(size, dtype, out, want, scale):
    """Units and gradients at the ends of their types: tokens of one value each, so that dW is dY times it, exactly."""
    if dtype == F16 and not 2.0 ** -24 <= scale <= 2.0 ** 8:
        pytest.skip("beyond 16-bit floats of five exponent bits")
    if dtype == F16 and out == F16:
        pytest.skip("products beyond the type")
    planned_gradient(size, dtype, out, want)
    m, n, k, _ = size
    t = min(m, k)
    x = torch.zeros(m, k, dtype=dtype, device="cuda")
    x[:t] = eye(t, k, dtype, scale)
    c = sg.int8_checkpoint(x)
    _, dy = gradient_inputs(size, dtype)
    factor = 2.0 ** 10 if scale < 1 else 2.0 ** -6                # the product far from the type's ends
    dy.copy_((dy.float() * factor / 64).to(dtype))
    same(sg.int8_weight_grad(dy, c, out_dtype=out)[:, :t].contiguous(), (dy[:t].float() * scale).t().to(out).contiguous())
    if dtype != F16:
        # Large times small.  The last of a 32-bit gradient's terms ends where bfloat16 does, at 2^-133: what a gradient has
        # below that is cut off, less than 2^-133 of it, which the one product multiplies by the kept value.
        dy.copy_((dy.float() / scale * 2.0 ** -4).to(dtype))
        dw = sg.int8_weight_grad(dy, c, out_dtype=out)[:, :t]
        exact = dy[:t].double().t() * scale
        assert ((dw.double() - exact).abs() <= (2.0 ** -133 * scale if dtype == F32 else 0.0)).all()


@pytest.mark.parametrize("size,out,want", [(g[0], g[2], g[3]) for g in GRADIENTS if g[1] == F16])
def test_subnormal_gradients_in_tiles(size, out, want):
    planned_gradient(size, F16, out, want)
    m, n, k, _ = size
    t = min(m, k)
    x = torch.zeros(m, k, dtype=F16, device="cuda")
    x[:t] = eye(t, k, F16, 512.0)
    _, dy = gradient_inputs(size, F16)
    dy.copy_(((torch.arange(m * n, device="cuda").view(m, n) % 1001) - 500).half() * 2.0 ** -24)
    same(sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out_dtype=out)[:, :t].contiguous(), (dy[:t].float().t() * 512).to(out).contiguous())


@gradient_cases
def test_what_is_not_finite_stays_apart_in_tiles(size, dtype, out, want):
    """What is not finite in dy or in x reaches the sums that it is part of, and no others: first and last tokens, whose stages
    of a 32-bit gradient's terms lie beside the next term's, and values around dy's rows and behind its columns."""
    planned_gradient(size, dtype, out, want)
    m, n, k, ld = size
    x, _ = gradient_inputs(size, dtype)
    around = torch.full((m + 2, ld), float("nan"), dtype=dtype, device="cuda")
    dy = around[1:-1, :n]
    assert dy.stride(0) == ld
    dy.copy_(gradient_inputs(size, dtype)[1])
    clean = sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out_dtype=out)
    check_gradient(clean, dy, x, dtype == F16)
    x[7, 40], dy[m - 1, 3], dy[0, 9], dy[m - 2, n - 1] = float("nan"), float("inf"), float("nan"), -float("inf")
    got = sg.int8_weight_grad(dy, sg.int8_checkpoint(x), out_dtype=out)
    bad = torch.zeros(n, k, dtype=torch.bool, device="cuda")
    bad[:, 32:64] = bad[9] = True
    assert got[bad].isnan().all()
    assert not got[3].isfinite().any() and not got[n - 1].isfinite().any()
    bad[3] = bad[n - 1] = True
    same(got[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(1030, 520, 512, 520), (4100, 130, 130, 136), (2050, 1000, 700, 1000), (5000, 260, 300, 261)])
def test_gradients_in_32_bits_are_near(dtype, size):
    """Random values of both signs, 2-norm.  Products of 8 by 7 bits lose nothing in an accumulator until its sum is 2^9 times
    one of them; a sum of 512 tokens is cut where its exponent grows, each time below 2^-23 of it then, together 2 * 2^-23.  Its runs
    are added with 2^-24 each, in the mean the square root of their number (at most ten here): 2.4e-7 + 1.9e-7.  (Without a 32-bit
    gradient's third term 4e-6 is missing.)"""
    planned_gradient(size, dtype, F32)
    x, dy = gradient_inputs(size, dtype)
    c = sg.int8_checkpoint(x)
    want = dy.double().t() @ c.restore().double()
    got = sg.int8_weight_grad(dy, c, out_dtype=F32).double()
    assert (got - want).norm() <= 5e-7 * want.norm()
