"""Weight gradients over many tokens: what the tensor core's accumulators cut off does not grow with them (GPU).

An accumulator adds 16 tokens at a time and cuts off what is below its last place.  Measured on sums of one sign, where the cuts add
up, that is at most 6.5e-9 of the sum a token.  A bfloat16 result's accumulators take at most 16384 tokens (1.1e-4 of the
sum: 2^-13.2), an fp16 result's 2048 (1.4e-5: 2^-16.2), a 32-bit one's 512 (3.4e-6: 2^-18.2), and what leaves them is added with
correct rounding (2^-24 of the sum each time, at most 2^20 / 512 times, 2^-13, if all went one way; they do not: the square root
of their number, 2^-18.5).  CUT is about twice the first: 1/16 of half a step of the 16-bit types.
"""
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg

import int8_plans
from test_int8_gpu import check_gradient, same, values

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
CUT = {BF16: 2.0 ** -12, F16: 2.0 ** -15, F32: 2.0 ** -17}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def positive(rows, cols, dtype, seed, scale):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, cols, dtype=dtype, device="cuda")
    for i in range(0, rows, 65536):
        x[i:i + 65536] = (torch.rand(min(65536, rows - i), cols, generator=gen, device="cuda") + 0.5) * scale
    return x


def in_64_bits(dy, kept):
    total = torch.zeros(dy.shape[1], kept.shape[1], dtype=torch.float64, device="cuda")
    for i in range(0, dy.shape[0], 16384):
        total += dy[i:i + 16384].double().t() @ kept[i:i + 16384].double()
    return total


def half_spacing(v, dtype):
    """Half the distance of `dtype`'s numbers at |v|."""
    return torch.finfo(dtype).eps / 2 * torch.exp2(torch.floor(torch.log2(v.abs())))


@pytest.mark.parametrize("out", ["own", "float32"])
@pytest.mark.parametrize("dtype,m,n,k", [(F16, 20000, 2048, 1600), (F16, 100000, 1500, 1024), (BF16, 262144, 2432, 1024), (BF16, 40000, 2048, 2048),
                                         (F16, 1 << 20, 8, 32), (BF16, 1 << 20, 8, 32)])
def test_sums_of_one_sign(dtype, m, n, k, out):
    kind = dtype if out == "own" else F32
    # Sums near 2^13: within the range of fp16.
    x, dy = positive(m, k, dtype, 1, 0.25), positive(m, n, dtype, 2, 2.0 ** 15 / m)
    dy *= torch.linspace(0.5, 1.0, n, device="cuda").to(dtype)          # sums all over a binade
    c = sg.int8_checkpoint(x)
    rows = torch.arange(0, n, max(1, n // 16), device="cuda")
    want = in_64_bits(dy[:, rows], c.restore())
    dw = sg.int8_weight_grad(dy, c, out_dtype=kind)[rows].double()
    assert ((dw - want).abs() <= CUT[kind] * want.abs() + half_spacing(want, kind)).all()
    if kind == F32:
        assert ((dw - want) / want).mean().abs() <= 2.0 ** -18.2         # what 512 tokens lose, and no more
    assert sg.query_device_status() == (0, 0)


@pytest.mark.parametrize("dtype,m,n,k", [(F16, 9000, 2001, 1056), (F16, 12289, 1793, 2079), (BF16, 33000, 2100, 1100)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_sums_that_leave_wide_tiles(dtype, m, n, k, accumulate):
    """Tiles of 256 columns whose sums leave the accumulator every 2048 tokens: ragged ones, part of a larger output, added to it."""
    p = int8_plans.gradient(m, n, k, dtype, aligned=False)
    assert (p.small, p.cols, p.run) == (0, 256, 16)
    x, dy = values(m, k, dtype, 1), values(m, n, dtype, 2, 1, 0.1)
    around = torch.full((n + 2, k + 5), 3.0, dtype=dtype, device="cuda")
    out = around[1:-1, 2:-3]
    before = out.clone()
    c = sg.int8_checkpoint(x)
    sg.int8_weight_grad(dy, c, out=out, accumulate=accumulate)
    some = [0, 1, n // 2, n - 2, n - 1]
    want = in_64_bits(dy[:, some], c.restore()) + (3.0 if accumulate else 0.0)
    size = dy[:, some].abs().double().t() @ c.restore().abs().double() + 3.0
    err = (out[some].double() - want).abs()
    # The cuts, relative to the largest partial sum, which the sum of magnitudes bounds.
    assert (err <= CUT[dtype] / 4 * size + torch.finfo(dtype).eps / 2 * want.abs() + (2.0 ** -25 if dtype == F16 else 0)).all()
    first = out.clone()
    out.copy_(before)
    sg.int8_weight_grad(dy, c, out=out, accumulate=accumulate)
    same(out, first)
    out.fill_(3.0)
    assert (around == 3.0).all()
    assert sg.query_device_status() == (0, 0)
