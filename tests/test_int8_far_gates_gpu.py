"""The gated activation where the sigmoid leaves the range of 32 bits and its products do not (GPU)."""
import numpy as np
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg

import int8_ref as ref
from test_int8_gpu import BF16, F16, F32, near, swiglu_bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def inputs(dtype, rows, cols, top):
    """Gates on both sides of -88.7, some far above; ups and gradients up to 10^top, of both signs."""
    gen = np.random.default_rng(rows)
    g = gen.uniform(-130, -60, (rows, cols))
    g[:, ::7] = gen.uniform(-190, -150, g[:, ::7].shape)
    g[:, 3::11] = gen.uniform(-10, 120, g[:, 3::11].shape)
    u, d = (gen.uniform(1, 10, (2, rows, cols)) * 10.0 ** gen.uniform(-5, top, (2, rows, cols))) * gen.choice([-1, 1], (2, rows, cols))
    return [torch.from_numpy(v).to(dtype).cuda() for v in (g, u, d)]


@pytest.mark.parametrize("dtype,top", [(F32, 37), (BF16, 37), (F16, 3)])
@pytest.mark.parametrize("rows,cols", [(3, 65), (9, 256), (700, 912)])
def test_far_gates(dtype, top, rows, cols):
    gate, up, _ = inputs(dtype, rows, cols, top)
    h, kept = sg.int8_swiglu(gate, up)
    g, u = ref.array(gate), ref.array(up)
    positive = g > 0
    want = ref.swiglu(g, u)
    big = positive & (np.abs(want) > torch.finfo(dtype).max)           # these overflow, as they should
    got = ref.array(h)
    assert np.isinf(got[big & (np.abs(want) > 1.01 * torch.finfo(dtype).max)]).all()
    h[torch.from_numpy(big).cuda()] = 0
    want[big] = 0
    near(h, want, swiglu_bounds(g, g, np.where(big, 0, u), dtype)[0], dtype)


@pytest.mark.parametrize("dtype,top", [(F32, 18), (BF16, 18), (F16, 2)])
@pytest.mark.parametrize("rows,cols", [(3, 65), (9, 256), (700, 912)])
def test_gradients_of_far_gates(dtype, top, rows, cols):
    gate, up, dh = inputs(dtype, rows, cols, top)
    _, kept = sg.int8_swiglu(gate, up)
    dgate, dup = sg.int8_swiglu_backward(dh, kept)
    g, u, d = ref.kept(ref.array(gate), dtype == F16), ref.kept(ref.array(up), dtype == F16), ref.array(dh)
    keep = np.abs(d * u) * np.maximum(1, np.abs(g)) < torch.finfo(dtype).max * (1 if dtype == F16 else 0.5)
    want, bounds = ref.swiglu_backward(d, g, u), swiglu_bounds(d, g, u, dtype)
    for out, w, b in ((dgate, want[0], bounds[1]), (dup, want[1], bounds[2])):
        there = keep & (np.abs(w) <= torch.finfo(dtype).max)           # others overflow, as they should
        out[torch.from_numpy(~there).cuda()] = 0
        near(out, np.where(there, w, 0), np.where(there, b, 0), dtype)


def test_one_gate_far_from_zero():
    """-88.8 with an up of 1e30 gives -2.4e-7: the sigmoid alone is below what 32 bits hold as 1 / (1 + e^88.8)."""
    for dtype in (F32, BF16):
        gate = torch.tensor([[-88.8, -100.0, -120.0, 88.8]], device="cuda").to(dtype)
        up = torch.full_like(gate, 1e30)
        h, kept = sg.int8_swiglu(gate, up)
        g, u = ref.array(gate), ref.array(up)
        assert np.allclose(ref.array(h), ref.swiglu(g, u), rtol=1e-6 + torch.finfo(dtype).eps / 2, atol=1e-38)
        ones = torch.ones_like(gate)
        dgate, dup = sg.int8_swiglu_backward(ones, kept)
        want = ref.swiglu_backward(1.0, ref.kept(g, False), ref.kept(u, False))
        for got, w in zip((dgate, dup), want):
            assert np.allclose(ref.array(got), w, rtol=1e-6 + torch.finfo(dtype).eps / 2, atol=1e-38)


def test_far_gates_that_are_not_finite():
    gate = torch.full((1, 64), -90.0, device="cuda")
    up = torch.full((1, 64), 1e30, device="cuda")
    gate[0, 0], up[0, 1], gate[0, 2], up[0, 40] = float("nan"), float("inf"), float("inf"), float("nan")
    h, _ = sg.int8_swiglu(gate, up)
    assert h[0, 0].isnan() and h[0, 1] == -float("inf") and h[0, 2] == float("inf") and h[0, 40].isnan()
    rest = [i for i in range(64) if i not in (0, 1, 2, 40)]
    assert h[0, rest].isfinite().all() and (h[0, rest] < 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_far_gates_of_many_values(dtype):
    """One far gate in a matrix whose blocks of threads have many steps: it alone changes."""
    rows, cols = 3000, 4104
    gen = torch.Generator(device="cuda").manual_seed(0)
    both = torch.randn(rows, 2 * cols, generator=gen, device="cuda").to(dtype)
    gate, up, dh = both[:, :cols], both[:, cols:], torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)
    h0, kept = sg.int8_swiglu(gate, up)
    d0 = sg.int8_swiglu_backward(dh, kept)
    spots = [(0, 0), (1, 4103), (1500, 2222), (2999, 4096)]
    for i, j in spots:
        gate[i, j], up[i, j] = -101.0, 1e30
    h1, kept = sg.int8_swiglu(gate, up)
    d1 = sg.int8_swiglu_backward(dh, kept)
    at = torch.zeros(rows, cols, dtype=torch.bool, device="cuda")
    for i, j in spots:
        at[i, j] = True
    assert (h1[~at] == h0[~at]).all()
    block = torch.zeros_like(at)                                # others of these blocks are kept in coarser units
    for i, j in spots:
        block[i, j // 32 * 32:j // 32 * 32 + 32] = True
    for a, b in zip(d0, d1):
        assert (a[~block] == b[~block]).all() and b.isfinite().all()
    g, u = ref.array(gate[at]), ref.array(up[at])
    assert np.allclose(ref.array(h1[at]), ref.swiglu(g, u), rtol=1e-6 + torch.finfo(dtype).eps / 2)
