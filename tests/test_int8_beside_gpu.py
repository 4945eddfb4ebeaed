"""Operands of the 8-bit integer operators that lie between one another's rows (GPU)."""
import pytest
import torch

import dense_fp32_gemm_03_gb300 as sg

from test_int8_gpu import BF16, F32, same, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 33, 70), (2, 33, 70), (7, 256, 512), (40, 65, 129), (600, 1024, 1000)])
def test_a_layer_writes_beside_its_input(dtype, m, n, k):
    """x and y are parts of the rows of one tensor; they share no memory."""
    w = sg.int8_quantize(values(n, k, F32, 1))
    for first in (True, False):
        both = values(m, n + k + 5, dtype, 2)
        before = both.clone()
        x, y = (both[:, 2:k + 2], both[:, k + 3:k + 3 + n]) if first else (both[:, n + 4:n + 4 + k], both[:, 1:n + 1])
        want = sg.int8_linear(x.contiguous(), w)
        sg.int8_linear(x, w, out=y)
        same(y.contiguous(), want)
        y.zero_()
        (before[:, k + 3:k + 3 + n] if first else before[:, 1:n + 1]).zero_()
        same(both, before)


@pytest.mark.parametrize("m", [1, 2, 40])
def test_a_layer_over_its_input_is_refused(m):
    n, k = 33, 70
    w = sg.int8_quantize(values(n, k, F32, 1))
    both = values(m, n + k, F32, 2)
    for x, y in ((both[:, :k], both[:, k - 1:k - 1 + n]), (both[:, n:], both[:, 1:n + 1]), (both[:, :k], both[:, 5:5 + n])):
        with pytest.raises(sg.SgemmError):
            sg.int8_linear(x, w, out=y)
