"""Long sums of the experts' products, of one sign, against 64 bits.

The tensor cores cut each product off where it enters a sum, by less than 2^-25 of that sum (two
bits below FP32's last place).  Sums of products of one sign grow evenly, so that the cuts are of
half the result on average: n 2^-26 for n products.  A result is then rounded, by eps / 2."""
import pytest
import torch

from gpu_util import ensure_lib
from test_gpu_expert_gemm import BF16, FP16, FP32, order, product, wgrad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def positive(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.rand(shape, generator=g, device="cuda") + 1) * 2.0 ** -5).to(dtype)


def far(got, want):
    return ((got.double() - want) / want).abs().max().item()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("n", [4096, 1 << 15, 1 << 17])
def test_gradients_of_many_rows(n, dtype):
    """FP32: at most 768 rows to a sum, and an addition for each, half of the result on average."""
    c, o, _ = order([n])
    d, x = positive(n, 64, dtype=dtype, seed=1), positive(n, 72, dtype=dtype, seed=2)
    want = d.double().T @ x.double()
    assert far(wgrad(d, x, c, o, dtype)[0], want) <= torch.finfo(dtype).eps / 2 + n * 2.0 ** -26
    assert far(wgrad(d, x, c, o, FP32)[0], want) <= 768 * 2.0 ** -26 + (n / 768 + 1) * 2.0 ** -25


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows", [1, 6, 40, 300])     # dot products, few rows, cut sums, whole tiles
@pytest.mark.parametrize("n", [4096, 1 << 15])
def test_products_of_long_rows(n, rows, transpose, dtype):
    K, N = (264, n) if transpose else (n, 264)
    c, o, _ = order([rows])
    x, w = positive(rows, n, dtype=dtype, seed=3), positive(1, N, K, dtype=dtype, seed=4)
    want = x.double() @ (w[0].double() if transpose else w[0].double().T)
    assert far(product(x, w, c, o, transpose), want) <= torch.finfo(dtype).eps / 2 + n * 2.0 ** -26
