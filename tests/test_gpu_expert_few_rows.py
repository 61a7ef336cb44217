"""The experts' product for a handful of rows: orders that the capacity does not tell apart, from
one row an expert to all rows in one, rows in groups of eight with every remainder.

Operands are small integers, so results are exact (see test_gpu_expert_gemm.py)."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord

from gpu_util import ensure_lib
from test_gpu_expert_gemm import BF16, FP16, LEFT, check_product, order, rows_of, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("counts,K,N", [
    ([8] * 16, 1024, 1024), ([0] * 5 + [128] + [0] * 10, 1024, 1024), ([1] * 128, 264, 136),
    ([40, 30, 20, 12, 8, 6, 4, 2, 2, 1, 1, 1, 1, 0, 0, 0], 520, 1000), ([0, 127, 1] + [0] * 13, 72, 264),
    ([2] * 64, 2048, 512), ([100] + [0] * 31, 8, 8), ([64] + [0] * 7, 7168, 24), ([3, 5] * 16, 40, 2056),
])
def test_packed_orders(counts, K, N, dtype):
    check_product(counts, K, N, False, dtype)


@pytest.mark.parametrize("rows", list(range(1, 18)))
def test_every_number_of_rows(rows):
    """Groups of eight and what is left, NaN between the experts' rows."""
    check_product([rows, 0, rows] + [0] * 5, 328, 200, False, BF16, gaps=[2] * 8, extra=1)


@pytest.mark.parametrize("K", [8, 24, 32, 40, 128, 136, 256, 264, 520, 4096, 4104])
def test_ends_of_the_contraction(K):
    check_product([5, 1, 2, 0, 9] + [0] * 11, K, 72, False, FP16, gaps=[1] * 16)


@pytest.mark.parametrize("counts", [[1] * 8, [8] * 8, [3, 0, 1, 12, 2, 5, 1, 6]])
def test_random_values_and_repetition(counts):
    """Sums of K products in FP32 are off by at most K 2^-23 of the sum of the magnitudes, in any order, and one
    rounding to BF16 by 2^-8 of the result; a call repeats itself bit for bit."""
    K, N = 1000, 520
    g = torch.Generator(device="cuda").manual_seed(7)
    c, o, rows = order(counts)
    x = torch.randn((rows, K), generator=g, device="cuda").to(BF16)
    w = torch.randn((len(counts), N, K), generator=g, device="cuda").to(BF16)
    outs = []
    for _ in range(2):
        out = torch.full((rows, N), LEFT, dtype=BF16, device="cuda")
        chord.chord_expert_gemm(x, w, c, o, out, workspace())
        outs.append(out)
    assert torch.equal(*outs)
    for e, at in rows_of(c, o):
        want, size = x[at].double() @ w[e].double().T, x[at].double().abs() @ w[e].double().abs().T
        assert ((outs[0][at].double() - want).abs() <= 2.0 ** -8 * want.abs() + K * 2.0 ** -23 * size).all()
