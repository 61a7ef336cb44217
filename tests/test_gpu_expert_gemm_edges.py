"""Ends of the experts' products that decide what may reach a result: the rows behind an expert's
last one in every place of a last box.

Operands are small integers, so results are exact (see test_gpu_expert_gemm.py)."""
import pytest

from test_gpu_expert_gemm import BF16, FP16, FP32, check_product, check_wgrad

pytestmark = pytest.mark.gpu


# boxes of 64 rows before the last one: none, two (three boxes an item), as many as the ring has
# stages, and more than an FP32 sum takes at once
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (FP16, FP16), (BF16, FP32)])
@pytest.mark.parametrize("boxes", [0, 1, 2, 6, 13])
def test_every_remainder_of_rows(boxes, dtype, out_dtype):
    """Experts whose rows end at each place of a box, NaN behind them, in both operands: two tiles of dW a side, so
    that both CTAs of a pair hold rows to be left out."""
    counts = [64 * boxes + r for r in range(1, 65)]
    check_wgrad(counts, 264, 520, dtype, out_dtype, gaps=[1 + i % 17 for i in range(64)], extra=70)


@pytest.mark.parametrize("count", [129, 191, 200, 385, 1000])
def test_many_tiles_of_one_remainder(count):
    """Each tile has its last box: tiles follow one another in every place of the ring."""
    check_wgrad([count, 0, count + 5], 1544, 2056, BF16, BF16, gaps=[2, 3, 1], extra=66)


@pytest.mark.parametrize("out_dtype", [BF16, FP32])
@pytest.mark.parametrize("counts", [list(range(1, 65)), [64, 0, 16, 48] * 16, [64] * 32 + [65] * 32])
def test_a_large_gradient_of_few_rows(counts, out_dtype):
    """64 x 1544 x 1544 is past the size from which the zeroing warps set the pace, for every remainder and none."""
    check_wgrad(counts, 1544, 1544, BF16, out_dtype, gaps=[i % 3 for i in range(64)], extra=66)
