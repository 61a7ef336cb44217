"""How far 8 bits are from what they hold: 2^-4 of a value, or 2^-10 of its block's scale where that is more."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord

from gpu_util import ensure_lib
from test_gpu_mxfp8 import BF16, FP16, FP32, quantize, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_blocks_with_an_outlier(dtype):
    """From no outlier to one that leaves the other values nothing.  (FP16 rounds what it reads by up to half its
    smallest step.)"""
    x = (randn(64, 128) * 2.0 ** -4).to(dtype)
    top = 15 if dtype == FP16 else 40
    x[:, ::32] = (2.0 ** torch.linspace(-4, top, 64, device="cuda"))[:, None].to(dtype)
    codes, scales = quantize(x)
    got = torch.empty(x.shape, device="cuda")
    chord.chord_mxfp8_dequantize(codes, scales, got)
    scale = 2.0 ** (scales.double() - 127).repeat_interleave(32, 1)
    v = x.double()
    bound = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * scale)
    assert ((got.double() - v).abs() <= bound).all()
    # the scale is the smallest with which the block's largest value is held
    amax = v.abs().reshape(64, 4, 32).amax(-1).repeat_interleave(32, 1)
    assert (amax <= 448 * scale).all() and (amax > 224 * scale).all()
    typed = torch.empty_like(x)
    chord.chord_mxfp8_dequantize(codes, scales, typed)
    assert ((typed.double() - v).abs() <= bound + (2.0 ** -25 if dtype == FP16 else 0)).all()
    # such values do fall to zero, which 2^-4 of a value does not allow
    assert ((got == 0) & (v != 0)).any()
