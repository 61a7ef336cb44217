"""Rows in 8 bits (MXFP8): codes, scales and values, bit for bit against an
implementation by search in 64 bits on the CPU."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord
from w4a16_int4_weight_sigmoid_gb300.layer import ExpertOrder

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
# E4M3 magnitudes by code, 0x7f (NaN) left out
LEVELS = torch.tensor([m * 2.0 ** -9 for m in range(8)]
                      + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1], dtype=torch.float64)
POWERS = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def oracle(x):
    """(codes, scales, values in 64 bits) of x [rows, K] on the CPU."""
    b = x.double().cpu().reshape(x.shape[0], -1, 32)
    fine = b.isfinite().all(-1, keepdim=True)
    v = torch.where(fine, b, 0.0)
    scale = torch.searchsorted(POWERS * 448, v.abs().amax(-1, keepdim=True))
    a = v.abs() / POWERS[scale]
    code = torch.searchsorted((LEVELS[1:] + LEVELS[:-1]) / 2, a)     # a tie goes to the lower code here
    tie = (code < 126) & (a == ((LEVELS[1:] + LEVELS[:-1]) / 2)[code.clamp(max=125)])
    code = code + (tie & (code % 2 == 1))
    code = torch.where(scale == 247, code.clamp(max=int((LEVELS == 240).nonzero())), code)
    values = torch.where(fine, LEVELS[code] * POWERS[scale] * torch.where(v.signbit(), -1.0, 1.0), float("nan"))
    bits = torch.where(fine, code + 128 * v.signbit(), 0)
    return (bits.reshape(x.shape).to(torch.uint8), torch.where(fine, scale, 255)[..., 0].to(torch.uint8),
            values.reshape(x.shape))


def quantize(x):
    rows, K = x.shape
    codes = torch.full((rows, K), 99, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, K // 32), 99, dtype=torch.uint8, device="cuda")
    chord.chord_mxfp8_quantize(x, codes, scales)
    return codes, scales


def in_type(values, dtype):
    """64-bit values rounded to a type as `dequantize` does."""
    out = values.float()          # exact: 4 bits and a power of two from 2^-136 on
    if dtype == FP16:
        out = out.clamp(-65504, 65504)
    return out.to(dtype)


def check(x):
    codes, scales = quantize(x)
    want_codes, want_scales, values = oracle(x)
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(codes.cpu() & 127, want_codes & 127)
    # (the sign of a zero code is the value's)
    assert torch.equal(codes.cpu(), want_codes)
    out = torch.empty(x.shape, dtype=x.dtype, device="cuda")
    chord.chord_mxfp8_dequantize(codes, scales, out)
    want = in_type(values, x.dtype)
    assert torch.equal(out.cpu().isnan(), want.isnan())
    assert torch.equal(out.cpu().nan_to_num(), want.nan_to_num())


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (70, 7168), (513, 416), (5000, 64)])
def test_random_rows(rows, K, dtype):
    check((randn(rows, K) * (1 + 9 * (randn(K, seed=1) > 2))).to(dtype))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_every_code_and_tie(dtype):
    """All E4M3 magnitudes and the middles between them, in blocks whose scale is 1 and 2^-3."""
    mid = (LEVELS[1:] + LEVELS[:-1]) / 2
    v = torch.cat([LEVELS, mid, -mid]).float()
    v = torch.cat([v, v.new_zeros(-v.numel() % 31)]).reshape(-1, 31)
    x = torch.cat([v.new_full((v.shape[0], 1), 448.0), v], 1)
    check(torch.cat([x, x * 0.125]).to(dtype).cuda())


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_borders_of_the_scale_and_the_type(dtype):
    top = torch.finfo(dtype).max
    x = torch.zeros(10, 64, dtype=torch.float64)
    x[0] = 448
    x[1], x[1, 5] = 1, 450                       # the next scale
    x[2] = torch.linspace(-1, 1, 64) * top
    x[3] = top
    x[4] = torch.finfo(dtype).tiny               # (subnormals below)
    x[5, ::3] = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    x[6, 40] = float("inf")
    x[7, 3] = float("nan")
    x[8] = -0.0
    x[9] = top / 2 * torch.linspace(0.9, 1.1, 64)
    check(x.to(dtype).cuda())


@pytest.mark.parametrize("dtype,offset,gap", [(BF16, 1, 3), (BF16, 8, 8), (FP16, 2, 2), (FP32, 1, 1), (FP32, 4, 4)])
def test_strides_and_alignment(dtype, offset, gap):
    """Rows at any element, further apart than they are long; what lies between is left."""
    rows, K = 37, 160
    wide = randn(rows, K + offset + gap).to(dtype)
    x = wide[:, offset:offset + K]
    codes, scales = quantize(x)
    want_codes, want_scales, values = oracle(x)
    assert torch.equal(scales.cpu(), want_scales) and torch.equal(codes.cpu(), want_codes)
    out = torch.full_like(wide, 7.0)
    chord.chord_mxfp8_dequantize(codes, scales, out[:, offset:offset + K])
    assert torch.equal(out[:, offset:offset + K].cpu(), in_type(values, dtype))
    out[:, offset:offset + K] = 7.0
    assert (out == 7.0).all()


def test_one_row_for_all():
    x = randn(1, 64).bfloat16().expand(9, 64)
    codes, scales = quantize(x)
    assert torch.equal(codes.cpu(), oracle(x)[0]) and (scales == scales[0]).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("M,K,block", [(1, 7168, 8), (37, 96, 16), (600, 256, 128)])
def test_permute(M, K, block, dtype):
    """The values of each token's row in its experts' places, zeros in padding, the rest left."""
    E, topk = 12, 3
    order = ExpertOrder(M, topk, 2, 5, block).route(randn(M, E), torch.zeros(E, device="cuda"))
    x = randn(M, K, seed=3).to(dtype)
    codes, scales = quantize(x)
    rows = torch.full((order.capacity, K), 7.0, dtype=dtype, device="cuda")
    chord.chord_mxfp8_permute(codes, scales, order.sorted_positions, order.sorted_token_ids,
                              order.num_tokens_post_padded, topk, rows)
    values = in_type(oracle(x)[2], dtype)
    total = order.num_tokens_post_padded.item()
    f = order.sorted_token_ids.cpu().long()[:total]        # (entries past the total hold anything)
    want = torch.full(rows.shape, 7.0, dtype=dtype)
    want[:total] = torch.where((f < M * topk)[:, None], values[f.clamp(max=M * topk - 1) // topk], 0.0)
    assert torch.equal(rows.cpu(), want)
