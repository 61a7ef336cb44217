"""The gated activation and its gradients against the formulas in 64 bits.

Tolerances: with eps/2 a type's rounding step, a result of FP32 arithmetic that
is rounded once is off by at most eps/2 of itself, plus what FP32 costs.  The
exponential of -|g| is off by at most (2 + 1.16 |g|) units of 2^-23 (the
documented bound of the fast one), a dozen further operations by one unit each:
(14 + 1.2 |g|) 2^-23 of the sum of the magnitudes that are added.  FP16 adds
half its smallest step, 2^-25.
"""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord
from w4a16_int4_weight_sigmoid_gb300.layer import ExpertOrder

from gpu_util import ensure_lib
from test_gpu_mxfp8 import oracle as in_8_bits

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
LEFT = 7.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def close(got, want, magnitude, g, dtype):
    """want, and the sum of magnitudes behind it, in 64 bits."""
    tol = torch.finfo(dtype).eps / 2 * want.abs() * 1.0001 + (14 + 1.2 * g.abs()) * 2.0 ** -23 * magnitude
    tol = tol + (2.0 ** -25 if dtype == FP16 else 1e-38)
    assert torch.isfinite(got).all()
    worst = ((got.double() - want).abs() - tol).max().item()
    assert worst <= 0, worst


def case(M, E, local, topk, block, I, dtype, seed=0, scale=3.0):
    order = ExpertOrder(M, topk, 0, local, block).route(randn(M, E, seed=seed), torch.zeros(E, device="cuda"))
    cap, n = order.capacity, M * topk
    gu = (randn(cap, 2 * I, seed=seed + 1) * scale).to(dtype)
    dh = randn(cap, I, seed=seed + 2).to(dtype)
    f = order.sorted_token_ids.long()
    total = order.num_tokens_post_padded.item()
    filled = (f < n) & (torch.arange(cap, device="cuda") < total)
    gu[~filled], dh[~filled] = float("nan"), float("inf")        # reaches no result
    return order, gu, dh, f.clamp(0, n - 1), filled, total


def check(M, E, local, topk, block, I, dtype, keep, strided=False):
    order, gu, dh, f, filled, total = case(M, E, local, topk, block, I, dtype)
    cap, n = order.capacity, M * topk
    weights = order.topk_weights

    def rows(width):
        if strided:   # one element further on, and rows apart
            return torch.full((cap, width + 3), LEFT, dtype=dtype, device="cuda")[:, 1:1 + width]
        return torch.full((cap, width), LEFT, dtype=dtype, device="cuda")

    if strided:
        wide_gu, wide_dh = rows(2 * I), rows(I)
        wide_gu.copy_(gu), wide_dh.copy_(dh)
        gu, dh = wide_gu, wide_dh
    h, again, dgu = rows(I), rows(I), rows(2 * I)
    dw = torch.full((M, topk), LEFT, device="cuda")
    codes = scales = None
    if keep:
        codes = torch.empty((cap, 2 * I), dtype=torch.uint8, device="cuda")
        scales = torch.empty((cap, 2 * I // 32), dtype=torch.uint8, device="cuda")
    chord.chord_swiglu(gu, weights, order.sorted_token_ids, order.num_tokens_post_padded, h, codes, scales)
    chord.chord_swiglu_backward(dh, None if keep else gu, codes, scales, weights, order.sorted_positions,
                                order.sorted_token_ids, order.num_tokens_post_padded, dgu, dw, again)

    w = weights.double().reshape(-1)[f][filled][:, None]
    x, d = gu.double()[filled], dh.double()[filled]

    def forward(x):
        g, u = x[:, :I], x[:, I:]
        return w * g * torch.sigmoid(g) * u, g

    want, g = forward(x)
    close(h[filled], want, want.abs(), g, dtype)
    if keep:
        want_codes, want_scales, values = in_8_bits(gu[filled])
        assert torch.equal(codes[filled].cpu(), want_codes) and torch.equal(scales[filled].cpu(), want_scales)
        x = values.cuda()
        want, g = forward(x)
    close(again[filled], want, want.abs(), g, dtype)
    u, s = x[:, I:], torch.sigmoid(g)
    slope, size = s + g * s * (1 - s), s + g.abs() * s * (1 - s)
    close(dgu[filled][:, :I], w * d * u * slope, (w * d * u).abs() * size, g, dtype)
    close(dgu[filled][:, I:], w * d * g * s, (w * d * g * s).abs(), g, dtype)
    # the sum of I terms, each off by (14 + 1.2 |g|) units, in any order
    terms = d * g * s * u
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    tol = want.clone()
    want[f[filled]] = terms.sum(1)
    tol[f[filled]] = (terms.abs() * (14 + 1.2 * g.abs() + I)).sum(1) * 2.0 ** -23
    assert ((dw.reshape(-1).double() - want).abs() <= tol).all()
    # padding rows are zeros, rows behind them are left
    pad = ~filled
    pad[total:] = False
    for t in (h, again, dgu):
        assert (t[pad] == 0).all() and (t[total:] == LEFT).all()
    if strided:
        assert all((t._base[:, 0] == LEFT).all() and (t._base[:, -2:] == LEFT).all() for t in (h, again, dgu))


SIZES = [(1, 8, 8, 2, 8, 32), (37, 12, 5, 3, 16, 160), (300, 48, 48, 8, 64, 2048), (900, 8, 8, 2, 128, 96)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("M,E,local,topk,block,I", SIZES)
def test_gated(M, E, local, topk, block, I, dtype, keep):
    check(M, E, local, topk, block, I, dtype, keep)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("I", [1, 7, 30, 333, 1031, 4100])
def test_row_lengths_that_no_vector_divides(I, dtype):
    check(45, 12, 5, 3, 16, I, dtype, False)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("keep", [False, True])
def test_strides_and_alignment(dtype, keep):
    check(45, 12, 5, 3, 16, 64, dtype, keep, strided=True)


def test_gates_far_from_zero():
    """silu and its slope keep their relative accuracy where the exponential is tiny, and end in zeros and the
    gate itself; no NaN from 0 * inf."""
    order = ExpertOrder(1, 1, 0, 1, 8).route(torch.zeros(1, 1, device="cuda"), torch.zeros(1, device="cuda"))
    g = torch.tensor([-200.0, -100, -88, -87, -50, -20, 20, 50, 87, 88, 100, 200], device="cuda")
    I = g.numel()
    gu = torch.zeros((order.capacity, 2 * I), device="cuda")
    gu[0, :I], gu[0, I:] = g, 2.0
    dh = torch.ones((order.capacity, I), device="cuda")
    h, dgu, dw = torch.empty_like(dh), torch.empty_like(gu), torch.empty((1, 1), device="cuda")
    o = (order.sorted_token_ids, order.num_tokens_post_padded)
    chord.chord_swiglu(gu, order.topk_weights, *o, h)
    chord.chord_swiglu_backward(dh, gu, None, None, order.topk_weights, order.sorted_positions, *o, dgu, dw)
    x = g.double()
    silu, slope = x * torch.sigmoid(x), torch.sigmoid(x) * (1 + x * torch.sigmoid(-x))
    tol = 20 * 2.0 ** -23
    assert torch.allclose(h[0].double(), 2 * silu, rtol=tol, atol=2.0 ** -125)
    assert torch.allclose(dgu[0, I:].double(), silu, rtol=tol, atol=2.0 ** -125)
    assert torch.allclose(dgu[0, :I].double(), 2 * slope, rtol=tol, atol=2.0 ** -125)


def test_gradient_against_differences():
    """dgu and dweights against differences of the forward pass, in FP32: a step of 2^-6 leaves an error of its
    square times a third derivative below 4, and 2^-23 / 2^-6 of the sums."""
    M, I = 5, 16
    order, gu, dh, f, filled, _ = case(M, 4, 4, 2, 8, I, FP32, scale=1.0)
    gu[~filled], dh[~filled] = 0.0, 0.0
    o = (order.sorted_token_ids, order.num_tokens_post_padded)
    w = order.topk_weights.clone()

    def loss(gu, w):
        h = torch.zeros((order.capacity, I), device="cuda")
        chord.chord_swiglu(gu, w, *o, h)
        return (h.double() * dh.double()).sum().item()

    dgu, dw = torch.zeros_like(gu), torch.empty_like(w)
    chord.chord_swiglu_backward(dh, gu, None, None, w, order.sorted_positions, *o, dgu, dw)
    step = 2.0 ** -6
    row = filled.nonzero()[:, 0]
    for r, c in ((row[0], 3), (row[2], I + 5), (row[-1], 0), (row[-1], 2 * I - 1)):
        a, b = gu.clone(), gu.clone()
        a[r, c] += step
        b[r, c] -= step
        size = 4 * dh[r, c % I].abs().item() * (1 + gu[r].abs().max().item()) + 1
        assert abs((loss(a, w) - loss(b, w)) / (2 * step) - dgu[r, c].item()) <= size * (step ** 2 + 2.0 ** -16)
    for t, j in ((0, 0), (4, 1)):
        a, b = w.clone(), w.clone()
        a[t, j] += step
        b[t, j] -= step
        assert abs((loss(gu, a) - loss(gu, b)) / (2 * step) - dw[t, j].item()) <= 2.0 ** -14 * (1 + dw.abs().max().item())
