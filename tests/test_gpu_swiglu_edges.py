"""The gated activation at the ends of the range: infinities, NaN and the largest values in rows
that hold assignments, and the forward pass's rows made again."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord
from w4a16_int4_weight_sigmoid_gb300.layer import ExpertOrder

from gpu_util import ensure_lib
from test_gpu_swiglu import BF16, FP16, FP32, case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def passes(order, gu, dh, weights, keep=False):
    cap, I = dh.shape
    h, again, dgu = torch.zeros_like(dh), torch.zeros_like(dh), torch.zeros_like(gu)
    dw = torch.empty_like(weights)
    kept = (torch.zeros((cap, 2 * I), dtype=torch.uint8, device="cuda"),
            torch.zeros((cap, I // 16), dtype=torch.uint8, device="cuda")) if keep else (None, None)
    o = (order.sorted_token_ids, order.num_tokens_post_padded)
    chord.chord_swiglu(gu, weights, *o, h, *kept)
    chord.chord_swiglu_backward(dh, None if keep else gu, *kept, weights, order.sorted_positions, *o, dgu, dw, again)
    return h, again, dgu, dw, kept


# (gate, silu, silu'): the limits at both ends
INF = float("inf")
ENDS = [(INF, INF, 1.0), (-INF, 0.0, 0.0), (float("nan"), float("nan"), float("nan"))]


@pytest.mark.parametrize("I", [32, 37])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_gates_at_the_ends(dtype, I):
    """One gate of each row at an end (powers of two elsewhere, so that results are exact but for the gate's own
    function): infinities stay infinities, -inf gates give 0, NaN stays where it is."""
    top = torch.finfo(dtype).max
    ends = ENDS + [(top, top, 1.0), (-top, 0.0, 0.0)]
    M = len(ends)
    order = ExpertOrder(M, 1, 0, 1, 8).route(torch.zeros(M, 1, device="cuda"), torch.zeros(1, device="cuda"))
    weights = torch.full((M, 1), 0.5, device="cuda")
    gu = torch.zeros((order.capacity, 2 * I), dtype=dtype, device="cuda")
    dh = torch.zeros((order.capacity, I), dtype=dtype, device="cuda")
    at = order.sorted_positions.long()
    gu[at, I:], dh[at] = -0.5, 0.25
    for i, (g, _, _) in enumerate(ends):
        gu[at[i], i] = g
    h, again, dgu, dw, _ = passes(order, gu, dh, weights)
    for i, (_, silu, slope) in enumerate(ends):
        want_h, want_up = torch.zeros(I, dtype=torch.float64), torch.zeros(I, dtype=torch.float64)
        want_gate = torch.full((I,), 0.5 * 0.25 * -0.5 * 0.5, dtype=torch.float64)     # silu'(0) = 1/2
        want_h[i], want_up[i], want_gate[i] = 0.5 * silu * -0.5, 0.5 * 0.25 * silu, 0.5 * 0.25 * -0.5 * slope
        for got in (h, again):
            assert torch.equal(got[at[i]].cpu().double().nan_to_num(7, 8, 9), want_h.nan_to_num(7, 8, 9))
        d = dgu[at[i]].cpu().double()
        assert torch.equal(d[:I].nan_to_num(7, 8, 9), want_gate.nan_to_num(7, 8, 9))
        assert torch.equal(d[I:].nan_to_num(7, 8, 9), want_up.nan_to_num(7, 8, 9))
        want = torch.tensor(0.25 * silu * -0.5)
        assert torch.equal(dw[i, 0].cpu().nan_to_num(7, 8, 9), want.nan_to_num(7, 8, 9))


def test_an_infinite_gate_while_rows_are_kept():
    """The rows of h are of gu itself; a block with an infinity reads as NaN in the backward pass, others do not."""
    order = ExpertOrder(2, 1, 0, 1, 8).route(torch.zeros(2, 1, device="cuda"), torch.zeros(1, device="cuda"))
    gu = torch.ones((order.capacity, 128), dtype=BF16, device="cuda")
    at = order.sorted_positions.long()
    gu[at[0], 3] = INF
    h, again, dgu, dw, _ = passes(order, gu, torch.ones_like(gu[:, :64]), torch.ones((2, 1), device="cuda"), keep=True)
    assert h[at[0], 3] == INF and torch.isfinite(h[at[0], 4:]).all()
    assert again[at[0], :32].isnan().all() and torch.equal(again[at[0], 32:], h[at[0], 32:])
    assert dgu[at[0], :32].isnan().all() and torch.isfinite(dgu[at[0], 32:64]).all()
    assert torch.isfinite(dgu[at[1]]).all() and dw[0, 0].isnan() and torch.isfinite(dw[1, 0])


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("I", [64, 333])
def test_the_rows_made_again_are_the_forward_pass_s(I, dtype):
    """Bit for bit, from whole rows and from what 8 bits hold of them."""
    order, gu, dh, _, filled, _ = case(60, 12, 5, 3, 16, I, dtype)
    gu[~filled], dh[~filled] = 0, 0
    w = order.topk_weights
    h, again, *_ = passes(order, gu, dh, w)
    assert torch.equal(h, again)
    if I % 32 or dtype == FP16:      # (FP16 rounds the largest values that 8 bits hold)
        return
    _, again, _, _, kept = passes(order, gu, dh, w, keep=True)
    values = torch.zeros_like(gu)
    chord.chord_mxfp8_dequantize(*kept, values)
    assert torch.equal(passes(order, values, dh, w)[0], again)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_products_past_the_range_on_the_way(dtype):
    """w silu(gate) up is a number where silu(gate) up is past FP32: in both passes."""
    order = ExpertOrder(1, 1, 0, 1, 8).route(torch.zeros(1, 1, device="cuda"), torch.zeros(1, device="cuda"))
    gu = torch.full((order.capacity, 64), 2.0 ** 70, dtype=dtype, device="cuda")
    h, again, *_ = passes(order, gu, torch.ones_like(gu[:, :32]), torch.full((1, 1), 2.0 ** -60, device="cuda"))
    at = order.sorted_positions.long()
    assert (h[at] == 2.0 ** 80).all() and (again[at] == 2.0 ** 80).all()
