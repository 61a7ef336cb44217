"""Host-side behaviour of the layer classes and the expert order that needs no GPU: calls
that are refused before anything is launched."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import build as B
from w4a16_int4_weight_sigmoid_gb300 import chord
from w4a16_int4_weight_sigmoid_gb300.layer import ExpertOrder


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()


@pytest.mark.parametrize("M,rows,topk", [(61, 65, 2), (9, 24, 1), (8, 7, 2), (8, 0, 2)])
def test_an_order_is_routed_for_its_own_tokens(M, rows, topk):
    """An order for 61 tokens has room for 65 in its padded rows, not in the arrays of its tokens."""
    order = ExpertOrder(M, topk, 0, 8, device="cpu")
    with pytest.raises(ValueError, match="logits must be"):
        order.route(torch.zeros((rows, 8)), torch.zeros(8))
    with pytest.raises(ValueError, match="logits must be"):
        order.route(torch.zeros(M * 8), torch.zeros(8))


def test_route_align_checks_what_its_arrays_hold():
    M, k, E, bm = 12, 2, 8, 16
    cap = chord.chord_moe_align_capacity(M, k, E, bm)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    full = dict(bias=torch.zeros(E), topk_weights=torch.zeros((M, k)), topk_ids=i32(M * k), sorted_token_ids=i32(cap),
                expert_ids=i32(cap // bm), num_tokens_post_padded=i32(1), expert_counts=i32(E),
                expert_offsets=i32(E + 1), sorted_positions=i32(M * k))

    def call(**kw):
        a = {**full, **kw}
        chord.chord_moe_route_align(torch.zeros((M, E)), a["bias"], k, 0, E, bm, a["topk_weights"], a["topk_ids"],
                                    a["sorted_token_ids"], a["expert_ids"], a["num_tokens_post_padded"],
                                    a["expert_counts"], a["expert_offsets"], a["sorted_positions"])

    for name, t in full.items():
        if name != "sorted_token_ids":               # its size is the capacity, which the library checks
            with pytest.raises(ValueError, match=f"{name} holds"):
                call(**{name: t.reshape(-1)[:-1]})
    with pytest.raises(ValueError, match="CUDA"):    # large enough, but host memory
        call()
