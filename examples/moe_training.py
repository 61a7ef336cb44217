"""A small MoE layer whose experts train in BF16 on the GPU, activations kept in 8 bits.

Each step routes the tokens (ExpertOrder), runs the experts over them and sums
their rows back with the routing weights (expert_mlp); the backward pass gives
the gradients of the tokens, the routing weights and both expert matrices.  No
step waits for the host.  The optimizer works on FP32 copies of the weights.

    python examples/moe_training.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from w4a16_int4_weight_sigmoid_gb300 import build  # noqa: E402
from w4a16_int4_weight_sigmoid_gb300.layer import ExpertOrder, expert_mlp  # noqa: E402


class MoE(torch.nn.Module):
    """Sigmoid routing and SiLU-gated experts; the routing weights' gradient reaches the router."""

    def __init__(self, H, I, E, topk, held_in_8_bits=True):
        super().__init__()
        self.topk, self.held = topk, held_in_8_bits
        self.router = torch.nn.Parameter(torch.randn(E, H, device="cuda") / H ** 0.5)
        self.bias = torch.zeros(E, device="cuda")
        self.w13 = torch.nn.Parameter(torch.randn(E, 2 * I, H, device="cuda") / H ** 0.5)
        self.w2 = torch.nn.Parameter(torch.randn(E, H, I, device="cuda") / I ** 0.5)

    def forward(self, x):
        logits = (x.float() @ self.router.T).contiguous()
        order = ExpertOrder(x.shape[0], self.topk, 0, self.w13.shape[0]).route(logits.detach(), self.bias)
        # the weights that the routing chose, as a function of the router
        score = torch.sigmoid(logits).gather(1, order.topk_ids.long())
        weights = score / score.sum(1, keepdim=True)
        return expert_mlp(x, weights, self.w13.to(x.dtype), self.w2.to(x.dtype), order, self.held)


def train(M=512, H=256, I=128, E=8, topk=2, steps=30, held_in_8_bits=True, seed=0):
    torch.manual_seed(seed)
    layer = MoE(H, I, E, topk, held_in_8_bits)
    x = torch.randn(M, H, device="cuda").bfloat16()
    target = torch.randn(M, H, device="cuda")
    optimizer = torch.optim.Adam(layer.parameters(), lr=2e-3)
    losses = []
    for _ in range(steps):
        loss = (layer(x).float() - target).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
    return layer, [v.item() for v in losses]


if __name__ == "__main__":
    build.build()
    for held in (False, True):
        _, losses = train(held_in_8_bits=held)
        print(f"activations kept {'in 8 bits' if held else 'whole'}: loss {losses[0]:.3f} -> {losses[-1]:.3f}")
