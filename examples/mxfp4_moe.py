"""A small MoE layer trained in FP32 and then served with MXFP4 experts.

Training: tokens are routed, sorted by expert (permute_rows), run through one
SiLU-gated MLP per expert, and summed back with the routing weights
(unpermute_rows); the gradients of both moves come from the library.
Serving: the trained experts are quantised to MXFP4 (quantize_mxfp4) and the
same tokens go through MXFP4MoELayer, one call, 4 bits on both operands.

    python examples/mxfp4_moe.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from w4a16_int4_weight_sigmoid_gb300 import build  # noqa: E402
from w4a16_int4_weight_sigmoid_gb300.layer import (ExpertOrder, MXFP4MoELayer, permute_rows, quantize_mxfp4,  # noqa: E402
                                                   unpermute_rows)


def experts(rows, w13, w2, order):
    """One MLP per expert over its run of rows (plain torch products)."""
    starts = order.expert_offsets.tolist()
    parts = []
    for e in range(order.E_local):
        gate, up = (rows[starts[e]:starts[e + 1]] @ w13[e].T).chunk(2, 1)
        parts.append((torch.nn.functional.silu(gate) * up) @ w2[e].T)
    parts.append(rows.new_zeros(order.capacity - starts[-1], w2.shape[1]))
    return torch.cat(parts)


def train_and_serve(M=256, H=256, I=128, E=8, topk=2, steps=40, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, target = rand(M, H), rand(M, H)
    router = rand(E, H) / H ** 0.5
    bias = torch.zeros(E, device="cuda")
    w13 = (rand(E, 2 * I, H) / H ** 0.5).requires_grad_()
    w2 = (rand(E, H, I) / I ** 0.5).requires_grad_()
    scale = torch.ones(E, device="cuda", requires_grad=True)     # trained through the routing weights' gradient
    optimizer = torch.optim.Adam([w13, w2, scale], lr=3e-3)
    logits = (x @ router.T).contiguous()
    order = ExpertOrder(M, topk, 0, E).route(logits, bias)
    losses = []
    for _ in range(steps):
        rows = permute_rows(x, order)
        weights = order.topk_weights * scale[order.topk_ids.long()]
        out = unpermute_rows(experts(rows, w13, w2, order), weights, order)
        loss = (out - target).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    with torch.no_grad():
        w2s = w2 * scale[:, None, None]                          # the scale belongs to its expert
        layer = MXFP4MoELayer(quantize_mxfp4(w13.detach()), quantize_mxfp4(w2s.contiguous()), E, 0, topk)
        served = layer.forward(x, logits, bias)
        full = unpermute_rows(experts(permute_rows(x, order), w13, w2s, order), order.topk_weights, order)
    assert layer.dev_status.item() == 0
    off = (served.float() - full).norm() / full.norm()
    return losses, off.item()


if __name__ == "__main__":
    build.build()
    losses, off = train_and_serve()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; MXFP4 output differs from FP32's by {100 * off:.1f} %")
