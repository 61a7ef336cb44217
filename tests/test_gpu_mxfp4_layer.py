"""GPU tests of the paths that run the operators together: MXFP4MoELayer step by
step against 64 bits, the differentiable row moves against autograd of their
formulas, and the example.

The layer's output depends on its quantised h: a last-bit difference of h can
move a 4-bit code by a whole step, so each step is checked from the tensors
that the step before it left, with the bounds of test_gpu_mxfp4.py and
test_gpu_expert_rows.py.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from w4a16_int4_weight_sigmoid_gb300 import chord
from w4a16_int4_weight_sigmoid_gb300 import workload as wl
from w4a16_int4_weight_sigmoid_gb300.layer import (ExpertOrder, MXFP4MoELayer, permute_rows, quantize_mxfp4, to_device,
                                                   unpermute_rows)

from gpu_util import ensure_lib
from test_gpu_mxfp4 import ref_quantize, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


SHAPES = [
    # tokens, H, I, experts, local, first local, topk
    (1, 256, 128, 8, 8, 0, 2),
    (16, 256, 128, 8, 8, 0, 2),
    (40, 512, 96, 16, 6, 5, 4),
    (300, 288, 192, 32, 32, 0, 6),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_layer_step_by_step(shape):
    M, H, I, E, local, begin, k = shape
    rng = np.random.default_rng(M + H)
    w13 = torch.from_numpy(rng.standard_normal((local, 2 * I, H)) / H ** 0.5).to(torch.bfloat16).cuda()
    w2 = torch.from_numpy(rng.standard_normal((local, H, I)) / I ** 0.5).to(torch.bfloat16).cuda()
    x = torch.from_numpy(rng.standard_normal((M, H))).to(torch.bfloat16).cuda()
    logits, bias = wl.router_inputs(M, E, M)
    layer = MXFP4MoELayer(quantize_mxfp4(w13), quantize_mxfp4(w2), E, begin, k)
    out = layer.forward(x, to_device(logits), to_device(bias))
    again = layer.forward(x, to_device(logits), to_device(bias))
    assert layer.dev_status.item() == 0 and torch.equal(out, again)

    w, ids, _ = oracle.route(logits, bias, k)
    assert np.array_equal(layer.order.topk_ids.cpu().numpy(), ids)
    pos = layer.order.sorted_positions.cpu().numpy().reshape(M, k)
    assert np.array_equal(pos >= 0, (ids >= begin) & (ids < begin + local))
    f64 = lambda t: t.double().cpu().numpy()
    q = lambda a: values(*ref_quantize(a))
    xq, q13 = q(f64(x)), q(f64(w13).reshape(-1, H)).reshape(w13.shape)
    q2 = q(f64(w2).reshape(-1, I)).reshape(w2.shape)
    h, y, got = f64(layer.h), f64(layer.y), f64(out)
    ref, terms = np.zeros((M, H)), np.zeros((M, H))
    for t in range(M):
        for j in range(k):
            if pos[t, j] < 0:
                continue
            r, e = pos[t, j], ids[t, j] - begin
            gu, d = q13[e] @ xq[t], H * 2.0 ** -23 * (np.abs(q13[e]) @ np.abs(xq[t]))
            g, u, dg, du = gu[:I], gu[I:], d[:I], d[I:]
            want = g / (1 + np.exp(-g)) * u
            bound = (2.0 ** -8 + 2.0 ** -18) * np.abs(want) + 1.1 * dg * np.abs(u) + np.abs(g) * du + 1.1 * dg * du
            assert (np.abs(h[r] - want) <= bound).all()
            hq = q(h[r][None])[0]
            want = q2[e] @ hq
            assert (np.abs(y[r] - want) <= 2.0 ** -8 * np.abs(want) + I * 2.0 ** -23 * (np.abs(q2[e]) @ np.abs(hq))).all()
            ref[t] += np.float64(w[t, j]) * y[r]
            terms[t] += np.abs(np.float64(w[t, j]) * y[r])
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -24 * terms * (1 + 2.0 ** -8)).all()


def test_layer_on_another_stream():
    """All steps follow the stream they are given."""
    M, H, I, E, k = 33, 256, 128, 8, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    w13, w2 = (torch.randn(s, generator=g, device="cuda") for s in ((E, 2 * I, H), (E, H, I)))
    x, logits, bias = torch.randn((M, H), generator=g, device="cuda"), torch.randn((M, E), generator=g, device="cuda"), torch.zeros(E, device="cuda")
    layer = MXFP4MoELayer(quantize_mxfp4(w13), quantize_mxfp4(w2), E, 0, k)
    want = layer.forward(x, logits, bias)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    layer.forward(x, logits, bias, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    assert layer.forward(x[:0], logits[:0], bias).shape == (0, H)


@pytest.mark.parametrize("local", [8, 3])
def test_autograd_is_exact_on_small_integers(local):
    """Integer rows and expert matrices and weights in quarters: every product and sum of
    forward and backward is exact in FP32, so the library's gradients equal autograd's of
    the formulas, for every expert or some of them, also where a token's row is used twice."""
    M, H, E, k = 37, 24, 8, 3
    rng = np.random.default_rng(local)
    ints = lambda *s: torch.from_numpy(rng.integers(-4, 5, s).astype(np.float32)).cuda()
    logits, bias = wl.router_inputs(M, E, 11)
    order = ExpertOrder(M, k, 1 if local < E else 0, local, block_m=8).route(to_device(logits), to_device(bias))
    x, dout, w = ints(M, H).requires_grad_(), ints(M, H), ints(local, H, H).requires_grad_()
    weights = (ints(M, k) / 4).requires_grad_()
    starts = order.expert_offsets.tolist()
    pos = order.sorted_positions.reshape(M, k).long()
    begin = order.expert_begin

    rows = permute_rows(x, order)
    y = torch.cat([rows[starts[e]:starts[e + 1]] @ w[e] for e in range(local)] +
                  [rows.new_zeros(order.capacity - starts[-1], H)])
    out = unpermute_rows(y, weights, order)
    out.backward(dout)
    got = [out.detach(), x.grad, w.grad, weights.grad]

    x2, w2, weights2 = (t.detach().double().requires_grad_() for t in (x, w, weights))
    e = order.topk_ids.long() - begin
    here = ((e >= 0) & (e < local)) & (pos >= 0)
    per = torch.einsum("mh,mkhn->mkn", x2, w2[e.clamp(0, local - 1)])
    ref = (per * (weights2 * here).unsqueeze(-1)).sum(1)
    ref.backward(dout.double())
    for a, b in zip(got, [ref.detach(), x2.grad, w2.grad, weights2.grad]):
        assert torch.equal(a.double(), b)


def test_gradients_of_sums_and_means():
    """A sum's gradient has stride 0 in both directions, a token mean's in one."""
    M, H, E, k = 20, 40, 8, 2
    logits, bias = wl.router_inputs(M, E, 12)
    order = ExpertOrder(M, k, 0, E).route(to_device(logits), to_device(bias))
    x = torch.ones((M, H), device="cuda", requires_grad=True)
    w = torch.full((M, k), 0.5, device="cuda", requires_grad=True)
    unpermute_rows(permute_rows(x, order), w, order).sum().backward()
    assert (x.grad == 1.0).all() and (w.grad == H).all()
    x.grad = w.grad = None
    row = torch.arange(H, device="cuda", dtype=torch.float32)
    (unpermute_rows(permute_rows(x, order), w, order).sum(0) * row).sum().backward()
    assert torch.equal(x.grad, row.expand(M, H)) and (w.grad == H * (H - 1) / 2).all()


def test_example_trains_and_serves():
    """The example's loss falls, and the MXFP4 layer stays within the format's error of the
    FP32 one: each quantised operand is within 2^-2 of its values in the worst case (a
    value between 4 and 6 in units of its scale) and about a tenth in the mean, through two
    products of both operands."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_moe.py")
    spec = importlib.util.spec_from_file_location("mxfp4_moe_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, off = m.train_and_serve(M=96, steps=12)
    assert losses[-1] < 0.8 * losses[0]
    assert off < 0.4
