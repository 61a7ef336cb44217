"""The experts' training path as a program uses it: expert_product and expert_mlp
against autograd in 64 bits, on their own, in graphs, on other streams."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300.layer import ExpertOrder, expert_mlp, expert_product, permute_rows, unpermute_rows

from gpu_util import ensure_lib
from test_gpu_mxfp8 import oracle as in_8_bits

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def make(M, H, I, E, local, topk, block=16, dtype=BF16, seed=0):
    order = ExpertOrder(M, topk, 0, local, block).route(randn(M, E, seed=seed), torch.zeros(E, device="cuda"))
    x = randn(M, H, seed=seed + 1).to(dtype)
    w13 = (randn(local, 2 * I, H, seed=seed + 2) / H ** 0.5).to(dtype)
    w2 = (randn(local, H, I, seed=seed + 3) / I ** 0.5).to(dtype)
    dout = randn(M, H, seed=seed + 4).to(dtype)
    return order, x, w13, w2, dout


def reference(order, x, weights, w13, w2, dout, held=None):
    """Output and gradients in 64 bits by autograd.  held: (x, gate and up) as the backward pass has them, which
    stand in for the values themselves wherever a gradient uses them."""
    x, weights, w13, w2 = (t.detach().double().requires_grad_() for t in (x, weights, w13, w2))
    M, k = weights.shape
    pos = order.sorted_positions.long().reshape(M, k)
    ids = order.topk_ids.long()
    out = x.new_zeros(x.shape)
    for e in range(w13.shape[0]):
        t, j = torch.nonzero((ids == e + order.expert_begin) & (pos >= 0), as_tuple=True)
        rows = x[t]
        if held is not None:
            rows = rows + (held[0].double()[t] - rows).detach()
        gu = rows @ w13[e].T
        if held is not None:
            gu = gu + (held[1].double()[pos[t, j]] - gu).detach()
        gate, up = gu.chunk(2, 1)
        h = weights[t, j][:, None] * torch.nn.functional.silu(gate) * up
        out = out.index_add(0, t, h @ w2[e].T)
    out.backward(dout.double())
    return out.detach(), [t.grad for t in (x, weights, w13, w2)]


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def run(order, x, weights, w13, w2, dout, held):
    leaves = [t.detach().clone().requires_grad_() for t in (x, weights, w13, w2)]
    out = expert_mlp(*leaves, order, held)
    out.backward(dout)
    assert order.dev_status.item() == 0
    return out.detach(), [t.grad for t in leaves]


def kept_values(order, x, w13):
    """What 8 bits hold of x and of the rows of gate and up (FP64); the rows as the 16-bit product rounds them."""
    with torch.no_grad():
        gu = expert_product(permute_rows(x, order), w13, order)
    return in_8_bits(x)[2].cuda(), in_8_bits(gu)[2].cuda()


SIZES = [(64, 128, 96, 8, 8, 2), (33, 64, 32, 12, 5, 3), (1, 256, 64, 8, 8, 2), (500, 512, 256, 16, 16, 4)]


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("M,H,I,E,local,topk", SIZES)
def test_expert_mlp(M, H, I, E, local, topk, dtype, held):
    """Five 16-bit roundings lie on the longest way to a result (rows, gate and up, h, y, out; backward: dy, dh, h or
    dgu, the rows' gradient), each of at most eps/2 relative in the 2-norm: 5 eps/2; a slope or product carries its
    operand's error on by a factor that stays below 2."""
    order, x, w13, w2, dout = make(M, H, I, E, local, topk, dtype=dtype)
    w = order.topk_weights
    out, grads = run(order, x, w, w13, w2, dout, held)
    want, exact = reference(order, x, w, w13, w2, dout)
    tol = 10 * torch.finfo(dtype).eps / 2
    assert off(out, want) <= tol
    if held:
        exact = reference(order, x, w, w13, w2, dout, kept_values(order, x, w13))[1]
    for got, g in zip(grads, exact):
        assert off(got, g) <= tol


def test_the_output_does_not_depend_on_what_is_kept():
    order, x, w13, w2, dout = make(*SIZES[0])
    a, b = (run(order, x, order.topk_weights, w13, w2, dout, held)[0] for held in (False, True))
    assert torch.equal(a, b)


def test_8_bits_keep_less_memory():
    """x and gate and up in 8 bits: at most 33/64 of what whole ones take (1 + 1/32 bytes of 2)."""
    order, x, w13, w2, _ = make(2048, 512, 512, 8, 8, 2)
    sizes = {}
    for held in (False, True):
        leaf = w13.detach().requires_grad_()
        kept = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
            expert_mlp(x, order.topk_weights, leaf, w2, order, held)
        large = [t for t in kept if t.numel() * t.element_size() > 1e5
                 and t.data_ptr() not in (w13.data_ptr(), w2.data_ptr())]
        sizes[held] = sum(t.numel() * t.element_size() for t in large)
    assert 0 < sizes[True] <= sizes[False] * 33 / 64


def test_expert_product_in_its_place():
    """permute, product, silu, product, weighted sum from the single operators, and the gradients of all leaves."""
    order, x, w13, w2, dout = make(70, 128, 64, 12, 6, 3)
    leaves = [t.detach().clone().requires_grad_() for t in (x, order.topk_weights, w13, w2)]
    rows = permute_rows(leaves[0], order)
    gate, up = expert_product(rows, leaves[2], order).chunk(2, 1)
    y = expert_product(torch.nn.functional.silu(gate) * up, leaves[3], order)
    out = unpermute_rows(y, leaves[1], order)
    out.backward(dout)
    want, exact = reference(order, x, order.topk_weights, w13, w2, dout)
    tol = 16 * torch.finfo(BF16).eps / 2      # silu, its product and their gradients round once more each
    assert off(out, want) <= tol
    for leaf, g in zip(leaves, exact):
        assert off(leaf.grad, g) <= tol


def test_gradients_that_are_not_asked_for():
    order, x, w13, w2, dout = make(*SIZES[0])
    want = run(order, x, order.topk_weights, w13, w2, dout, True)[1]
    for i in range(4):
        leaves = [t.detach().clone().requires_grad_(j == i) for j, t in enumerate((x, order.topk_weights, w13, w2))]
        expert_mlp(*leaves, order).backward(dout)
        assert [t.grad is not None for t in leaves] == [j == i for j in range(4)]
        assert torch.equal(leaves[i].grad, want[i])


@pytest.mark.parametrize("held", [False, True])
def test_no_tokens_and_no_local_tokens(held):
    order = ExpertOrder(0, 2, 0, 4).route(torch.zeros(0, 8, device="cuda"), torch.zeros(8, device="cuda"))
    x, w = torch.zeros(0, 64, dtype=BF16, device="cuda"), order.topk_weights
    w13, w2 = randn(4, 64, 64).to(BF16), randn(4, 64, 32).to(BF16)
    out, grads = run(order, x, w, w13, w2, x, held)
    assert out.shape == (0, 64) and all((g == 0).all() for g in grads)
    # every token goes to experts 0 and 1, none of which is local
    logits = torch.tensor([[9.0, 8.0] + [0.0] * 6], device="cuda").repeat(5, 1)
    order = ExpertOrder(5, 2, 4, 4).route(logits, torch.zeros(8, device="cuda"))
    x = randn(5, 64).to(BF16)
    out, grads = run(order, x, order.topk_weights, w13, w2, x, held)
    assert (out == 0).all() and all((g == 0).all() for g in grads)


def test_gradient_of_a_sum_and_of_a_transposed_input():
    """A gradient that is one value for all, and inputs whose rows are not the memory's."""
    order, x, w13, w2, _ = make(40, 64, 32, 8, 8, 2)
    ones = torch.ones(40, 64, dtype=BF16, device="cuda")
    want = run(order, x, order.topk_weights, w13, w2, ones, False)[1]
    leaves = [x.T.contiguous().T.detach().requires_grad_(), order.topk_weights.clone().requires_grad_(),
              w13.clone().requires_grad_(), w2.clone().requires_grad_()]
    expert_mlp(*leaves, order, False).sum().backward()
    for leaf, g in zip(leaves, want):
        assert torch.equal(leaf.grad, g)
    rows = permute_rows(x, order).requires_grad_()
    w = w13.clone().requires_grad_()
    expert_product(rows, w, order).sum().backward()
    assert torch.isfinite(rows.grad).all() and torch.isfinite(w.grad).all()
    # rows at an odd element, further apart
    wide = torch.zeros((rows.shape[0], 67), dtype=BF16, device="cuda")
    wide[:, 1:65] = rows.detach()
    out = expert_product(wide[:, 1:65], w13, order)
    assert torch.equal(out, expert_product(rows.detach(), w13, order))


def test_routing_again_before_the_backward_pass_is_an_error():
    order, x, w13, w2, dout = make(*SIZES[0])
    leaf = w13.clone().requires_grad_()
    out = expert_mlp(x, order.topk_weights.clone(), leaf, w2, order)
    order.route(randn(64, 8, seed=9), torch.zeros(8, device="cuda"))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward(dout)


def test_a_second_derivative_is_an_error():
    order, x, w13, w2, dout = make(*SIZES[0])
    leaf = w13.clone().requires_grad_()
    g, = torch.autograd.grad(expert_mlp(x, order.topk_weights, leaf, w2, order), leaf, dout, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_shapes_are_refused():
    order, x, w13, w2, _ = make(64, 128, 96, 8, 8, 2)
    w = order.topk_weights
    for bad in ((x[:63], w, w13, w2), (x, w[:63], w13, w2), (x, w, w13[:7], w2), (x, w, w13, w2[:7]),
                (x, w, w13[:, :160], w2), (x, w, w13, w2[:, :64]), (x[:, :96], w, w13, w2),
                (x[:, :120].contiguous(), w, w13[:, :, :120].contiguous(), w2[:, :120].contiguous())):
        with pytest.raises(ValueError):
            expert_mlp(*bad, order)
    rows = permute_rows(x, order)
    for bad in ((rows[:-1], w13), (rows, w13[:7]), (rows[:, :64], w13)):
        with pytest.raises(ValueError):
            expert_product(*bad, order)
    with pytest.raises(TypeError):
        expert_product(rows, w13.half(), order)


def test_captured_training_steps_of_two_sizes():
    """Forward and backward captured for two batch sizes, replayed in turn between eager steps on new inputs."""
    steps = {}
    for M in (24, 130):
        order, x, w13, w2, dout = make(M, 128, 64, 8, 8, 2, seed=M)
        w = order.topk_weights.detach()
        logits, bias = randn(M, 8, seed=M), torch.zeros(8, device="cuda")
        leaves = [t.detach().clone().requires_grad_() for t in (x, w13, w2)]

        def step(order=order, leaves=leaves, w=w, dout=dout, logits=logits, bias=bias):
            order.route(logits, bias)
            out = expert_mlp(leaves[0], w, leaves[1], leaves[2], order)
            return (out, *torch.autograd.grad(out, leaves, dout))

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        steps[M] = (graph, got, step, leaves, logits)
    for seed in range(3):
        for M, (graph, got, step, leaves, logits) in steps.items():
            with torch.no_grad():
                leaves[0].copy_(randn(M, 128, seed=50 + seed))
                logits.copy_(randn(M, 8, seed=60 + seed))
            graph.replay()
            graph_values = [t.clone() for t in got]
            for a, b in zip(graph_values, step()):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    """Passes on two streams share nothing: each gives what it gives alone."""
    sets = [make(300, 256, 128, 8, 8, 2, seed=s) for s in (0, 5)]
    alone = [run(*s[:2], s[0].topk_weights, *s[2:], True) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    results = [None, None]
    for _ in range(5):
        for i, (s, stream) in enumerate(zip(sets, streams)):
            order, x, w13, w2, dout = s
            with torch.cuda.stream(stream):
                leaves = [t.detach().clone().requires_grad_() for t in (x, order.topk_weights, w13, w2)]
                out = expert_mlp(*leaves, order)
                results[i] = (out.detach(), torch.autograd.grad(out, leaves, dout))
    torch.cuda.synchronize()
    for (out, grads), (want, exact) in zip(results, alone):
        assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(grads, exact))


@pytest.mark.parametrize("held", [False, True])
def test_example(held):
    """The training example runs, and its router's and experts' gradients are those of its formula in 64 bits."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_training.py")
    spec = importlib.util.spec_from_file_location("moe_training", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer, losses = example.train(M=96, H=64, I=32, steps=3, held_in_8_bits=held)
    assert all(torch.isfinite(torch.tensor(losses)))
    assert all(torch.isfinite(p).all() for p in layer.parameters())
    if held:
        return
    x, target = randn(96, 64, seed=1).to(BF16), randn(96, 64, seed=2)
    layer.zero_grad()
    (layer(x).float() - target).square().mean().backward()
    router, w13, w2 = (p.detach().double() for p in (layer.router, layer.w13.to(BF16), layer.w2.to(BF16)))
    leaves = [t.requires_grad_() for t in (router, w13, w2)]
    xd = x.double()
    logits = xd @ router.T
    ids = torch.topk(torch.sigmoid((x.float() @ layer.router.T)), layer.topk, 1).indices
    score = torch.sigmoid(logits).gather(1, ids)
    weights = score / score.sum(1, keepdim=True)
    out = torch.zeros_like(xd)
    for e in range(w13.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gate, up = (xd[t] @ w13[e].T).chunk(2, 1)
        out = out.index_add(0, t, (weights[t, j][:, None] * torch.nn.functional.silu(gate) * up) @ w2[e].T)
    (out - target.double()).square().mean().backward()
    # the 16-bit roundings on the way (see test_expert_mlp), and that of the loss's gradient
    tol = 12 * torch.finfo(BF16).eps / 2
    for p, leaf in zip((layer.router, layer.w13, layer.w2), leaves):
        assert off(p.grad, leaf.grad) <= tol


def test_without_gradients():
    """The same output in inference mode and without gradients, also with an order made there."""
    order, x, w13, w2, _ = make(64, 128, 96, 8, 8, 2)
    w = order.topk_weights
    want = run(order, x, w, w13, w2, torch.zeros_like(x), True)[0]
    with torch.no_grad():
        assert torch.equal(expert_mlp(x, w, w13, w2, order), want)
    with torch.inference_mode():
        inner = ExpertOrder(64, 2, 0, 8, 16).route(randn(64, 8), torch.zeros(8, device="cuda"))
        assert torch.equal(expert_mlp(x, inner.topk_weights, w13, w2, inner), want)
    leaf = w13.clone().requires_grad_()
    out = expert_mlp(x, w, leaf, w2, inner)
    out.sum().backward()
    assert torch.equal(out.detach(), want) and torch.isfinite(leaf.grad).all()


FIRST_CALL_IN_A_CAPTURE = """
import torch
from w4a16_int4_weight_sigmoid_gb300.layer import ExpertOrder, expert_mlp
order = ExpertOrder(40, 2, 0, 4).route(torch.randn(40, 4, device="cuda"), torch.zeros(4, device="cuda"))
x = torch.randn(40, 64, device="cuda").bfloat16()
w13, w2 = torch.randn(4, 64, 64, device="cuda").bfloat16(), torch.randn(4, 64, 32, device="cuda").bfloat16()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = expert_mlp(x, order.topk_weights, w13, w2, order)
graph.replay()
assert torch.equal(out, expert_mlp(x, order.topk_weights, w13, w2, order))
print("FINE")
"""


def test_the_first_call_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "FINE" in r.stdout, r.stdout + r.stderr
