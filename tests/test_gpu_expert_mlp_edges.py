"""expert_mlp does only what its gradients need, and takes part in graphs, checkpoints and shared leaves."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord
from w4a16_int4_weight_sigmoid_gb300.layer import expert_mlp

from gpu_util import ensure_lib
from test_gpu_expert_mlp import SIZES, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.fixture
def calls(monkeypatch):
    """The arguments of each call of the operators, by name."""
    seen = {}
    for name in ("chord_mxfp8_quantize", "chord_swiglu", "chord_swiglu_backward", "chord_expert_wgrad"):
        def call(*args, _name=name, _f=getattr(chord, name)):
            seen.setdefault(_name, []).append(args)
            return _f(*args)
        monkeypatch.setattr(chord, name, call)
    return seen


def test_nothing_is_quantised_without_gradients(calls):
    order, x, w13, w2, dout = make(*SIZES[0])
    want = run(order, x, order.topk_weights, w13, w2, dout, True)[0]
    for grad in (False, True):
        calls.clear()
        leaf = w13.clone().requires_grad_(not grad)
        with torch.set_grad_enabled(grad):
            assert torch.equal(expert_mlp(x, order.topk_weights, leaf, w2, order), want)
        assert "chord_mxfp8_quantize" not in calls
        assert calls["chord_swiglu"][0][5:] in ((), (None, None))


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("asked", [(0,), (1,), (2,), (3,), (0, 1), (2, 3)])
def test_what_single_gradients_need(calls, asked, held):
    """x is kept for w13's gradient alone, the rows of h are made again for w2's alone; the gradients are those
    of a pass that asks for all."""
    order, x, w13, w2, dout = make(*SIZES[0])
    want = run(order, x, order.topk_weights, w13, w2, dout, held)[1]
    calls.clear()
    leaves = [t.detach().clone().requires_grad_(i in asked) for i, t in enumerate((x, order.topk_weights, w13, w2))]
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        out = expert_mlp(*leaves, order, held)
    assert ("chord_mxfp8_quantize" in calls) == (held and 2 in asked)
    assert any(t.data_ptr() == leaves[0].data_ptr() for t in kept) == (not held and 2 in asked)
    out.backward(dout)
    assert (calls["chord_swiglu_backward"][0][10] is not None) == (3 in asked)
    assert len(calls.get("chord_expert_wgrad", [])) == (2 in asked) + (3 in asked)
    for i, leaf in enumerate(leaves):
        assert (leaf.grad is not None) == (i in asked)
        if i in asked:
            assert torch.equal(leaf.grad, want[i])


def leaves_of(*tensors):
    return [t.detach().clone().requires_grad_() for t in tensors]


@pytest.mark.parametrize("held", [False, True])
def test_a_captured_backward_call(held):
    """loss.backward() captured after a warm-up on the capture's stream, replayed on new inputs: the gradients of the
    graph's leaves are those of an eager pass on leaves of its own."""
    order, x, w13, w2, dout = make(*SIZES[0])
    weights = order.topk_weights.detach().clone()
    leaves = leaves_of(x, weights, w13, w2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):
            for leaf in leaves:
                leaf.grad = None
            expert_mlp(*leaves, order, held).backward(dout)
    torch.cuda.current_stream().wait_stream(stream)
    for leaf in leaves:
        leaf.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        expert_mlp(*leaves, order, held).backward(dout)
    for seed in (5, 6):
        new = make(*SIZES[0], seed=seed)[1]
        with torch.no_grad():
            leaves[0].copy_(new)
        graph.replay()
        want = run(order, new, weights, w13, w2, dout, held)[1]
        for leaf, g in zip(leaves, want):
            assert torch.equal(leaf.grad, g)


@pytest.mark.parametrize("held", [False, True])
def test_a_checkpointed_pass_and_a_second_backward(held):
    """Recomputed under torch.utils.checkpoint, and taken twice from one graph: the same gradients."""
    from torch.utils.checkpoint import checkpoint
    order, x, w13, w2, dout = make(*SIZES[1])
    want = run(order, x, order.topk_weights, w13, w2, dout, held)[1]
    leaves = leaves_of(x, order.topk_weights, w13, w2)
    out = checkpoint(lambda *t: expert_mlp(*t, order, held), *leaves, use_reentrant=False)
    for a, b in zip(torch.autograd.grad(out, leaves, dout), want):
        assert torch.equal(a, b)
    out = expert_mlp(*leaves, order, held)
    for again in (True, False):
        for a, b in zip(torch.autograd.grad(out, leaves, dout, retain_graph=again), want):
            assert torch.equal(a, b)


def test_gradients_add_up_in_their_leaves():
    """Two passes of one set of leaves through two orders: the sum of what each gives."""
    first, second = make(*SIZES[0]), make(*SIZES[0], seed=9)
    _, x, w13, w2, dout = first
    weights = [o.topk_weights for o, *_ in (first, second)]
    alone = [run(o, x, w, w13, w2, dout, True)[1] for (o, *_), w in zip((first, second), weights)]
    shared = leaves_of(x, w13, w2)
    outs = [expert_mlp(shared[0], w, *shared[1:], o) for (o, *_), w in zip((first, second), weights)]
    (outs[0] + outs[1]).backward(dout)
    for i, leaf in zip((0, 2, 3), shared):
        assert torch.equal(leaf.grad, alone[1][i] + alone[0][i])
