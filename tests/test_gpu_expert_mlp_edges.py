"""expert_mlp does only what its gradients need: what is kept and made again by what is asked for."""
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
