"""GPU tests of the layer classes as programs use them: other shapes than the layer's,
batches of changing size, captured graphs, other streams, repeated routing and second
derivatives."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300.layer import (ExpertOrder, MXFP4MoELayer, permute_rows, quantize_mxfp4,
                                                   unpermute_rows)

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

E, K, H, I = 8, 2, 256, 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def make_layer(seed=0):
    return MXFP4MoELayer(quantize_mxfp4(randn(E, 2 * I, H, seed=seed) / H ** 0.5),
                         quantize_mxfp4(randn(E, H, I, seed=seed + 1) / I ** 0.5), E, 0, K)


def inputs(M, seed=0):
    return randn(M, H, seed=10 + seed), randn(M, E, seed=20 + seed), torch.zeros(E, device="cuda")


def test_the_layer_refuses_other_shapes():
    """Rows of another length, and logits of other tokens or experts, are refused before anything runs."""
    layer = make_layer()
    x, logits, bias = inputs(12)
    out = torch.full((12, H), 7.0, dtype=torch.bfloat16, device="cuda")
    for a in ((x[:, :128], logits, bias), (x[:, :224].contiguous(), logits, bias), (x.reshape(-1), logits, bias),
              (x, logits[:11], bias), (x, logits[:0], bias), (x[:11], logits, bias), (x[:0], logits, bias),
              (x, logits[:, :7].contiguous(), bias), (x, logits, bias[:7]), (x, logits, torch.zeros(9, device="cuda"))):
        with pytest.raises(ValueError):
            layer.forward(*a, out=out)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    layer.forward(x, logits, bias, out=out)
    assert not (out == 7.0).all() and layer.dev_status.item() == 0
    assert layer.forward(x[:0], logits[:0], bias).shape == (0, H)


def test_unpermute_takes_the_rows_of_its_order():
    """Rows of another order would lose assignments without a word."""
    order = ExpertOrder(12, K, 0, E).route(randn(12, E), torch.zeros(E, device="cuda"))
    y, w = randn(order.capacity, H), order.topk_weights
    assert unpermute_rows(y, w, order).shape == (12, H)
    for bad in (y[:16], torch.cat([y, y[:8]])):
        with pytest.raises(ValueError, match="rows"):
            unpermute_rows(bad, w, order)


def test_the_layer_is_ready_when_made():
    """Its weights and counters are complete when the constructor returns, whatever the
    current stream has to do before, so that the first call may be on any stream."""
    args = [quantize_mxfp4(randn(E, 2 * I, H)), quantize_mxfp4(randn(E, H, I))]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                    # about 10 ms
    MXFP4MoELayer(*args, E, 0, K)
    assert torch.cuda.current_stream().query()


def test_buffers_are_memory_of_the_stream_they_are_used_on():
    """Batches of two sizes in turn on a side stream, kept busy, while the current stream
    allocates and overwrites what the allocator gives it: a call's buffers and output come
    from its own stream's memory, so nothing that is dropped is handed to the other."""
    layer = make_layer()
    batches = [inputs(M, seed=M) for M in (40, 9)]
    want = [layer.forward(*b) for b in batches]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for i in range(6):
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)             # about a millisecond ahead of each call
        got.append(layer.forward(*batches[i % 2], stream=s if i < 3 else s.cuda_stream))
        for _ in range(8):                            # the sizes of the layer's own buffers and output
            for t in (layer.h, layer.y, layer._rows, got[-1]):
                torch.empty_like(t).fill_(1)
    s.synchronize()
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % 2])
    assert layer.dev_status.item() == 0


def test_quantising_strided_weights_on_another_stream():
    """Rows that have to be copied together first are copied on the call's stream, and what
    the current stream allocates meanwhile is not theirs."""
    w = randn(E, H, 2 * I).transpose(1, 2)            # rows of H, not contiguous
    want = quantize_mxfp4(w.contiguous())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0):              # 0: the default stream's handle
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
        got = quantize_mxfp4(w, stream=stream)
        for _ in range(8):
            for t in (w, *got):
                torch.empty(t.shape, dtype=t.dtype, device="cuda").fill_(1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_graphs_keep_their_buffers():
    """One graph per batch size on one layer, calls of other sizes between, and tensors that
    take any memory set free: every replay gives what its own batch should, and touches
    nobody else's memory."""
    layer = make_layer()
    sizes = (64, 5, 130, 32)
    static, fresh, want = {}, {}, {}
    for M in sizes:
        static[M], fresh[M] = inputs(M, seed=M), inputs(M, seed=M + 1)
        want[M] = layer.forward(*fresh[M])
    graphs, outs, kept, watched = {}, {}, {}, []
    for M in sizes:
        graphs[M], outs[M] = torch.cuda.CUDAGraph(), torch.empty((M, H), dtype=torch.bfloat16, device="cuda")
        with torch.cuda.graph(graphs[M]):
            layer.forward(*static[M], out=outs[M])
        kept[M] = [t.data_ptr() for t in (layer.order.sorted_positions, layer._rows, layer.h, layer.y)]
        layer.forward(*static[32])
        watched += [torch.full_like(t, 1) for t in (layer._rows, layer.h, layer.y) for _ in range(4)]
    mine = {t.data_ptr() for t in watched} | {t.data_ptr() for t in (layer._rows, layer.h, layer.y)}
    for M in sizes:                                   # nothing that lives now is a captured buffer
        assert not mine & set(kept[M])
    for M in (32, 64, 5, 130, 64):
        for a, b in zip(static[M], fresh[M]):
            a.copy_(b)
        graphs[M].replay()
        assert torch.equal(outs[M], want[M])
        assert torch.equal(layer.forward(*fresh[5]), want[5])
    assert all((t == 1).all() for t in watched)
    assert layer.dev_status.item() == 0


def test_second_derivatives_are_refused():
    """Neither move's gradient is differentiable: a second derivative is an error, not a lost term."""
    order = ExpertOrder(12, K, 0, E).route(randn(12, E), torch.zeros(E, device="cuda"))
    x, w = randn(12, H).requires_grad_(), torch.rand((12, K), device="cuda").requires_grad_()
    rows = permute_rows(x, order)
    (dx,) = torch.autograd.grad(rows.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        dx.square().sum().backward()
    y = randn(order.capacity, H).requires_grad_()
    dy, dw = torch.autograd.grad(unpermute_rows(y, w, order).square().sum(), (y, w), create_graph=True)
    for g in (dy, dw):
        with pytest.raises(RuntimeError, match="differentiate twice"):
            g.sum().backward(retain_graph=True)


def test_routing_again_before_backward_is_noticed():
    """The gradients belong to the routing of their forward; a second route() into the same
    order makes backward an error.  Forwards of both routings keep their own when each has its order."""
    x = randn(12, H).requires_grad_()
    bias = torch.zeros(E, device="cuda")
    order = ExpertOrder(12, K, 0, E).route(randn(12, E, seed=1), bias)
    w = torch.rand((12, K), device="cuda").requires_grad_()
    rows = permute_rows(x, order)
    order.route(randn(12, E, seed=2), bias)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        rows.sum().backward()
    out = unpermute_rows(permute_rows(x, order).detach().requires_grad_(), w, order)
    order.route(randn(12, E, seed=3), bias)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    # weights taken from the order are overwritten as well
    scale = torch.ones(K, device="cuda", requires_grad=True)
    weights = order.topk_weights * scale
    order.route(randn(12, E, seed=4), bias)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        weights.sum().backward()
    # once more, in order
    unpermute_rows(permute_rows(x, order), w, order).sum().backward()
    here = order.sorted_positions.reshape(12, K) >= 0
    assert torch.allclose(x.grad, (w.detach() * here).sum(1, keepdim=True).expand(12, H))


def test_an_order_made_in_inference_mode():
    """Its tensors carry no versions and cannot be saved; routing it, moving rows and their
    gradients work all the same."""
    with torch.inference_mode():
        order = ExpertOrder(12, K, 0, E).route(randn(12, E), torch.zeros(E, device="cuda"))
        layer = make_layer()
        a = layer.forward(*inputs(12))
    order.route(randn(12, E), torch.zeros(E, device="cuda"))
    b = layer.forward(*inputs(12))
    assert torch.equal(a, b)
    x, w = randn(12, H).requires_grad_(), torch.full((12, K), 0.5, device="cuda", requires_grad=True)
    unpermute_rows(permute_rows(x, order), w, order).sum().backward()
    assert (x.grad == 1).all()


def test_an_order_of_no_tokens():
    """A rank without tokens routes, moves and differentiates nothing."""
    order = ExpertOrder(0, K, 0, E).route(torch.empty((0, E), device="cuda"), torch.zeros(E, device="cuda"))
    assert order.num_tokens_post_padded.item() == 0
    assert not order.expert_counts.any() and not order.expert_offsets.any()
    x = torch.empty((0, H), device="cuda", requires_grad=True)
    w = torch.empty((0, K), device="cuda", requires_grad=True)
    out = unpermute_rows(permute_rows(x, order), w, order)
    out.sum().backward()
    assert out.shape == (0, H) and x.grad.shape == (0, H) and w.grad.shape == (0, K)


def test_an_order_dropped_while_its_stream_is_busy():
    """Its memory is handed out again only when the stream that routes it is done."""
    logits, bias = randn(1000, E), torch.zeros(E, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    order = ExpertOrder(1000, K, 0, E)
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)               # about 50 ms
    order.route(logits, bias, stream=s)
    at = {order.sorted_token_ids.data_ptr(), order.sorted_positions.data_ptr(), order.topk_ids.data_ptr()}
    sizes = [order.sorted_token_ids.numel(), order.sorted_positions.numel(), order.topk_ids.numel()]
    del order
    new = [torch.empty(n, dtype=torch.int32, device="cuda") for n in sizes for _ in range(4)]
    assert not s.query()                              # it was busy all the while
    assert not at & {t.data_ptr() for t in new}
    s.synchronize()
