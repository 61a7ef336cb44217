"""The experts' products as programs call them: strides, large offsets, bad orders, the timeout
path, streams and graphs."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord

from gpu_util import ensure_lib
from test_gpu_expert_gemm import BF16, FP16, FP32, LEFT, expected_product, integers, order, rows_of, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def inputs(counts, K, N, transpose, dtype=BF16, seed=0, gaps=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, o, rows = order(counts, gaps)
    x = integers(g, rows, N if transpose else K, dtype=dtype)
    return c, o, x, integers(g, len(counts), N, K, dtype=dtype)


@pytest.mark.parametrize("transpose", [False, True])
def test_strides(transpose):
    """Rows and weights apart from one another, and what lies between the rows of the output is left."""
    c, o, x, w = inputs([70, 3, 0, 130], 136, 264, transpose)
    want = expected_product(x, w, c, o, transpose)
    wide_x = torch.full((x.shape[0], x.shape[1] + 24), float("nan"), dtype=BF16, device="cuda")
    wide_w = torch.full((w.shape[0], w.shape[1] + 3, w.shape[2] + 16), float("nan"), dtype=BF16, device="cuda")
    wide_out = torch.full((x.shape[0], want.shape[1] + 40), LEFT, dtype=BF16, device="cuda")
    xs, ws, out = wide_x[:, 8:8 + x.shape[1]], wide_w[:, :w.shape[1], 8:8 + w.shape[2]], wide_out[:, 16:16 + want.shape[1]]
    xs.copy_(x), ws.copy_(w)
    chord.chord_expert_gemm(xs, ws, c, o, out, workspace(), transpose)
    assert torch.equal(out, want)
    out.fill_(LEFT)
    assert (wide_out == LEFT).all()


def test_strides_of_the_gradient():
    c, o, x, w = inputs([70, 3, 0, 130], 136, 264, False)
    d = integers(torch.Generator(device="cuda").manual_seed(9), x.shape[0], 264, dtype=BF16)
    want = torch.stack([d[o[e]:o[e] + c[e]].double().T @ x[o[e]:o[e] + c[e]].double() for e in range(4)]).to(FP32)
    wide_x = torch.full((x.shape[0], 136 + 8), float("nan"), dtype=BF16, device="cuda")
    wide_d = torch.full((x.shape[0], 264 + 16), float("nan"), dtype=BF16, device="cuda")
    wide_x[:, 8:], wide_d[:, 8:-8] = x, d
    dw = torch.full((4, 264, 136), LEFT, device="cuda")
    chord.chord_expert_wgrad(wide_d[:, 8:-8], wide_x[:, 8:], c, o, dw, workspace())
    assert torch.equal(dw, want)


def test_offsets_beyond_32_bits():
    """Rows of the input and of the output more than 2^32 bytes behind the first."""
    c, o, x, w = inputs([40, 30], 64, 72, False)
    far = 1 << 26                                        # 70 rows: 2^32.1 values apart
    out = torch.empty(69 * far + 72, dtype=BF16, device="cuda").as_strided((70, 72), (far, 1))
    out.fill_(LEFT)
    chord.chord_expert_gemm(x, w, c, o, out, workspace())
    want = expected_product(x, w, c, o, False)
    assert torch.equal(out, want)
    back = out[:, :64]
    back.copy_(x)
    near = torch.full((70, 72), LEFT, dtype=BF16, device="cuda")
    chord.chord_expert_gemm(back, w, c, o, near, workspace())
    assert torch.equal(near, want)


def test_one_weight_for_a_single_expert_and_single_rows():
    """Strides of dimensions with one entry mean nothing."""
    x = integers(torch.Generator(device="cuda").manual_seed(1), 9, 72, dtype=BF16)
    c, o, _ = order([1])
    row = x.as_strided((1, 64), (77, 1))
    w = x.as_strided((1, 8, 64), (5, 72, 1))
    out = torch.empty((1, 8), dtype=BF16, device="cuda")
    chord.chord_expert_gemm(row, w, c, o, out, workspace())
    assert torch.equal(out, (row.double() @ w[0].double().T).to(BF16))


@pytest.mark.parametrize("counts,offsets", [
    ([4, 5], [0, 3, 9]),               # rows that two experts share
    ([4, 5], [6, 0, 12]),              # descending
    ([4, -1], [0, 4, 8]),
    ([4, 9], [0, 4, 13]),              # past the capacity
    ([4, 5], [-4, 4, 9]),
    ([4, 2147483647], [0, 4, 12]),
])
def test_orders_that_are_none(counts, offsets):
    """Recorded on the device, and nothing is computed."""
    i32 = dict(dtype=torch.int32, device="cuda")
    c, o = torch.tensor(counts, **i32), torch.tensor(offsets, **i32)
    x, w = torch.ones((12, 64), dtype=BF16, device="cuda"), torch.ones((2, 72, 64), dtype=BF16, device="cuda")
    out, dw = torch.full((12, 72), LEFT, dtype=BF16, device="cuda"), torch.full((2, 72, 64), LEFT, device="cuda")
    d = torch.ones((12, 72), dtype=BF16, device="cuda")
    ws = workspace()
    for call in (lambda s: chord.chord_expert_gemm(x, w, c, o, out, ws, dev_status=s),
                 lambda s: chord.chord_expert_wgrad(d, x, c, o, dw, ws, dev_status=s)):
        status = torch.zeros(1, **i32)
        call(status)
        assert status.item() == chord.CHORD_ERR_INVALID_ARG
    assert (out == LEFT).all() and (dw == LEFT).all() and not ws[:chord.CHORD_EXPERT_GEMM_COUNTER_BYTES].any()


def test_the_timeout_is_recorded_and_the_next_call_is_right():
    c, o, x, w = inputs([3] * 8, 2048, 512, False)
    ws, status = workspace(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((24, 512), LEFT, dtype=BF16, device="cuda")
    dw = torch.full((8, 512, 2048), LEFT, device="cuda")
    d = integers(torch.Generator(device="cuda").manual_seed(2), 24, 512, dtype=BF16)
    chord.lib().chord_debug_force_timeout(1)
    try:
        for call in (lambda: chord.chord_expert_gemm(x, w, c, o, out, ws, dev_status=status),
                     lambda: chord.chord_expert_wgrad(d, x, c, o, dw, ws, dev_status=status)):
            status.zero_()
            call()
            assert status.item() == chord.CHORD_ERR_TIMEOUT
    finally:
        chord.lib().chord_debug_force_timeout(0)
    assert (out == LEFT).all() and (dw == LEFT).all()
    status.zero_()
    chord.chord_expert_gemm(x, w, c, o, out, ws, dev_status=status)
    chord.chord_expert_wgrad(d, x, c, o, dw, ws, dev_status=status)
    assert status.item() == 0
    assert torch.equal(out, expected_product(x, w, c, o, False))
    for e, at in rows_of(c, o):
        assert torch.equal(dw[e], (d[at].double().T @ x[at].double()).float())


def test_refused_calls():
    c, o, x, w = inputs([8, 8], 64, 72, False)
    out, ws = torch.empty((16, 72), dtype=BF16, device="cuda"), workspace()
    f = lambda x=x, w=w, c=c, o=o, out=out, ws=ws, t=False: chord.chord_expert_gemm(x, w, c, o, out, ws, t)
    f()
    for bad in (dict(x=x.half()), dict(w=w.float()), dict(out=out.float()), dict(c=c.long()), dict(ws=ws.view(torch.int8))):
        with pytest.raises(TypeError):
            f(**bad)
    for bad in (dict(x=x[:, :56]), dict(out=out[:, :64]), dict(out=out[:15]), dict(c=c[:1]), dict(o=o[:2]), dict(t=True),
                dict(w=w[0]), dict(w=w.transpose(1, 2)), dict(x=x.T.contiguous().T)):
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(x=torch.empty(16 * 64 + 1, dtype=BF16, device="cuda")[1:].view(16, 64)), dict(ws=ws[:2048]),
                dict(x=x.float(), w=w.float(), out=out.float())):
        with pytest.raises(chord.ChordError):
            f(**bad)
    dw = torch.empty((2, 72, 64), device="cuda")
    d = torch.empty((16, 72), dtype=BF16, device="cuda")
    for bad in ((d, x.half(), dw), ):
        with pytest.raises(TypeError):
            chord.chord_expert_wgrad(bad[0], bad[1], c, o, bad[2], ws)
    for bad in ((d[:8], x, dw), (d, x, dw[:, :64]), (d, x, dw.transpose(1, 2).contiguous().transpose(1, 2)), (d, x, dw[:1])):
        with pytest.raises(ValueError):
            chord.chord_expert_wgrad(bad[0], bad[1], c, o, bad[2], ws)
    with pytest.raises(chord.ChordError):
        chord.chord_expert_wgrad(d, x, c, o, dw.half(), ws)


@pytest.mark.parametrize("counts,K,N", [([1] * 8, 2048, 512), ([300, 0, 17], 200, 520)])
def test_captured_and_on_two_streams(counts, K, N):
    """Graphs with a workspace of their own, replayed at the same time on two streams: what the calls give alone, also
    after the counts have changed."""
    sets = []
    for seed in (0, 1):
        c, o, x, w = inputs(counts, K, N, False, seed=seed)
        out = torch.empty((x.shape[0], N), dtype=BF16, device="cuda")
        dw = torch.empty((len(counts), N, K), dtype=FP32, device="cuda")
        ws, stream = workspace(), torch.cuda.Stream()

        def call(s=None, c=c, o=o, x=x, w=w, out=out, dw=dw, ws=ws):
            chord.chord_expert_gemm(x, w, c, o, out, ws, stream=s)
            chord.chord_expert_wgrad(out, x, c, o, dw, ws, stream=s)

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(3):
                call()
        sets.append((c, o, x, w, out, dw, stream, graph, call))
    for turn in range(4):
        for c, o, *_ in sets:
            c[0] = max(1, counts[0] - turn)
        for c, o, x, w, out, dw, stream, graph, call in sets:
            out.fill_(LEFT)
        torch.cuda.synchronize()
        for *_, stream, graph, call in sets:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for c, o, x, w, out, dw, *_ in sets:
            want = expected_product(x, w, c, o, False)
            assert torch.equal(out, want)
            for e in range(len(counts)):
                at = slice(o[e].item(), o[e].item() + c[e].item())
                exact = want[at].double().T @ x[at].double()
                assert ((dw[e].double() - exact).abs() <= exact.abs() * 2.0 ** -24 + 300 * 2.0 ** -23
                        * (want[at].double().abs().T @ x[at].double().abs())).all()
    # a call on a stream that is not the current one
    c, o, x, w, out, dw, stream, graph, call = sets[0]
    out.fill_(LEFT)
    torch.cuda.synchronize()
    call(stream)
    stream.synchronize()
    assert torch.equal(out, expected_product(x, w, c, o, False))
