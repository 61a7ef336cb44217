"""GPU tests of the rows in expert order (permute, unpermute and their
gradients) against their formulas in 64 bits, and of the gradients against
differences.

Bounds.  u is the unit roundoff of one result, half the spacing above 1: 2^-8
(BF16, 8 significant bits), 2^-11 (FP16, 11 bits), 2^-24 (FP32, 24 bits), and
half of FP16's smallest subnormal, 2^-25.  A sum of n FP32
terms in any order is within n * 2^-24 * sum |terms| of the exact one (each of
at most n roundings, products included, is relative to a partial sum no larger
than that).  Copies are exact.
"""
import numpy as np
import pytest
import torch

import oracle
from w4a16_int4_weight_sigmoid_gb300 import chord

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp16": (torch.float16, 2.0 ** -11),
         "fp32": (torch.float32, 2.0 ** -24)}
TINY = 2.0 ** -25


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


class Order:
    """A routing of M tokens to topk of E experts, `local` of them here from `begin`
    on, aligned to block_m by the library; host copies of the maps."""

    def __init__(self, M, E, begin, local, k, bm, seed):
        rng = np.random.default_rng(seed)
        ids = np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32).reshape(M, k)
        self.M, self.k = M, k
        self.w = torch.from_numpy(rng.random((M, k), dtype=np.float32) - 0.25).cuda()
        self.cap = max(chord.chord_moe_align_capacity(M, k, local, bm), bm)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.sorted = torch.full((self.cap,), M * k, **i32)
        self.pos = torch.full((M * k,), -1, **i32)
        self.ntpp = torch.zeros(1, **i32)
        counts, offsets = torch.empty(local, **i32), torch.empty(local + 1, **i32)
        nbytes = chord.chord_moe_align_workspace_bytes(M, k, local)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
        chord.chord_moe_align(torch.from_numpy(ids).cuda(), begin, local, bm, self.sorted,
                              torch.empty(self.cap // bm, **i32), self.ntpp, counts, offsets, self.pos, ws)
        torch.cuda.synchronize()
        self.n = int(self.ntpp)
        self.p = self.pos.cpu().numpy().reshape(M, k)
        s = self.sorted.cpu().numpy()[:self.n]
        self.pad = np.nonzero(s >= M * k)[0]
        self.fill = np.nonzero(s < M * k)[0]
        self.f = s[self.fill]


def rows(n, H, dtype, seed, stride=None, offset=0):
    """[n, H] N(0, 1) rows of `dtype`, optionally inside a wider, shifted buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = stride or H
    buf = torch.randn((n * ld + offset + 16,), generator=g, device="cuda").to(dtype)
    return buf[offset:offset + n * ld].view(n, ld)[:, :H]


def f64(t):
    return t.double().cpu().numpy()


def close(got, ref, terms, n, u, what):
    err = np.abs(f64(got) - ref)
    bound = u * np.abs(ref) + n * 2.0 ** -24 * terms * (1 + u) + TINY
    bad = err > bound
    assert not bad.any(), f"{what}: {bad.sum()} values beyond the bound, worst {np.max(err / bound):.2f} of it"


# tokens, experts, first local, local, topk, block
ORDERS = [
    (1, 8, 0, 8, 2, 16),        # one token
    (1, 384, 0, 48, 8, 8),      # one token, most assignments elsewhere
    (3, 8, 4, 2, 1, 128),       # top-1, tokens without a local expert
    (33, 64, 16, 16, 6, 32),
    (130, 8, 0, 8, 8, 8),       # every expert of every token
    (40, 32, 0, 32, 32, 16),    # topk at its limit
    (700, 384, 96, 48, 8, 64),  # several chunks of the align
]
# row length, row stride (None: dense), offset of the first element
SHAPES = [(1, None, 0), (7, None, 0), (64, None, 0), (250, 256, 0), (1000, None, 3), (2051, None, 0), (4100, 4104, 0)]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("name", list(TYPES))
def test_rows_and_gradients(order, shape, name):
    dtype, u = TYPES[name]
    o, (H, ld, off) = Order(*order, seed=sum(order)), shape
    x = rows(o.M, H, dtype, 1, ld, off)
    # permute: copies, zeros in the padding, nothing past the padded total
    out = torch.full((o.cap, H), 7.0, dtype=dtype, device="cuda")
    chord.chord_moe_permute(x, o.pos, o.sorted, o.ntpp, o.k, out)
    xs, got = f64(x), f64(out)
    assert np.array_equal(got[o.fill], xs[o.f // o.k])
    assert not got[o.pad].any() and (got[o.n:] == 7.0).all()

    # what padding rows hold (NaN) must reach nothing
    y = rows(o.cap, H, dtype, 2, ld, off)
    y[torch.from_numpy(o.pad).cuda()] = float("nan")
    y[o.n:] = float("nan")
    ys = f64(y)
    local = o.p >= 0
    gathered = np.where(local[..., None], ys[np.maximum(o.p, 0)], 0.0)      # [M, k, H]
    w = f64(o.w)[..., None]

    dx = torch.full((o.M, H), 7.0, dtype=dtype, device="cuda")
    chord.chord_moe_permute_backward(y, o.pos, o.k, dx)
    close(dx, gathered.sum(1), np.abs(gathered).sum(1), o.k, u, "permute_backward")

    out = torch.full((o.M, H), 7.0, dtype=dtype, device="cuda")
    chord.chord_moe_unpermute(y, o.w, o.pos, out)
    close(out, (w * gathered).sum(1), np.abs(w * gathered).sum(1), o.k, u, "unpermute")

    dy = torch.full((o.cap, H), 7.0, dtype=dtype, device="cuda")
    dw = torch.full((o.M, o.k), 7.0, device="cuda")
    chord.chord_moe_unpermute_backward(x, y, o.w, o.pos, o.sorted, o.ntpp, dy, dw)
    ref = xs[o.f // o.k] * f64(o.w).reshape(-1)[o.f][:, None]
    got = f64(dy)
    err = np.abs(got[o.fill] - ref)
    assert (err <= (u + 2.0 ** -24) * np.abs(ref) + TINY).all()
    assert not got[o.pad].any() and (got[o.n:] == 7.0).all()
    t = xs[:, None] * gathered
    close(dw, t.sum(-1), np.abs(t).sum(-1), H, 2.0 ** -24, "dweights")
    assert not f64(dw)[~local].any()


@pytest.mark.parametrize("name", list(TYPES))
def test_unaligned_outputs_and_broadcast_inputs(name):
    """Outputs inside wider buffers keep what lies around them; one row broadcast to
    all tokens (stride 0) is read as such, and its gradients follow."""
    dtype, u = TYPES[name]
    o, H = Order(37, 16, 0, 16, 3, 16, seed=5), 519
    one = rows(1, H, dtype, 3)
    buf = torch.full((o.cap, 531), 7.0, dtype=dtype, device="cuda")
    out = buf[:, 5:5 + H]
    chord.chord_moe_permute(one.expand(o.M, H), o.pos, o.sorted, o.ntpp, o.k, out)
    assert np.array_equal(f64(out)[o.fill], np.broadcast_to(f64(one), (len(o.fill), H)))
    assert (f64(buf)[:, :5] == 7.0).all() and (f64(buf)[:, 5 + H:] == 7.0).all()
    # the gradient of a mean over tokens: dout is one row for all
    y = rows(o.cap, H, dtype, 4)
    dy = torch.empty((o.cap, H), dtype=dtype, device="cuda")
    dw = torch.empty((o.M, o.k), device="cuda")
    chord.chord_moe_unpermute_backward(one.expand(o.M, H), y, o.w, o.pos, o.sorted, o.ntpp, dy, dw)
    t = f64(one)[0] * f64(y)[o.p]
    close(dw, t.sum(-1), np.abs(t).sum(-1), H, 2.0 ** -24, "dweights")
    # every expert row the same (stride 0)
    out = torch.empty((o.M, H), dtype=dtype, device="cuda")
    chord.chord_moe_unpermute(one.expand(o.cap, H), o.w, o.pos, out)
    t = f64(o.w)[..., None] * f64(one)[0]
    close(out, t.sum(1), np.abs(t).sum(1), o.k, u, "unpermute")


@pytest.mark.parametrize("H", [1, 9, 1024, 1030, 4113])
@pytest.mark.parametrize("name", ["bf16", "fp32"])
def test_permute_at_every_alignment(name, H):
    """Rows that begin at each element of 16 bytes, source and destination apart, land
    whole; the elements between them stay."""
    dtype, _ = TYPES[name]
    o = Order(19, 8, 0, 6, 2, 16, seed=H)
    for off in range(16 // dtype.itemsize):
        x = rows(o.M, H, dtype, off, H + 13, off)
        buf = torch.full((o.cap, H + 11), 7.0, dtype=dtype, device="cuda")
        out = buf.view(-1)[off // 2:off // 2 + (o.cap - 1) * (H + 11) + H].as_strided((o.cap, H), (H + 11, 1))
        chord.chord_moe_permute(x, o.pos, o.sorted, o.ntpp, o.k, out)
        ref = torch.full_like(buf, 7.0)
        view = ref.view(-1)[off // 2:].as_strided((o.cap, H), (H + 11, 1))
        view[torch.from_numpy(o.pad).cuda()] = 0.0
        view[torch.from_numpy(o.fill).cuda()] = x[torch.from_numpy(o.f // o.k).long().cuda()]
        assert torch.equal(buf, ref)


def test_gradients_against_differences():
    """L = <g, unpermute(y, w)> and <g, permute(x)>: central differences along random
    directions.  Both maps are linear in the direction, so the difference is exact up
    to the FP32 rounding of the two values: each of M*H terms of L carries an error
    below (k + 1) * 2^-24 of its magnitude, divided by the step of 2."""
    o, H = Order(50, 16, 4, 8, 4, 16, seed=6), 96
    y, v = rows(o.cap, H, torch.float32, 1), rows(o.cap, H, torch.float32, 2)
    g = rows(o.M, H, torch.float32, 3)
    dw_dir = torch.rand((o.M, o.k), device="cuda") - 0.5
    out = torch.empty((o.M, H), device="cuda")

    def loss(yy, ww):
        chord.chord_moe_unpermute(yy, ww, o.pos, out)
        return float((g.double() * out.double()).sum()), float((g.double() * out.double()).abs().sum())

    dy, dw = torch.zeros((o.cap, H), device="cuda"), torch.empty((o.M, o.k), device="cuda")
    chord.chord_moe_unpermute_backward(g, y, o.w, o.pos, o.sorted, o.ntpp, dy, dw)
    for yy, ww, grad in (((y + v, y - v), (o.w, o.w), (dy.double() * v.double()).sum()),
                         ((y, y), (o.w + dw_dir, o.w - dw_dir), (dw.double() * dw_dir.double()).sum())):
        (a, ta), (b, tb) = loss(yy[0].contiguous(), ww[0]), loss(yy[1].contiguous(), ww[1])
        # terms before cancellation inside a token's sum: k rows of |w y g|
        size = float((g.double().abs().sum() * 4 * o.k * 5))
        assert abs((a - b) / 2 - float(grad)) <= (o.k + 2) * 2.0 ** -24 * max(size, ta + tb)

    x, vx = rows(o.M, H, torch.float32, 4), rows(o.M, H, torch.float32, 5)
    gy = rows(o.cap, H, torch.float32, 6)
    up = torch.zeros((o.cap, H), device="cuda")

    def loss_x(xx):
        chord.chord_moe_permute(xx, o.pos, o.sorted, o.ntpp, o.k, up)
        return float((gy.double() * up.double()).sum())

    dx = torch.empty((o.M, H), device="cuda")
    chord.chord_moe_permute_backward(gy, o.pos, o.k, dx)
    diff = (loss_x((x + vx).contiguous()) - loss_x((x - vx).contiguous())) / 2
    size = float(gy.double().abs().sum() * 10)
    assert abs(diff - float((dx.double() * vx.double()).sum())) <= (o.k + 2) * 2.0 ** -24 * size


def test_weighted_sum_agrees_with_moe_sum():
    """BF16 rows: the same sums in the same order as chord_moe_sum, bit for bit."""
    o, H = Order(65, 384, 0, 384, 8, 16, seed=7), 1024
    y = rows(o.cap, H, torch.bfloat16, 1).contiguous()
    a, b = (torch.empty((o.M, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    chord.chord_moe_sum(y, o.w, o.pos, a)
    chord.chord_moe_unpermute(y, o.w, o.pos, b)
    assert torch.equal(a, b)


def test_another_stream_and_repeats():
    """Calls follow their own stream's order, and repeat bit for bit."""
    o, H = Order(300, 64, 0, 32, 6, 32, seed=8), 1536
    x = rows(o.M, H, torch.bfloat16, 1)
    y = torch.zeros((o.cap, H), dtype=torch.bfloat16, device="cuda")
    out, first = torch.empty_like(x), None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        chord.chord_moe_permute(x, o.pos, o.sorted, o.ntpp, o.k, y, stream=s)
        chord.chord_moe_unpermute(y, o.w, o.pos, out, stream=s)
        s.synchronize()
        first = out.clone() if first is None else first
        assert torch.equal(first, out)
    xs, w = f64(x), f64(o.w)
    ws = np.where(o.p >= 0, w, 0.0)
    close(out, xs * ws.sum(1)[:, None], np.abs(xs) * np.abs(ws).sum(1)[:, None], o.k, 2.0 ** -8, "round trip")


def test_offsets_beyond_32_bits():
    """Rows whose element offsets pass 2^31 and byte offsets pass 2^32."""
    M, H = 70000, 32768
    assert M * H > 2 ** 31
    x = torch.zeros((M, H), dtype=torch.bfloat16, device="cuda")
    x[-3:] = rows(3, H, torch.bfloat16, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    pos = torch.arange(M - 1, -1, -1, **i32)                 # reversed, then turned back
    pos[0], pos[M - 1] = M - 1, 0
    f, ntpp, w = torch.empty(M, **i32), torch.tensor([M], **i32), torch.ones((M, 1), device="cuda")
    f[pos.long()] = torch.arange(M, **i32)
    y, back = torch.empty_like(x), torch.empty_like(x)
    chord.chord_moe_permute(x, pos, f, ntpp, 1, y)
    assert torch.equal(y[pos[-3:].long()], x[-3:]) and not y[3:M - 3].any()
    chord.chord_moe_unpermute(y, w, pos, back)
    assert torch.equal(back, x)
    dw = torch.empty((M, 1), device="cuda")
    chord.chord_moe_unpermute_backward(x, y, w, pos, f, ntpp, back, dw)
    assert torch.equal(back, y)
    t = f64(x[-3:]) ** 2
    close(dw[-3:, 0], t.sum(1), t.sum(1), H, 2.0 ** -24, "dweights")


def test_in_a_cuda_graph():
    o, H = Order(16, 8, 0, 8, 2, 16, seed=9), 256
    x = rows(o.M, H, torch.bfloat16, 1).contiguous()
    y, out = torch.zeros((o.cap, H), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)

    def step():
        chord.chord_moe_permute(x, o.pos, o.sorted, o.ntpp, o.k, y)
        chord.chord_moe_unpermute(y, o.w, o.pos, out)

    step()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_tokens_and_refusals():
    o, H = Order(8, 8, 0, 8, 2, 16, seed=10), 64
    x, y = rows(o.M, H, torch.bfloat16, 1), rows(o.cap, H, torch.bfloat16, 2)
    out, big = torch.full_like(x, 7.0), torch.full_like(y, 7.0)
    dw = torch.zeros((o.M, o.k), device="cuda")
    # no tokens: nothing happens
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    chord.chord_moe_permute(x[:0], none, o.sorted, o.ntpp, o.k, big)
    chord.chord_moe_unpermute(y, o.w[:0], none, out[:0])
    chord.chord_moe_permute_backward(y, none, o.k, out[:0])
    with pytest.raises(TypeError):
        chord.chord_moe_permute(x.float(), o.pos, o.sorted, o.ntpp, o.k, big)           # two types
    with pytest.raises(TypeError):
        chord.chord_moe_permute(x.double(), o.pos, o.sorted, o.ntpp, o.k, big)          # FP64
    with pytest.raises(ValueError):
        chord.chord_moe_permute(x.T, o.pos, o.sorted, o.ntpp, o.k, big)                 # column-major
    with pytest.raises(ValueError):
        chord.chord_moe_permute(x, o.pos[:-1], o.sorted, o.ntpp, o.k, big)              # short positions
    with pytest.raises(ValueError):
        chord.chord_moe_permute(x, o.pos, o.sorted, o.ntpp, o.k, big[:, :32])           # row lengths differ
    with pytest.raises(ValueError):
        chord.chord_moe_unpermute(y.cpu(), o.w, o.pos, out)                             # host memory
    with pytest.raises(ValueError):
        chord.chord_moe_unpermute(y, o.w, o.pos, out[:-1])                              # too few tokens
    with pytest.raises(ValueError):
        chord.chord_moe_unpermute_backward(x, y, o.w, o.pos, o.sorted, o.ntpp, big, dw[:-1])
    with pytest.raises(chord.ChordError) as e:                                          # rows overlap
        chord.chord_moe_permute(x, o.pos, o.sorted, o.ntpp, o.k, big[:1].expand(o.cap, H))
    assert e.value.code == chord.CHORD_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (big == 7.0).all()
