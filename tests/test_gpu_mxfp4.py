"""GPU tests of MXFP4 quantisation and of the experts' product against their
definitions in 64 bits.

Quantisation and its inverse are exact operations (a power-of-two scale and a
rounding to eight magnitudes), so codes, scales and values are compared bit
for bit.  The product's operands are exact as well; its FP32 accumulation adds
at most one error of 2^-23 of the running magnitude for each of the K terms
(the tensor core may truncate), and one rounding to BF16 ends it (unit
roundoff 2^-8: 8 significant bits):
  |C - exact| <= 2^-8 |exact| + d,  d = K * 2^-23 * sum_k |a_k w_k|.
SiLU(g) * u with errors d_g, d_u: |silu'| <= 1.1 and |silu(g)| <= |g|, so
  |C - exact| <= 2^-8 |exact| + 1.1 d_g |u| + |g| d_u + 1.1 d_g d_u
                 + 2^-18 |exact|    (the fast exponential and division).
"""
import numpy as np
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def ref_quantize(x):
    """float64 x [rows, K] -> codes per value (uint8 0..15), scale codes [rows, K/32]."""
    b = x.reshape(x.shape[0], -1, 32)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(all="ignore"):
        e = np.frexp(np.where(bad, 1.0, top))[1] - 3           # floor(log2 top) - 2
        s = np.where(top == 0, 0, np.maximum(e + 127, 0))
        s = np.where(bad, 255, s)
        a = np.abs(b) / np.ldexp(1.0, np.where(bad, 0, s - 127))[..., None]
    a = np.where(bad[..., None], 0.0, a)
    code = np.zeros(a.shape, np.uint8)
    for i in range(7):
        mid = (LEVELS[i] + LEVELS[i + 1]) / 2
        code += (a > mid) | ((a == mid) & (i % 2 == 1))        # a tie goes to the even code
    code |= np.where(np.signbit(b) & ~bad[..., None], 8, 0).astype(np.uint8)
    return code.reshape(x.shape), s.astype(np.uint8)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def values(code, s):
    """float64 values of codes [..., K] and scale codes [..., K/32]."""
    v = np.where(code & 8, -1.0, 1.0) * LEVELS[code & 7]
    return v * np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), 32, -1)


def inputs(rows, K, dtype, seed):
    """Values over many magnitudes, with ties, zeros and signed zeros among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-9, 9, (rows, K // 32)).repeat(32, 1))
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.5, 4.0, 0.0], (rows, K)) * rng.choice([-1, 1], (rows, K))
    ties[:, ::32] = 4.0
    x = np.where(rng.random((rows, 1)) < 0.3, ties, x)
    x[rng.random((rows, K // 32)).repeat(32, 1) < 0.05] = 0.0
    return torch.from_numpy(x).to(dtype).cuda()


@pytest.mark.parametrize("shape", [(1, 32), (1, 7168), (3, 96), (65, 256), (300, 2048), (17, 1056)])
@pytest.mark.parametrize("name", list(TYPES))
def test_quantize_and_back_are_exact(shape, name):
    rows, K = shape
    x = inputs(rows, K, TYPES[name], sum(shape))
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, K // 32), dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_quantize(x, codes, scales)
    code, s = ref_quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), pack(code))
    for out_type in TYPES.values():
        out = torch.empty((rows, K), dtype=out_type, device="cuda")
        chord.chord_mxfp4_dequantize(codes, scales, out)
        want = torch.from_numpy(values(code, s)).to(out_type)
        assert torch.equal(out.cpu(), want)


def test_quantize_extremes():
    """The largest and smallest magnitudes, infinities and NaNs, every block its own case."""
    x = torch.zeros((12, 32), device="cuda")
    x[0] = torch.finfo(torch.float32).max
    x[1] = -torch.finfo(torch.float32).max
    x[2, 3] = 2.0 ** -126                      # smallest normal
    x[3, 3], x[3, 4] = 2.0 ** -149, -2.0 ** -149   # subnormals
    x[4, 5] = float("inf")
    x[5, 6] = float("nan")
    x[6, 7], x[6, 8] = float("-inf"), 1.0
    x[7] = -0.0
    x[8, 0], x[8, 1] = 2.0 ** 127, 2.0 ** -149
    x[9, 0] = 6 * 2.0 ** -127
    x[10, 0], x[10, 1:] = 1.0, 0.0625
    codes = torch.empty((12, 16), dtype=torch.uint8, device="cuda")
    scales = torch.empty((12, 1), dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_quantize(x, codes, scales)
    code, s = ref_quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), pack(code))
    out = torch.empty_like(x)
    chord.chord_mxfp4_dequantize(codes, scales, out)
    got = out.cpu().numpy()
    assert np.isnan(got[4:7]).all()
    keep = [0, 1, 2, 3, 7, 8, 9, 10, 11]
    assert np.array_equal(got[keep].astype(np.float64), values(code, s)[keep])


@pytest.mark.parametrize("name", ["bf16", "fp16"])
def test_quantize_extremes_of_16_bits(name):
    """Each power of two of the type as a block's maximum, subnormals included, with ties and
    the type's largest value: the scaled values stay exact in 16 bits."""
    dtype = TYPES[name]
    lo, hi = (-133, 127) if name == "bf16" else (-24, 15)
    n = hi - lo + 1
    x = torch.zeros((n + 1, 32), dtype=torch.float64)
    for i, e in enumerate(range(lo, hi + 1)):
        x[i] = torch.tensor([1, -1, 0.75, 0.625, -0.375, 0.4375, 0.0625, 0.1875, 0.3125, -0.21875, 0, -0.0,
                             0.25, 0.5, 0.125, 1e-3] * 2, dtype=torch.float64) * 2.0 ** e
    x[n] = torch.finfo(dtype).max
    x[n, 1::2] = -torch.finfo(dtype).max
    x = x.to(dtype).cuda()
    codes = torch.empty((n + 1, 16), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n + 1, 1), dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_quantize(x, codes, scales)
    code, s = ref_quantize(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), pack(code))
    for i, bad in enumerate((float("inf"), float("-inf"), float("nan"))):
        x[i, 5 * i] = bad
    chord.chord_mxfp4_quantize(x, codes, scales)
    assert (scales[:3] == 255).all() and (codes[:3] == 0).all() and (scales[3:] != 255).all()


def test_quantize_strides():
    """Rows inside a wider, unaligned buffer, and one row for all (stride 0)."""
    base = inputs(9, 512, torch.bfloat16, 3)
    wide = torch.zeros((9, 523), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:515] = base
    want = [torch.empty((9, 256), dtype=torch.uint8, device="cuda"), torch.empty((9, 16), dtype=torch.uint8, device="cuda")]
    got = [torch.empty_like(t) for t in want]
    chord.chord_mxfp4_quantize(base, *want)
    chord.chord_mxfp4_quantize(wide[:, 3:515], *got)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    chord.chord_mxfp4_quantize(base[:1].expand(9, 512), *got)
    assert torch.equal(got[0], want[0][:1].expand(9, 256)) and torch.equal(got[1], want[1][:1].expand(9, 16))
    out = torch.full((9, 523), 7.0, dtype=torch.bfloat16, device="cuda")
    chord.chord_mxfp4_dequantize(*want, out[:, 3:515])
    dense = torch.empty((9, 512), dtype=torch.bfloat16, device="cuda")
    chord.chord_mxfp4_dequantize(*want, dense)
    assert torch.equal(out[:, 3:515], dense) and (out[:, :3] == 7.0).all() and (out[:, 515:] == 7.0).all()


# ---------------------------------------------------------------- the product
class Experts:
    """counts[e] rows of expert e in blocks of bm; tokens in a random order, one assignment each."""

    def __init__(self, counts, bm, N, K, seed, dtype=torch.bfloat16):
        rng = np.random.default_rng(seed)
        E = len(counts)
        self.counts, self.E, self.N, self.K = np.array(counts), E, N, K
        padded = -(-self.counts // bm) * bm
        self.offsets = np.concatenate([[0], np.cumsum(padded)])
        self.cap = int(max(self.offsets[-1], bm))
        at = np.concatenate([self.offsets[e] + np.arange(c) for e, c in enumerate(counts)]).astype(np.int64)
        self.M = len(at)
        self.pos = rng.permutation(at)                            # row of token t
        self.expert = np.searchsorted(self.offsets[1:], self.pos, side="right")
        self.x = torch.from_numpy(rng.standard_normal((self.M, K)).astype(np.float32)).to(dtype).cuda()
        self.code = rng.integers(0, 16, (E, N, K)).astype(np.uint8)
        self.scale = rng.integers(118, 128, (E, N, K // 32)).astype(np.uint8)
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        self.d_counts, self.d_offsets, self.d_pos = i32(self.counts), i32(self.offsets), i32(self.pos)
        self.ntpp = i32([self.offsets[-1]])

    def pack(self, silu):
        packed = torch.empty(chord.chord_mxfp4_prepack_bytes(self.E, self.N, self.K), dtype=torch.uint8, device="cuda")
        chord.chord_mxfp4_prepack(torch.from_numpy(pack(self.code)).cuda(), torch.from_numpy(self.scale).cuda(), silu,
                                  packed)
        return packed

    def rows(self):
        r = torch.empty(chord.chord_mxfp4_rows_bytes(self.cap, self.K), dtype=torch.uint8, device="cuda")
        # padding holds what it happens to hold: nothing of it may reach a result
        r.fill_(0xFF)
        chord.chord_mxfp4_quantize_rows(self.x, self.d_pos, 1, None, self.cap, r)
        return r

    def product(self, silu, packed=None, rows=None, ws=None, status=None, stream=None):
        C = torch.full((self.cap, self.N // 2 if silu else self.N), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = workspace() if ws is None else ws
        chord.chord_mxfp4_moe_gemm(self.rows() if rows is None else rows, self.pack(silu) if packed is None else packed,
                                   self.E, self.N, self.K, self.d_counts, self.d_offsets, self.cap,
                                   chord.CHORD_EPI_SILU_MUL if silu else chord.CHORD_EPI_STORE, C, ws, status, stream)
        return C

    def check(self, C, silu):
        a = values(*ref_quantize(self.x.double().cpu().numpy()))
        got = C.double().cpu().numpy()
        seen = np.zeros(self.cap, bool)
        for e in range(self.E):
            t = np.nonzero(self.expert == e)[0]
            if not len(t):
                continue
            w = values(self.code[e], self.scale[e])
            y, d = a[t] @ w.T, self.K * 2.0 ** -23 * (np.abs(a[t]) @ np.abs(w).T)
            bound = 0.0
            if silu:
                h = self.N // 2
                g, u, dg, du = y[:, :h], y[:, h:], d[:, :h], d[:, h:]
                with np.errstate(over="ignore"):
                    y = g / (1 + np.exp(-g)) * u
                bound = 1.1 * dg * np.abs(u) + np.abs(g) * du + 1.1 * dg * du + 2.0 ** -18 * np.abs(y)
            else:
                bound = d
            bound = bound + 2.0 ** -8 * np.abs(y) + 2.0 ** -126
            err = np.abs(got[self.pos[t]] - y)
            assert (err <= bound).all(), f"expert {e}: worst {np.max(err / bound):.2f} of the bound"
            seen[self.pos[t]] = True
        assert (got[~seen] == 7.0).all(), "a padding row was written"


_ws = {}


def workspace():
    if not _ws:
        _ws["w"] = torch.zeros(chord.chord_mxfp4_moe_gemm_workspace_bytes(), dtype=torch.uint8, device="cuda")
    return _ws["w"]


CASES = [
    # counts, block, N, K
    ([1], 8, 128, 256),                              # one token, one tile, one unit
    ([1], 8, 8, 32),                                 # the smallest operand
    ([0, 0, 3, 0], 16, 136, 96),                     # experts without rows; N and K inside a tile and a unit
    ([16, 1, 15, 17], 16, 256, 512),
    ([9, 8, 7], 8, 384, 288),                        # tiles that start at multiples of 8 only
    ([128, 129, 127], 128, 256, 1024),
    ([240, 241, 33], 32, 128, 768),                  # one and two row tiles
    ([700, 1, 0, 480], 16, 264, 320),
    ([2, 1, 1], 8, 512, 7168),                       # few items: K split over many CTAs
    ([1] * 40, 8, 64, 2048),
    ([5] * 300, 16, 16, 64),                         # more experts than threads
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("silu", [False, True])
def test_product(case, silu):
    counts, bm, N, K = CASES[case]
    N = -(-N // 16) * 16 if silu else N
    ex = Experts(counts, bm, N, K, case)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    C = ex.product(silu, status=status)
    assert status.item() == 0
    ex.check(C, silu)
    # the same call again: the workspace's counters are zero, the sums in the same order
    assert torch.equal(C, ex.product(silu))


DIVIDED = [
    ([1] * 200, 8, 128, 2048),                       # K in parts, whole items behind them
    ([48, 33, 47], 16, 392, 4096),                   # K in parts, the largest row tile for that
    ([7] * 80, 8, 264, 1792),                        # parts of one unit; an odd number of weight tiles
    ([90] * 160, 32, 128, 512),                      # rows in runs, whole items behind them
    ([64] * 77, 16, 128, 512),                       # more than half the CTAs busy: not divided
    ([300, 50], 16, 392, 7168),                      # rows in runs, unequal row tiles
    ([0] * 70 + [1] + [0] * 500 + [2] + [0] * 451 + [1], 8, 16, 64),   # 1024 experts, few with rows
]


@pytest.mark.parametrize("case", range(len(DIVIDED)))
@pytest.mark.parametrize("silu", [False, True])
def test_product_of_divided_items(case, silu):
    counts, bm, N, K = DIVIDED[case]
    N = -(-N // 16) * 16 if silu else N
    ex = Experts(counts, bm, N, K, 100 + case)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    C = ex.product(silu, status=status)
    assert status.item() == 0
    ex.check(C, silu)
    assert torch.equal(C, ex.product(silu))


@pytest.mark.parametrize("name", ["fp16", "fp32"])
def test_product_of_other_row_types(name):
    ex = Experts([3, 20, 0, 7], 16, 128, 512, 21, TYPES[name])
    ex.check(ex.product(False), False)


def test_rows_without_positions():
    """Row r of x to row r below the padded total: a product's output quantised for the next."""
    ex = Experts([5, 0, 18], 16, 128, 288, 22)
    x = torch.zeros((ex.cap, ex.K), dtype=torch.bfloat16, device="cuda")
    x[torch.from_numpy(ex.pos).cuda()] = ex.x
    r = torch.full((chord.chord_mxfp4_rows_bytes(ex.cap, ex.K),), 0xFF, dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_quantize_rows(x, None, 1, ex.ntpp, ex.cap, r)
    assert torch.equal(ex.product(False, rows=r), ex.product(False))


def test_shared_tokens_and_absent_experts():
    """topk 3 with assignments elsewhere (-1): each token quantised once, to each of its rows."""
    ex = Experts([4, 4, 4], 16, 128, 256, 23)
    x = ex.x[:4]
    pos = np.full((4, 3), -1, np.int32)
    for t in range(4):
        pos[t] = [ex.offsets[e] + t for e in range(3)]
    pos[1, 2] = pos[3, 0] = -1
    r = torch.full((chord.chord_mxfp4_rows_bytes(ex.cap, ex.K),), 0xFF, dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_quantize_rows(x, torch.from_numpy(pos.reshape(-1)).cuda(), 3, None, ex.cap, r)
    got = ex.product(False, rows=r).double().cpu().numpy()
    a = values(*ref_quantize(x.double().cpu().numpy()))
    for t in range(4):
        for e in range(3):
            if pos[t, e] < 0:
                continue
            w = values(ex.code[e], ex.scale[e])
            bound = 2.0 ** -8 * np.abs(w @ a[t]) + ex.K * 2.0 ** -23 * (np.abs(w) @ np.abs(a[t]))
            assert (np.abs(got[pos[t, e]] - w @ a[t]) <= bound).all()


def test_a_row_with_infinities_stays_alone():
    """A row that holds an infinity or a NaN gives NaN; every other row is untouched by it."""
    ex = Experts([6, 18], 16, 128, 512, 24)
    clean = ex.product(False)
    ex.x[2, 40], ex.x[5, 511] = float("inf"), float("nan")
    C = ex.product(False)
    bad = ex.pos[[2, 5]]
    assert torch.isnan(C[torch.from_numpy(bad).cuda()]).all()
    keep = np.setdiff1d(np.arange(ex.cap), bad)
    assert torch.equal(C[keep], clean[keep])


def test_many_rows():
    """Thousands of rows of few experts: every CTA walks several items and cuts two."""
    ex = Experts([1500, 700], 128, 640, 512, 25)
    ex.check(ex.product(True), True)


def test_offsets_beyond_32_bits():
    """x beyond 2^32 elements, the row operand beyond 2^31 bytes: the last rows' product."""
    M, K, N = 270000, 16384, 16
    ex = Experts([3], 16, N, K, 29)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = ex.x
    i32 = dict(dtype=torch.int32, device="cuda")
    pos, counts, offsets = torch.arange(M, **i32), torch.tensor([M], **i32), torch.tensor([0, M], **i32)
    cap = M
    assert M * K > 2 ** 32 and chord.chord_mxfp4_rows_bytes(cap, K) > 2 ** 31
    r = torch.empty(chord.chord_mxfp4_rows_bytes(cap, K), dtype=torch.uint8, device="cuda")
    C = torch.full((cap, N), 7.0, dtype=torch.bfloat16, device="cuda")
    chord.chord_mxfp4_quantize_rows(x, pos, 1, None, cap, r)
    chord.chord_mxfp4_moe_gemm(r, ex.pack(False), 1, N, K, counts, offsets, cap, chord.CHORD_EPI_STORE, C, workspace())
    a, w = values(*ref_quantize(ex.x.double().cpu().numpy())), values(ex.code[0], ex.scale[0])
    bound = 2.0 ** -8 * np.abs(a @ w.T) + K * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)
    assert (np.abs(C[-3:].double().cpu().numpy() - a @ w.T) <= bound).all()
    assert not C[:-3].any()
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((M, K // 32), dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_quantize(x, codes, scales)
    chord.chord_mxfp4_dequantize(codes, scales, x)
    assert np.array_equal(x[-3:].double().cpu().numpy(), a) and not x[:-3].any()


def test_stream_and_graph():
    ex = Experts([3, 2, 9], 16, 256, 512, 26)
    packed, rows, ws = ex.pack(False), ex.rows(), torch.zeros_like(workspace())
    want = ex.product(False, packed, rows, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ex.product(False, packed, rows, ws, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    C = torch.full_like(want, 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chord.chord_mxfp4_quantize_rows(ex.x, ex.d_pos, 1, None, ex.cap, rows)
        chord.chord_mxfp4_moe_gemm(rows, packed, ex.E, ex.N, ex.K, ex.d_counts, ex.d_offsets, ex.cap,
                                   chord.CHORD_EPI_STORE, C, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, want)


def test_device_errors():
    """A header of other weights and an order beyond the capacity are recorded; nothing is written for them."""
    ex = Experts([3, 2], 16, 128, 256, 27)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    C = ex.product(True, packed=ex.pack(False), status=status)      # packed without gate_up
    assert status.item() == chord.CHORD_ERR_PREPACK_MISMATCH and (C == 7.0).all()
    status.zero_()
    ex.d_offsets[1] = ex.cap
    C = ex.product(False, status=status)
    assert status.item() == chord.CHORD_ERR_INVALID_ARG
    assert (C[16:] == 7.0).all() and not (C[:3] == 7.0).all()


def test_a_wait_that_runs_out():
    """With the items withheld every role's wait runs out: the status says so, nothing is
    written, and the next call on the same workspace is exact."""
    ex = Experts([3, 20], 16, 256, 512, 30)
    packed, rows, ws = ex.pack(False), ex.rows(), torch.zeros_like(workspace())
    want = ex.product(False, packed, rows, ws)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    chord.chord_debug_force_timeout(True)
    try:
        C = ex.product(False, packed, rows, ws, status)
        torch.cuda.synchronize()
    finally:
        chord.chord_debug_force_timeout(False)
    assert status.item() == chord.CHORD_ERR_TIMEOUT and (C == 7.0).all()
    status.zero_()
    assert torch.equal(ex.product(False, packed, rows, ws, status), want) and status.item() == 0


def test_refusals():
    ex = Experts([3, 2], 16, 128, 256, 28)
    packed, rows, ws = ex.pack(False), ex.rows(), workspace()
    u8 = dict(dtype=torch.uint8, device="cuda")

    def refused(code, f, *args, **kw):
        with pytest.raises(chord.ChordError) as e:
            f(*args, **kw)
        assert e.value.code == code

    arg = chord.CHORD_ERR_INVALID_ARG
    x = torch.zeros((2, 48), dtype=torch.bfloat16, device="cuda")
    refused(arg, chord.chord_mxfp4_quantize, x, torch.empty((2, 24), **u8), torch.empty(3, **u8))   # K % 32
    refused(arg, chord.chord_mxfp4_quantize_rows, ex.x, ex.d_pos, 1, None, ex.cap, rows[:-16])      # short operand
    refused(arg, chord.chord_mxfp4_quantize_rows, ex.x, None, 1, None, ex.cap, rows)                # no row count
    refused(arg, chord.chord_mxfp4_prepack, torch.empty((1, 4, 16), **u8), torch.empty(4, **u8), False,
            torch.empty(1 << 20, **u8))                                                             # N % 8
    refused(arg, chord.chord_mxfp4_prepack, torch.empty((1, 8, 16), **u8), torch.empty(8, **u8), True,
            torch.empty(1 << 20, **u8))                                                             # gate_up: N % 16
    refused(arg, chord.chord_mxfp4_prepack, torch.empty((1, 8, 16), **u8), torch.empty(8, **u8), False,
            torch.empty(64, **u8))                                                                  # small blob
    C = torch.full((ex.cap, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    call = lambda **kw: chord.chord_mxfp4_moe_gemm(*[kw.get(k, v) for k, v in dict(
        rows=rows, w=packed, E=ex.E, N=ex.N, K=ex.K, counts=ex.d_counts, offsets=ex.d_offsets, cap=ex.cap,
        epi=chord.CHORD_EPI_STORE, C=C, ws=ws).items()])
    refused(arg, call, epi=chord.CHORD_EPI_WEIGHTED_ADD)
    refused(arg, call, rows=rows[:-16])
    refused(chord.CHORD_ERR_WORKSPACE_TOO_SMALL, call, ws=ws[:1024])
    with pytest.raises(ValueError):
        call(C=C[:-1])
    with pytest.raises(ValueError):
        call(w=packed[:-16])
    with pytest.raises(ValueError):
        call(counts=ex.d_counts[:1])
    with pytest.raises(TypeError):
        call(ws=ws.int())
    with pytest.raises(TypeError):
        chord.chord_mxfp4_quantize(x.double(), torch.empty((2, 24), **u8), torch.empty(3, **u8))
    torch.cuda.synchronize()
    assert (C == 7.0).all()
