"""The experts' product in 16 bits and its weights' gradient.

Operands are small integers, so that every product and every partial sum is
exact in FP32 whatever the order of the sum, and the result is the exact sum
rounded once: compared bit for bit with the 64-bit product.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
LEFT = 77.0          # what rows that are not written hold


def order(counts, gaps=None):
    """Counts and offsets of experts whose rows follow one another after `gaps` rows each."""
    gaps = gaps or [0] * len(counts)
    offsets, at = [], 0
    for c, g in zip(counts, gaps):
        at += g
        offsets.append(at)
        at += c
    i32 = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(counts, **i32), torch.tensor(offsets + [at], **i32), at


def integers(g, *shape, dtype, most=2):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dtype)


def rows_of(counts, offsets):
    """A mask of the rows that are an expert's."""
    c, o = counts.tolist(), offsets.tolist()
    return [(e, slice(o[e], o[e] + c[e])) for e in range(len(c)) if c[e]]


def workspace():
    from w4a16_int4_weight_sigmoid_gb300 import chord
    return torch.zeros(chord.chord_expert_gemm_workspace_bytes(), dtype=torch.uint8, device="cuda")


def product(x, w, counts, offsets, transpose, out=None):
    from w4a16_int4_weight_sigmoid_gb300 import chord
    E, N, K = w.shape
    if out is None:
        out = torch.full((x.shape[0], K if transpose else N), LEFT, dtype=x.dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    chord.chord_expert_gemm(x, w, counts, offsets, out, workspace(), transpose, status)
    assert status.item() == 0
    return out


def expected_product(x, w, counts, offsets, transpose):
    E, N, K = w.shape
    out = torch.full((x.shape[0], K if transpose else N), LEFT, dtype=x.dtype, device="cuda")
    for e, at in rows_of(counts, offsets):
        out[at] = (x[at].double() @ (w[e].double() if transpose else w[e].double().T)).to(x.dtype)
    return out


def check_product(counts, K, N, transpose, dtype, gaps=None, extra=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, o, rows = order(counts, gaps)
    inner = N if transpose else K
    x = torch.full((rows + extra, inner), float("nan"), dtype=dtype, device="cuda")
    for _, at in rows_of(c, o):
        x[at] = integers(g, at.stop - at.start, inner, dtype=dtype)
    w = integers(g, len(counts), N, K, dtype=dtype)
    got = product(x, w, c, o, transpose)
    assert torch.equal(got, expected_product(x, w, c, o, transpose))


SHAPES = [
    ([5], 64, 64),                        # one box of the contraction
    ([1], 8, 8),                          # the smallest
    ([32], 64, 256),                      # a whole tile
    ([33, 0, 1], 72, 264),                # tiles end behind the tensors' edges
    ([256, 257, 31], 200, 520),           # one and two row tiles
    ([0, 0, 3, 0, 700], 640, 328),        # more boxes than stages
    ([2000], 136, 600),                   # eight row tiles
    ([2305, 7], 72, 1032),                # groups of row tiles
    ([1] * 40, 256, 512),                 # decoding
]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_product(counts, K, N, transpose, dtype):
    check_product(counts, K, N, transpose, dtype)
    if not transpose:
        check_product(counts, K, N, False, dtype, extra=200)     # (no longer a handful of rows for the host)


# a handful of rows: dot products, K shared by all warps, by some, by one; runs of many lengths; more rows of an
# expert than go at once; experts without rows; more than one run a CTA (an order of other counts than the host expects)
FEW = [
    ([1], 8, 8), ([1], 256, 7168), ([2], 264, 72), ([3], 1000, 520), ([1, 0, 2, 0, 7], 4104, 136), ([1] * 8, 7168, 512),
    ([0] * 500 + [1, 2] * 6, 136, 264), ([8], 520, 4096), ([1] * 100, 72, 1000), ([5] * 16, 2048, 512),
    ([0, 64, 0, 0, 0, 0, 0, 0], 512, 264), ([1] * 12 + [0] * 4, 16400, 200), ([0] * 1000 + [3] * 24, 72, 40),
    ([1] * 100, 520, 520),
]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("counts,K,N", FEW)
def test_product_of_a_handful_of_rows(counts, K, N, dtype):
    check_product(counts, K, N, False, dtype)
    check_product(counts, K, N, False, dtype, gaps=[1 if i < 5 else 0 for i in range(len(counts))], seed=1)


@pytest.mark.parametrize("transpose", [False, True])
def test_product_rows_between_experts_are_left(transpose):
    check_product([17, 0, 260, 1], 128, 264, transpose, BF16, gaps=[3, 7, 1, 64], extra=9)


@pytest.mark.parametrize("transpose", [False, True])
def test_product_many_experts(transpose):
    check_product([i % 3 for i in range(1024)], 64, 72, transpose, BF16)


def wgrad(dout, x, counts, offsets, out_dtype):
    from w4a16_int4_weight_sigmoid_gb300 import chord
    dw = torch.full((counts.numel(), dout.shape[1], x.shape[1]), LEFT, dtype=out_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    chord.chord_expert_wgrad(dout, x, counts, offsets, dw, workspace(), status)
    assert status.item() == 0
    return dw


def check_wgrad(counts, K, N, dtype, out_dtype, gaps=None, extra=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, o, rows = order(counts, gaps)
    dout = torch.full((rows + extra, N), float("nan"), dtype=dtype, device="cuda")
    x = torch.full((rows + extra, K), float("nan"), dtype=dtype, device="cuda")
    want = torch.zeros((len(counts), N, K), dtype=out_dtype, device="cuda")
    for e, at in rows_of(c, o):
        n = at.stop - at.start
        dout[at], x[at] = integers(g, n, N, dtype=dtype), integers(g, n, K, dtype=dtype)
        want[e] = (dout[at].double().T @ x[at].double()).to(out_dtype)
    assert torch.equal(wgrad(dout, x, c, o, out_dtype), want)


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (FP16, FP16), (BF16, FP32), (FP16, FP32)])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_weight_gradient(counts, K, N, dtype, out_dtype):
    check_wgrad(counts, K, N, dtype, out_dtype)


@pytest.mark.parametrize("count", [1, 15, 16, 17, 63, 64, 65, 80, 127, 128])
def test_weight_gradient_ends_inside_a_box(count):
    check_wgrad([count, 3, count], 136, 264, BF16, FP32, gaps=[1, 2, 0], extra=5)


# few rows and a long contraction: items are cut (one tile in 76 parts, parts of
# different lengths, an odd number of steps, cut items before whole ones)
CUT = [
    ([1], 7168, 8),
    ([3], 1032, 264),
    ([1] * 8, 2056, 512),
    ([64, 0, 33, 5], 1640, 520),
    ([2] * 90, 1024, 72),
    ([7] * 50, 1096, 512),
    ([32] * 3, 1984, 2600),
]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts,K,N", CUT)
def test_product_cut_along_the_contraction(counts, K, N, transpose):
    check_product(counts, N if transpose else K, K if transpose else N, transpose, BF16, gaps=[3] * len(counts), extra=200)


def test_one_workspace_for_many_calls():
    """Calls that cut their items, one after another on one workspace, and random values: the same bits every time,
    and every counter zero after each call."""
    from w4a16_int4_weight_sigmoid_gb300 import chord
    g = torch.Generator(device="cuda").manual_seed(3)
    ws = workspace()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = {}
    for turn in range(6):
        for i, (counts, K, N) in enumerate(CUT):
            c, o, rows = order(counts)
            rows += 200                  # (not a handful for the host)
            if turn == 0:
                x = torch.randn((rows, K), generator=g, device="cuda").to(BF16)
                w = torch.randn((len(counts), N, K), generator=g, device="cuda").to(BF16)
                first[i] = (x, w, None)
            x, w, want = first[i]
            out = torch.full((rows, N), LEFT, dtype=BF16, device="cuda")
            chord.chord_expert_gemm(x, w, c, o, out, ws, False, status)
            assert not ws[:chord.CHORD_EXPERT_GEMM_COUNTER_BYTES].any()
            if want is None:
                first[i] = (x, w, out)
            else:
                assert torch.equal(out, want)
    assert status.item() == 0


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("counts,K,N", [([2] * 8, 7168, 512), ([2] * 80, 2048, 328), ([700, 30], 1000, 328)])
def test_random_values(counts, K, N, transpose):
    """Sums of n products in FP32, in any order, are off by at most n 2^-23 of the sum of the magnitudes, and one
    rounding to BF16 by 2^-8 of the result."""
    g = torch.Generator(device="cuda").manual_seed(5)
    c, o, rows = order(counts)
    inner = N if transpose else K
    x = torch.randn((rows, inner), generator=g, device="cuda").to(BF16)
    w = torch.randn((len(counts), N, K), generator=g, device="cuda").to(BF16)
    got = product(x, w, c, o, transpose)
    for e, at in rows_of(c, o):
        we = w[e].double() if transpose else w[e].double().T
        want, size = x[at].double() @ we, x[at].double().abs() @ we.abs()
        assert ((got[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + inner * 2.0 ** -23 * size).all()


# uneven popularity: experts are taken by falling rows up to 256 of them, in their order above
@pytest.mark.parametrize("experts", [2, 40, 255, 256, 257, 300])
def test_uneven_popularity(experts):
    counts = [(i * i * 37 + 11) % 290 if i % 5 else 0 for i in range(experts)]
    counts[experts // 2] = 700
    for transpose in (False, True):
        check_product(counts, 72, 136, transpose, BF16, gaps=[i % 3 for i in range(experts)])
    check_wgrad(counts, 72, 136, FP16, FP32, gaps=[i % 3 for i in range(experts)])


def test_equal_experts_in_many_rounds():
    """More items than clusters, dealt forth and back."""
    check_product([96] * 60, 136, 1288, False, BF16)
    check_wgrad([96] * 60, 520, 520, BF16, BF16)


@pytest.mark.parametrize("count", [767, 768, 769, 832, 1536, 1537, 3000, 5001])
def test_fp32_gradient_added_up_in_parts(count):
    """Sums over more than 768 rows: the parts between others' rows, edges of dW, an empty expert, short ones."""
    check_wgrad([count, 0, 70], 328, 264, BF16, FP32, gaps=[3, 0, 5], extra=70)


@pytest.mark.parametrize("mean", [0.0, 1.0])
def test_fp32_gradient_of_many_rows_keeps_its_accuracy(mean):
    """16 rows at a time go into an FP32 sum that is cut off: 48 times 2^-23 of the partial sum at most in a part, and
    each of the 11 additions of parts rounds by 2^-24: below 2^-17 of the sum of the magnitudes.  The result was off by
    2e-5 of itself in the 2-norm where one sum took all rows; here by less than 3e-6 (48 / 2 cuts of 2^-24 on average,
    against sums of growing size)."""
    rows = 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    c, o, _ = order([rows])
    d = (torch.randn((rows, 256), generator=g, device="cuda") + mean).to(BF16)
    x = (torch.randn((rows, 264), generator=g, device="cuda") + mean).to(BF16)
    got = wgrad(d, x, c, o, FP32)[0].double()
    want, size = d.double().T @ x.double(), d.double().abs().T @ x.double().abs()
    assert ((got - want).abs() <= 2.0 ** -17 * size).all()
    assert (got - want).norm() <= 3e-6 * want.norm()
    assert torch.equal(got, wgrad(d, x, c, o, FP32)[0].double())


@pytest.mark.parametrize("K,N", [(1 << 20, 8), (8, 1 << 20)])
def test_the_largest_sizes(K, N):
    """Up to 2^20 of N and K: the sums of 2^20 products of at most 4 are below 2^24, exact in FP32."""
    for transpose in (False, True):
        check_product([3, 0, 1], K, N, transpose, BF16)
        check_product([3, 0, 1], K, N, transpose, BF16, extra=200)
    check_wgrad([3, 0, 1], K, N, BF16, FP32)


def test_no_rows_at_all():
    for extra in (3, 300):
        for transpose in (False, True):
            check_product([0, 0, 0], 64, 72, transpose, BF16, extra=extra)
        check_wgrad([0, 0, 0], 64, 72, BF16, BF16, extra=extra)


# last rounds that leave most of the clusters idle: few items in all, few behind whole rounds, one, edges of a tile
# that hold next to nothing
@pytest.mark.parametrize("counts,K,N", [
    ([200], 136, 264), ([256] * 3, 64, 512), ([255] * 20, 72, 1024), ([90] * 77, 64, 200), ([33, 250, 100], 328, 2056),
    ([129], 1000, 8), ([70], 8, 520), ([1024], 264, 264),
])
def test_last_rounds(counts, K, N):
    for transpose in (False, True):
        check_product(counts, K, N, transpose, BF16, gaps=[1] * len(counts), extra=200)
    for out in (BF16, FP32):
        check_wgrad(counts, K, N, BF16, out, gaps=[1] * len(counts))
        check_wgrad(counts, N, K, BF16, out, gaps=[1] * len(counts))
