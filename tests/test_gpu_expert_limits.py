"""GPU tests of the rows in expert order and of the MXFP4 product at the ends of their
ranges: the longest rows, gates far below zero, orders that are none, and launches whose
CTAs walk many items.  Bounds as derived in test_gpu_expert_rows.py and test_gpu_mxfp4.py."""
import numpy as np
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord

from gpu_util import ensure_lib
from test_gpu_mxfp4 import LEVELS, Experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


# ------------------------------------------------------------------ long rows
LONGEST = 1 << 24


@pytest.mark.parametrize("name,H,off", [
    ("fp32", LONGEST, 0), ("fp32", LONGEST, 1), ("fp32", LONGEST, 4), ("fp32", LONGEST - 4, 0),
    ("bf16", LONGEST, 0), ("bf16", LONGEST, 1), ("bf16", LONGEST - 1, 0), ("fp16", LONGEST, 3),
])
def test_the_longest_rows(name, H, off):
    """One token of the longest rows, at each size of access that they allow: to two rows,
    back, and both gradients.  Small integers and weights of 1/2 and 1/4, so sums are exact."""
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]
    g = torch.Generator(device="cuda").manual_seed(H + off)

    def row(n=1):
        b = torch.empty(n * H + off, dtype=dtype, device="cuda")
        b[:] = torch.randint(-4, 5, b.shape, generator=g, dtype=torch.int8, device="cuda")
        return b[off:].view(n, H)

    i32 = dict(dtype=torch.int32, device="cuda")
    pos, order, total = torch.tensor([1, 0], **i32), torch.tensor([1, 0], **i32), torch.tensor([2], **i32)
    w = torch.tensor([[0.5, 0.25]], device="cuda")
    x, y = row(), row(2)
    out, back, dx, dy = torch.empty_like(y), row(), row(), row(2)
    chord.chord_moe_permute(x, pos, order, total, 2, out)
    assert torch.equal(out, x.expand(2, H))
    chord.chord_moe_permute_backward(y, pos, 2, dx)
    assert torch.equal(dx[0], y[0] + y[1])
    chord.chord_moe_unpermute(y, w, pos, back)
    assert torch.equal(back[0], y[1] / 2 + y[0] / 4)
    dw = torch.empty((1, 2), device="cuda")
    chord.chord_moe_unpermute_backward(x, y, w, pos, order, total, dy, dw)
    assert torch.equal(dy[1], x[0] / 2) and torch.equal(dy[0], x[0] / 4)
    # integer terms whose partial sums stay far below 2^24: exact too
    assert torch.equal(dw[0].double(), (x.double() * y.double()).sum(1).flip(0))


# ------------------------------------------------------- gates far below zero
def encode(v):
    """The code and the scale code that hold v exactly."""
    for e in range(-4, 7):
        if abs(v) / 2.0 ** e in LEVELS:
            return int(np.nonzero(LEVELS == abs(v) / 2.0 ** e)[0][0]) | (8 if v < 0 else 0), 127 + e
    raise ValueError(v)


@pytest.mark.parametrize("K", [256, 4096])            # whole items, and items divided along K
def test_gates_far_below_zero(K):
    """silu(g) u with g from -82 to -100 and u = 6 * 2^120: small factors, ordinary results.

    g and u are exact.  Of silu's own value, in units of it: exp(-|g|) from the fast
    exponential within 2 + 1.173 |g| last places (CUDA's documented bound), the product with
    g and the sum 1 + t half a place each, the fast quotient two, u's product a half: (6 + 1.173
    |g|) 2^-23.  Below FP32's normal range roundings are of 2^-150 instead: one of exp(-|g|),
    two of silu.  And BF16's rounding."""
    third = [-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 2, 3, 4, 6, 8, 12]
    n = len(third)
    ex = Experts([1, 3], 8, 2 * n, K, 40)
    ex.x.zero_()
    ex.x[:, [5, 37, 69]] = 1.0                         # three blocks, so three terms of a gate
    ex.code[:], ex.scale[:] = 0, 127
    for i, v in enumerate(third):
        for block, term in enumerate((-64, -24, -v)):
            ex.code[:, i, 32 * block + 5], ex.scale[:, i, block] = encode(term)
    ex.code[:, n:, 5], ex.scale[:, n:, 0] = 7, 127 + 120
    g, u = -88.0 - np.array(third), LEVELS[7] * 2.0 ** 120
    C = ex.product(True).double().cpu().numpy()[ex.pos]
    silu = g / (1 + np.exp(-g))
    rel = 2.0 ** -8 + (6 + 1.173 * np.abs(g)) * 2.0 ** -23 + 2.0 ** -150 * (1 / np.exp(g) + 2 / np.abs(silu))
    assert (np.abs(C - silu * u) <= rel * np.abs(silu * u)).all(), C[0] / (silu * u)


# --------------------------------------------------------- orders that are none
@pytest.mark.parametrize("counts,offsets,written", [
    ([3, 20, 5], [0, 16, 32, 48], [False] * 3),               # 16 + 20 ends past 32: the next expert's rows
    ([17, 5, 5], [0, 0, 32, 48], [False] * 3),                # two experts at one place
    ([3, 5, 5], [0, 32, 16, 48], [False] * 3),                # descending
    ([3, 5, 5], [32, 16, 0, 48], [False] * 3),
    ([3, 5, 5], [0, 16, 32, -8], [False] * 3),
    ([3, 0, 5], [0, 1 << 20, 0, 48], [False] * 3),            # up and down again
    ([3, -5, 5], [0, 32, 16, 48], [False] * 3),
    ([3, 5, 40], [0, 16, 32, 48], [True, True, False]),       # the last expert past the end of the order
    ([3, 5, 5], [0, 20, 32, 48], [True, False, True]),        # not a multiple of 8
    ([3, -5, 5], [0, 16, 32, 48], [True, False, True]),
    ([3, 2 ** 31 - 1, 5], [0, 16, 32, 48], [True, False, True]),
])
def test_counts_and_offsets_that_are_no_order(counts, offsets, written):
    """An expert whose rows are misaligned or past the capacity is skipped; experts whose rows
    overlap, and offsets that descend, stop the launch.  So the rows of all experts together
    stay within the capacity, as the host assumes."""
    ex = Experts([3, 5, 5], 16, 128, 256, 41)
    good = ex.product(False)
    packed, rows = ex.pack(False), ex.rows()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    C, status = torch.full_like(good, 7.0), i32([0])
    ws = torch.zeros(chord.chord_mxfp4_moe_gemm_workspace_bytes(), dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_moe_gemm(rows, packed, 3, 128, 256, i32(counts), i32(offsets), ex.cap, chord.CHORD_EPI_STORE, C,
                               ws, status)
    assert status.item() == chord.CHORD_ERR_INVALID_ARG
    touched = (C != 7.0).any(1).cpu()
    for e, w in enumerate(written):
        if w and offsets[e] == 16 * e:                        # an expert in its own place: its own values
            at = slice(offsets[e], offsets[e] + counts[e])
            assert torch.equal(C[at], good[at])
    expect = torch.zeros(ex.cap, dtype=torch.bool)
    for e, w in enumerate(written):
        if w:
            expect[offsets[e]:offsets[e] + counts[e]] = True
    assert torch.equal(touched, expect)
    # the counters are zero: a good call on the same workspace is right
    status.zero_()
    assert torch.equal(ex.product(False, packed, rows, ws, status), good) and status.item() == 0


def test_many_experts_of_all_rows():
    """1024 experts that each claim the whole capacity, each of them within it."""
    n, cap, N, K = 1024, 256, 8, 32
    ex = Experts([cap], 16, N, K, 42)
    ex.code, ex.scale = ex.code.repeat(n, 0), ex.scale.repeat(n, 0)
    ex.E = n
    ex.d_counts = torch.full((n,), cap, dtype=torch.int32, device="cuda")
    ex.d_offsets = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    ex.d_offsets[n] = cap
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert (ex.product(False, status=status) == 7.0).all() and status.item() == chord.CHORD_ERR_INVALID_ARG
