"""GPU tests of the rows in expert order and of the MXFP4 product at the ends of their
ranges: the longest rows, gates far below zero, orders that are none, and launches whose
CTAs walk many items.  Bounds as derived in test_gpu_expert_rows.py and test_gpu_mxfp4.py."""
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord

from gpu_util import ensure_lib

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
