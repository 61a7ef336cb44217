"""GPU tests of the MXFP4 product where every CTA walks many items with random data: the
item ring wraps, accumulators and stages are used again and again, at each layout that the
largest row tile selects, with an even and an odd number of weight tiles.  Every row is
compared with 64 bits under the bounds derived in test_gpu_mxfp4.py."""
import numpy as np
import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import chord

from gpu_util import ensure_lib
from test_gpu_mxfp4 import LEVELS, ref_quantize, values, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def row_tile(counts, K):
    """Items' row tiles: how many there are, and the rows of the largest, for runs of counts[e] rows."""
    most = 96 if -(-K // 256) <= 14 else 224
    tiles = [-(-c // most) for c in counts]
    return sum(tiles), max(-(-(-(-c // t)) // 16) * 16 for c, t in zip(counts, tiles) if t)


CASES = {
    # counts, block, N, K, largest row tile, least items per CTA
    "full tiles, odd": ([5] * 220 + [1344, 1000], 16, 1408, 3840, 224, 9),
    "full tiles, even": ([1000, 224, 448, 223] + [3] * 220, 8, 1536, 3840, 224, 9),
    "tiles of 160": ([160] * 24 + [9] * 130, 32, 2304, 4096, 160, 9),
    "short K, tiles of 96": ([960] * 6 + [97, 5, 96, 200] + [30] * 40, 16, 4096, 512, 96, 9),
    "one unit": ([96] * 40 + [1] * 60, 16, 3968, 256, 96, 9),
    "three accumulators": ([64, 1, 50] * 100, 16, 1152, 768, 64, 9),
    "four accumulators": ([5, 16, 1] * 100, 8, 1280, 2048, 16, 9),
    "four accumulators of 48": ([48, 20, 33, 1] * 75, 16, 1152, 1024, 48, 9),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("silu", [False, True])
def test_many_items_per_cta(name, silu):
    counts, bm, N, K, tile, least = CASES[name]
    tiles, largest = row_tile(counts, K)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert largest == tile
    assert -(-N // 256) * tiles >= least * sms

    E = len(counts)
    rng = np.random.default_rng(E + K)
    g = torch.Generator(device="cuda").manual_seed(E + N)
    offsets = np.concatenate([[0], np.cumsum(-(-np.array(counts) // bm) * bm)])
    cap = int(offsets[-1])
    at = np.concatenate([offsets[e] + np.arange(c) for e, c in enumerate(counts)])
    pos = rng.permutation(at)                                 # row of token t
    x = torch.randn((len(at), K), generator=g, device="cuda").to(torch.bfloat16)
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g, device="cuda")
    scales = torch.randint(118, 128, (E, N, K // 32), dtype=torch.uint8, generator=g, device="cuda")
    packed = torch.empty(chord.chord_mxfp4_prepack_bytes(E, N, K), dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_prepack(codes, scales, silu, packed)
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    rows = torch.full((chord.chord_mxfp4_rows_bytes(cap, K),), 0xFF, dtype=torch.uint8, device="cuda")
    chord.chord_mxfp4_quantize_rows(x, i32(pos), 1, None, cap, rows)
    status = i32([0])
    cols = N // 2 if silu else N

    def product():
        C = torch.full((cap, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        chord.chord_mxfp4_moe_gemm(rows, packed, E, N, K, i32(counts), i32(offsets), cap,
                                   chord.CHORD_EPI_SILU_MUL if silu else chord.CHORD_EPI_STORE, C, workspace(), status)
        return C

    C = product()
    assert status.item() == 0

    order = np.empty(cap, np.int64)
    order[pos] = np.arange(len(pos))
    a_all = torch.from_numpy(values(*ref_quantize(x.double().cpu().numpy()))).cuda()
    signed = torch.tensor(np.concatenate([LEVELS, -LEVELS]), device="cuda")
    seen = torch.zeros(cap, dtype=torch.bool, device="cuda")
    for e, c in enumerate(counts):
        w = torch.empty((N, K), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = signed[(codes[e] & 15).long()], signed[(codes[e] >> 4).long()]
        w *= torch.exp2(scales[e].double() - 127).repeat_interleave(32, 1)
        here = slice(int(offsets[e]), int(offsets[e]) + c)
        a = a_all[torch.from_numpy(order[here]).cuda()]
        y, d = a @ w.T, K * 2.0 ** -23 * (a.abs() @ w.abs().T)
        bound = d
        if silu:
            h = N // 2
            gate, up, dg, du = y[:, :h], y[:, h:], d[:, :h], d[:, h:]
            y = gate * torch.sigmoid(gate) * up
            bound = 1.1 * dg * up.abs() + gate.abs() * du + 1.1 * dg * du + 2.0 ** -18 * y.abs()
        bound = bound + 2.0 ** -8 * y.abs() + 2.0 ** -126
        err = (C[here].double() - y).abs()
        assert (err <= bound).all(), f"expert {e}: worst {(err / bound).max().item():.2f} of the bound"
        seen[here] = True
    assert (C[~seen] == 7.0).all(), "a padding row was written"
    assert torch.equal(C, product())
