"""Host-side checks of the rows in expert order and the MXFP4 entry points that need
no GPU: sizes, and argument checks that reject bad calls before any launch."""
import ctypes

import pytest

from w4a16_int4_weight_sigmoid_gb300 import build as B
from w4a16_int4_weight_sigmoid_gb300 import chord

P = ctypes.c_void_p(16)     # never dereferenced: the checks fail first
ARG, WS = chord.CHORD_ERR_INVALID_ARG, chord.CHORD_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module")
def L():
    B.build()
    return chord.lib()


def refused(L, code, word, rc):
    assert rc == code
    assert word in L.chord_last_error_string().decode()


def test_sizes(L):
    unit = 128 * 128 + 128 * 8                                    # 128 weight rows x 256 of K, and their scales
    assert L.chord_mxfp4_prepack_bytes(1, 8, 32) == 256 + unit    # N padded to 128, K to 256
    assert L.chord_mxfp4_prepack_bytes(48, 4096, 7168) == 256 + 48 * 32 * 28 * unit
    assert L.chord_mxfp4_prepack_bytes(1, 8, 48) == 0             # K % 32
    assert L.chord_mxfp4_prepack_bytes(1, 12, 32) == 0            # N % 8
    assert L.chord_mxfp4_prepack_bytes(0, 8, 32) == 0
    assert L.chord_mxfp4_rows_bytes(1, 32) == 256 * 136           # a slab of 256 rows, one unit
    assert L.chord_mxfp4_rows_bytes(241, 512) == 256 * 2 * 136
    assert L.chord_mxfp4_rows_bytes(242, 512) == 512 * 2 * 136    # a tile may read 15 rows past the last
    assert L.chord_mxfp4_rows_bytes(8, 40) == 0
    assert L.chord_mxfp4_moe_gemm_workspace_bytes() > 0


def test_rows_are_checked(L):
    f = lambda dtype=0, xs=64, M=4, k=2, H=64, cap=64, os=64, x=P, pos=P: L.chord_moe_permute(
        x, dtype, xs, pos, P, P, M, k, H, cap, P, os, None)
    refused(L, ARG, "dtype", f(dtype=3))
    refused(L, ARG, "topk", f(k=0))
    refused(L, ARG, "topk", f(k=33))
    refused(L, ARG, "M=-1", f(M=-1))
    refused(L, ARG, "row length", f(H=0))
    refused(L, ARG, "row length", f(H=(1 << 24) + 1, xs=1 << 25, os=1 << 25))
    refused(L, ARG, "stride", f(os=63))
    refused(L, ARG, "stride", f(xs=-1))
    refused(L, ARG, "x", f(x=None))
    refused(L, ARG, "aligned", f(x=ctypes.c_void_p(17)))
    refused(L, ARG, "aligned", f(dtype=2, x=ctypes.c_void_p(18)))
    refused(L, ARG, "null", f(pos=None))
    refused(L, ARG, "rows", f(cap=1 << 31))
    assert f(M=0) == 0 and f(cap=0) == 0
    refused(L, ARG, "dx", L.chord_moe_permute_backward(P, 0, 64, P, 4, 2, 64, 64, None, 64, None))
    refused(L, ARG, "null", L.chord_moe_unpermute(P, 0, 64, None, P, 4, 2, 64, 64, P, 64, None))
    refused(L, ARG, "dy", L.chord_moe_unpermute_backward(P, P, 0, 64, 64, P, P, P, P, 4, 2, 64, 64, P, 8, P, None))
    refused(L, ARG, "null", L.chord_moe_unpermute_backward(P, P, 0, 64, 64, P, P, P, P, 4, 2, 64, 64, P, 64, None, None))


def test_quantisation_is_checked(L):
    refused(L, ARG, "K=40", L.chord_mxfp4_quantize(P, 0, 64, 4, 40, P, P, None))
    refused(L, ARG, "dtype", L.chord_mxfp4_quantize(P, 9, 64, 4, 64, P, P, None))
    refused(L, ARG, "rows", L.chord_mxfp4_quantize(P, 0, 64, -1, 64, P, P, None))
    refused(L, ARG, "null", L.chord_mxfp4_quantize(P, 0, 64, 4, 64, P, None, None))
    refused(L, ARG, "16-byte", L.chord_mxfp4_quantize(P, 0, 64, 4, 64, ctypes.c_void_p(20), P, None))
    refused(L, ARG, "stride", L.chord_mxfp4_dequantize(P, P, 4, 64, P, 0, 32, None))
    assert L.chord_mxfp4_quantize(None, 0, 64, 0, 64, None, None, None) == 0
    big = 1 << 30
    refused(L, ARG, "K=8", L.chord_mxfp4_quantize_rows(P, 0, 64, 4, 8, P, 2, P, 64, P, big, None))
    refused(L, ARG, "bytes", L.chord_mxfp4_quantize_rows(P, 0, 64, 4, 64, P, 2, P, 64, P, 100, None))
    refused(L, ARG, "null", L.chord_mxfp4_quantize_rows(P, 0, 64, 4, 64, None, 2, None, 64, P, big, None))
    refused(L, ARG, "N=12", L.chord_mxfp4_prepack(P, P, 1, 12, 64, 0, P, big, None))
    refused(L, ARG, "gate_up", L.chord_mxfp4_prepack(P, P, 1, 8, 64, 1, P, big, None))
    refused(L, ARG, "packed_bytes", L.chord_mxfp4_prepack(P, P, 1, 16, 64, 1, P, 100, None))


def test_product_is_checked(L):
    big = 1 << 40
    f = lambda rb=big, E=4, N=128, K=256, cap=64, epi=0, C=P, ws=big, w=P: L.chord_mxfp4_moe_gemm(
        P, rb, w, E, N, K, P, P, cap, epi, C, P, ws, None, None)
    refused(L, ARG, "E_local", f(E=0))
    refused(L, ARG, "E_local", f(E=1025))
    refused(L, ARG, "N=12", f(N=12))
    refused(L, ARG, "K=100", f(K=100))
    refused(L, ARG, "epilogue", f(epi=chord.CHORD_EPI_WEIGHTED_ADD))
    refused(L, ARG, "SiLU", f(N=8, epi=chord.CHORD_EPI_SILU_MUL))
    refused(L, ARG, "2^24", f(K=1 << 25))
    refused(L, ARG, "too large", f(cap=1 << 30, N=1 << 20))
    refused(L, ARG, "null", f(C=None))
    refused(L, ARG, "16-byte", f(w=ctypes.c_void_p(24)))
    refused(L, ARG, "rows", f(rb=100))
    refused(L, WS, "workspace", f(ws=100))
    assert f(cap=0) == 0


def test_extension_is_built_and_refuses_host_tensors(L):
    """The C++ binding loads without a GPU and checks before it calls."""
    import torch
    t = torch.zeros((4, 64), dtype=torch.bfloat16)
    i = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        chord.chord_moe_permute(t, i, i, i[:1], 2, t)
    with pytest.raises(TypeError, match="torch.Tensor"):
        chord.chord_mxfp4_quantize([1, 2], i, i)
    with pytest.raises(ValueError, match="CUDA"):
        chord.chord_mxfp4_dequantize(i, i, t)


def test_rows_without_positions_have_no_topk(L):
    """topk is not read when row r of x is row r of the order; the other checks hold."""
    f = lambda k, M=1 << 27, cap=0, pos=None, total=P: L.chord_mxfp4_quantize_rows(P, 0, 64, M, 64, pos, k, total, cap,
                                                                                   P, 1 << 40, None)
    assert f(0) == 0 and f(33) == 0 and f(16) == 0
    refused(L, ARG, "topk", f(0, pos=P))
    refused(L, ARG, "M*topk", f(16, pos=P))
    refused(L, ARG, "M=-1", f(0, M=-1))
    refused(L, ARG, "null", f(0, M=4, cap=64, total=None))
