"""Host-side checks of the experts' 16-bit products, the gated activation and the rows in 8 bits
that need no GPU: argument checks that reject bad calls before any launch."""
import ctypes

import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import build as B
from w4a16_int4_weight_sigmoid_gb300 import chord

P = ctypes.c_void_p(16)     # never dereferenced: the checks fail first
ARG, WS = chord.CHORD_ERR_INVALID_ARG, chord.CHORD_ERR_WORKSPACE_TOO_SMALL
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    B.build()
    return chord.lib()


def refused(L, code, word, rc):
    assert rc == code
    assert word in L.chord_last_error_string().decode()


def test_workspace_size(L):
    assert L.chord_expert_gemm_workspace_bytes() > chord.CHORD_EXPERT_GEMM_COUNTER_BYTES


def test_product_is_checked(L):
    f = lambda x=P, dtype=0, xs=256, w=P, ws_=256, es=1 << 15, E=4, N=128, K=256, t=0, c=P, o=P, cap=64, out=P, os=128, \
        wk=P, wb=BIG: L.chord_expert_gemm(x, dtype, xs, w, ws_, es, E, N, K, t, c, o, cap, out, os, wk, wb, None, None)
    refused(L, ARG, "dtype", f(dtype=2))
    refused(L, ARG, "dtype", f(dtype=9))
    refused(L, ARG, "E_local", f(E=0))
    refused(L, ARG, "E_local", f(E=1025))
    for bad in (0, -8, 12, (1 << 20) + 8):
        refused(L, ARG, "multiples of 8", f(N=bad))
        refused(L, ARG, "multiples of 8", f(K=bad))
    refused(L, ARG, "rows", f(cap=(1 << 30) + 1))
    refused(L, ARG, "too large", f(cap=1 << 30, N=1 << 20))
    refused(L, ARG, "too large", f(cap=1 << 30, K=1 << 20, t=1))
    for name in ("x", "w", "out"):
        refused(L, ARG, name, f(**{name: None}))
        refused(L, ARG, "16-byte", f(**{name: ctypes.c_void_p(24)}))
    refused(L, ARG, "null", f(c=None))
    refused(L, ARG, "null", f(o=None))
    refused(L, ARG, "x: row stride", f(xs=248))
    refused(L, ARG, "x: row stride", f(xs=260))
    refused(L, ARG, "x: row stride", f(xs=0))
    refused(L, ARG, "x: row stride", f(xs=(1 << 36) + 8))
    refused(L, ARG, "w: row stride", f(ws_=128))
    refused(L, ARG, "out: row stride", f(os=120))
    refused(L, ARG, "expert stride", f(es=0))
    refused(L, ARG, "expert stride", f(es=100))
    refused(L, ARG, "x: row stride", f(t=1, xs=64))            # N wide then
    refused(L, ARG, "out: row stride", f(t=1, os=128))         # K wide then
    refused(L, WS, "workspace", f(wb=100))
    refused(L, WS, "workspace", f(wk=None))
    refused(L, ARG, "workspace", f(wk=ctypes.c_void_p(24)))
    assert f(cap=0, x=None, w=None, out=None) == 0


def test_weight_gradient_is_checked(L):
    f = lambda d=P, x=P, dtype=0, ds=128, xs=256, E=4, N=128, K=256, c=P, o=P, cap=64, dw=P, dt=0, wk=P, wb=BIG: \
        L.chord_expert_wgrad(d, x, dtype, ds, xs, E, N, K, c, o, cap, dw, dt, wk, wb, None, None)
    refused(L, ARG, "dtype", f(dtype=2, dt=2))
    refused(L, ARG, "dw_dtype", f(dt=1))
    refused(L, ARG, "dw_dtype", f(dtype=1, dt=0))
    refused(L, ARG, "E_local", f(E=1025))
    refused(L, ARG, "multiples of 8", f(N=4))
    refused(L, ARG, "too large", f(E=1024, N=1 << 20, K=1 << 20))
    refused(L, ARG, "dw", f(dw=None))
    refused(L, ARG, "16-byte", f(dw=ctypes.c_void_p(8)))
    refused(L, ARG, "dout", f(d=None))
    refused(L, ARG, "dout: row stride", f(ds=120))
    refused(L, ARG, "x: row stride", f(xs=255))
    refused(L, ARG, "null", f(c=None))
    refused(L, WS, "workspace", f(wb=100))


def test_rows_in_8_bits_are_checked(L):
    q = lambda x=P, dtype=0, xs=64, rows=4, K=64, c=P, s=P: L.chord_mxfp8_quantize(x, dtype, xs, rows, K, c, s, None)
    refused(L, ARG, "dtype", q(dtype=3))
    refused(L, ARG, "rows", q(rows=-1))
    refused(L, ARG, "K=40", q(K=40))
    refused(L, ARG, "K=0", q(K=0))
    refused(L, ARG, "x", q(x=None))
    refused(L, ARG, "aligned", q(x=ctypes.c_void_p(17)))
    refused(L, ARG, "codes", q(c=None))
    refused(L, ARG, "codes", q(c=ctypes.c_void_p(24)))
    refused(L, ARG, "scales", q(s=None))
    assert q(rows=0, x=None, c=None, s=None) == 0
    refused(L, ARG, "stride", L.chord_mxfp8_dequantize(P, P, 4, 64, P, 0, 32, None))
    refused(L, ARG, "dtype", L.chord_mxfp8_dequantize(P, P, 4, 64, P, 4, 64, None))
    p = lambda c=P, s=P, t=P, n=P, M=4, k=2, K=64, cap=64, out=P, os=64: L.chord_mxfp8_permute(
        c, s, t, n, M, k, K, cap, out, 0, os, None)
    refused(L, ARG, "topk", p(k=0))
    refused(L, ARG, "M=-1", p(M=-1))
    refused(L, ARG, "K=8", p(K=8))
    refused(L, ARG, "stride", p(os=63))
    refused(L, ARG, "null", p(t=None))
    refused(L, ARG, "null", p(n=None))
    refused(L, ARG, "codes", p(c=None))
    assert p(M=0) == 0 and p(cap=0) == 0


def test_gated_activation_is_checked(L):
    f = lambda gu=P, dtype=0, gs=64, w=P, t=P, n=P, M=4, k=2, I=32, cap=64, h=P, hs=32, c=None, s=None: L.chord_swiglu(
        gu, dtype, gs, w, t, n, M, k, I, cap, h, hs, c, s, None)
    refused(L, ARG, "dtype", f(dtype=3))
    refused(L, ARG, "topk", f(k=33))
    refused(L, ARG, "row length", f(I=0))
    refused(L, ARG, "2^23", f(I=(1 << 23) + 1, gs=1 << 25, hs=1 << 24))
    refused(L, ARG, "gu: row stride", f(gs=-1))
    refused(L, ARG, "h: row stride", f(hs=31))
    refused(L, ARG, "gu", f(gu=None))
    refused(L, ARG, "null", f(w=None))
    refused(L, ARG, "null", f(t=None))
    refused(L, ARG, "null", f(n=None))
    refused(L, ARG, "scales", f(c=P))
    refused(L, ARG, "scales", f(s=P))
    refused(L, ARG, "16-byte", f(c=ctypes.c_void_p(24), s=P))
    refused(L, ARG, "I=40", f(I=40, gs=80, hs=40, c=P, s=P))
    assert f(M=0) == 0 and f(cap=0) == 0
    b = lambda dh=P, dtype=0, ds=32, gu=P, gs=64, c=None, s=None, w=P, pos=P, t=P, n=P, M=4, k=2, I=32, cap=64, dgu=P, \
        os=64, dw=P, h=None, hs=0: L.chord_swiglu_backward(dh, dtype, ds, gu, gs, c, s, w, pos, t, n, M, k, I, cap, dgu,
                                                          os, dw, h, hs, None)
    refused(L, ARG, "one of them", b(c=P, s=P))
    refused(L, ARG, "gu", b(gu=None))
    refused(L, ARG, "dweights", b(dw=None))
    refused(L, ARG, "dgu: row stride", b(os=32))
    refused(L, ARG, "dgu", b(dgu=None))
    refused(L, ARG, "dh", b(dh=None))
    refused(L, ARG, "null", b(pos=None))
    refused(L, ARG, "h: row stride", b(h=P, hs=31))
    refused(L, ARG, "I=40", b(I=40, ds=40, gu=None, os=80, c=P, s=P))
    refused(L, ARG, "codes", b(gu=None, s=P))
    assert b(M=0) == 0


def test_the_extension_refuses_host_tensors(L):
    t = torch.zeros((4, 64), dtype=torch.bfloat16)
    i = torch.zeros(8, dtype=torch.int32)
    u = torch.zeros((4, 64), dtype=torch.uint8)
    for call in (lambda: chord.chord_expert_gemm(t, t, i, i, t, u), lambda: chord.chord_expert_wgrad(t, t, i, i, t, u),
                 lambda: chord.chord_mxfp8_quantize(t, u, u), lambda: chord.chord_mxfp8_dequantize(u, u, t),
                 lambda: chord.chord_mxfp8_permute(u, u, i, i, i, 2, t), lambda: chord.chord_swiglu(t, t, i, i, t),
                 lambda: chord.chord_swiglu_backward(t, t, None, None, t, i, i, i, t, t)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError, match="torch.Tensor"):
        chord.chord_expert_gemm(None, t, i, i, t, u)
