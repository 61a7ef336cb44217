"""Thin Python binding of libchord_moe.so (ctypes, and a small extension).

Argument marshalling only: every function here checks tensor dtypes and
devices, passes raw device pointers and the current CUDA stream to the C
entry point of the same name, and raises ChordError on a non-zero status.
The rows in expert order and the MXFP4 operators are called from layers that
run a dozen of them per step, so their checks and marshalling are in C++
(csrc_py/binding.cpp, built as _chord.so).  All computation happens in the
library's CUDA kernels; there is no CPU fallback, and a missing library is an
error.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libchord_moe.so")
EXT_PATH = os.path.join(_HERE, "_chord.so")

CHORD_OK = 0
CHORD_ERR_INVALID_ARG = -1
CHORD_ERR_UNSUPPORTED = -2
CHORD_ERR_CUDA = -3
CHORD_ERR_WORKSPACE_TOO_SMALL = -4
CHORD_ERR_PREPACK_MISMATCH = -5
CHORD_ERR_TIMEOUT = -6
CHORD_ERR_ROUTING_INVALID = -7

CHORD_EPI_STORE = 0
CHORD_EPI_SILU_MUL = 1
CHORD_EPI_WEIGHTED_ADD = 2

CHORD_DTYPE_BF16 = 0
CHORD_DTYPE_FP16 = 1
CHORD_DTYPE_FP32 = 2

# what of the experts' product's workspace has to be zero when it is first used
CHORD_EXPERT_GEMM_COUNTER_BYTES = 1024

CHORD_PATH_AUTO = 0
CHORD_PATH_SMALL_M = 1
CHORD_PATH_LARGE_M = 2


class ChordError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"chord error {code}: {msg}")
        self.code = code


class chord_tuning(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("rows_per_pass", ctypes.c_int),
                ("use_f16_accum", ctypes.c_int), ("batch_invariant", ctypes.c_int)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
_L = ctypes.c_int64
_SIGS = {
    "chord_last_error_string": (ctypes.c_char_p, []),
    "chord_version": (_I, []),
    "chord_debug_force_timeout": (_I, [_I]),
    "chord_moe_route": (_I, [_P, _P, _I, _I, _I, _P, _P, _P]),
    "chord_moe_align_capacity": (_Z, [_I, _I, _I, _I]),
    "chord_moe_align_workspace_bytes": (_Z, [_I, _I, _I]),
    "chord_moe_align": (_I, [_P, _I, _I, _I, _I, _I, _Z, _P, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "chord_moe_align_noalloc": (_I, [_P, _I, _I, _I, _I, _I, _Z, _P, _P, _P, _P, _P, _P, _P]),
    "chord_moe_route_align": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _Z, _P, _P, _P, _P, _P, _P, _P, _P,
                                   _P, _Z, _P]),
    "chord_w4a16_prepack_bytes": (_Z, [_I, _I, _I, _I]),
    "chord_w4a16_prepack": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _Z, _P]),
    "chord_w4a16_moe_gemm_workspace_bytes": (_Z, [_Z, _I, _I]),
    "chord_w4a16_moe_gemm": (_I, [_P, _I, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _I, _Z, _I,
                                  _P, _P, _P, _P, _Z, _P, _P]),
    "chord_moe_sum": (_I, [_P, _P, _P, _I, _I, _I, _P, _P]),
    "chord_w4a16_gemm_workspace_bytes": (_Z, [_I]),
    "chord_w4a16_gemm": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _Z, _P, _P]),
    "chord_w4a16_grouped_workspace_bytes": (_Z, [_I, _Z]),
    "chord_w4a16_grouped_gemm_contiguous": (_I, [_P, _Z, _P, _I, _I, _P, _I, _I, _I, _P, _P, _P, _Z,
                                                 _P, _P]),
    "chord_w4a16_grouped_gemm_masked": (_I, [_P, _P, _I, _I, _I, _P, _I, _I, _I, _P, _P, _P, _Z, _P, _P]),
    "chord_moe_layer_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "chord_moe_layer_plan": (_I, [_I, _I, _I, _P]),
    "chord_moe_layer": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _Z,
                             _P, _P, _P]),
    "chord_moe_permute": (_I, [_P, _I, _L, _P, _P, _P, _I, _I, _I, _Z, _P, _L, _P]),
    "chord_moe_permute_backward": (_I, [_P, _I, _L, _P, _I, _I, _I, _Z, _P, _L, _P]),
    "chord_moe_unpermute": (_I, [_P, _I, _L, _P, _P, _I, _I, _I, _Z, _P, _L, _P]),
    "chord_moe_unpermute_backward": (_I, [_P, _P, _I, _L, _L, _P, _P, _P, _P, _I, _I, _I, _Z, _P, _L, _P, _P]),
    "chord_mxfp4_quantize": (_I, [_P, _I, _L, _L, _I, _P, _P, _P]),
    "chord_mxfp4_dequantize": (_I, [_P, _P, _L, _I, _P, _I, _L, _P]),
    "chord_mxfp4_rows_bytes": (_Z, [_Z, _I]),
    "chord_mxfp4_quantize_rows": (_I, [_P, _I, _L, _I, _I, _P, _I, _P, _Z, _P, _Z, _P]),
    "chord_mxfp4_prepack_bytes": (_Z, [_I, _I, _I]),
    "chord_mxfp4_prepack": (_I, [_P, _P, _I, _I, _I, _I, _P, _Z, _P]),
    "chord_mxfp4_moe_gemm_workspace_bytes": (_Z, []),
    "chord_mxfp4_moe_gemm": (_I, [_P, _Z, _P, _I, _I, _I, _P, _P, _Z, _I, _P, _P, _Z, _P, _P]),
    "chord_expert_gemm_workspace_bytes": (_Z, []),
    "chord_expert_gemm": (_I, [_P, _I, _L, _P, _L, _L, _I, _I, _I, _I, _P, _P, _Z, _P, _L, _P, _Z, _P, _P]),
    "chord_mxfp8_quantize": (_I, [_P, _I, _L, _L, _I, _P, _P, _P]),
    "chord_mxfp8_dequantize": (_I, [_P, _P, _L, _I, _P, _I, _L, _P]),
    "chord_mxfp8_permute": (_I, [_P, _P, _P, _P, _I, _I, _I, _Z, _P, _I, _L, _P]),
    "chord_swiglu": (_I, [_P, _I, _L, _P, _P, _P, _I, _I, _I, _Z, _P, _L, _P, _P, _P]),
    "chord_swiglu_backward": (_I, [_P, _I, _L, _P, _L, _P, _P, _P, _P, _P, _P, _I, _I, _I, _Z, _P, _L, _P, _P, _L,
                                   _P]),
    "chord_expert_wgrad": (_I, [_P, _P, _I, _L, _L, _I, _I, _I, _P, _P, _Z, _P, _I, _P, _Z, _P, _P]),
}

_lib = None


def lib():
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "w4a16_int4_weight_sigmoid_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


_ext_module = None


def _ext():
    """Load the extension (once).  Raises if it has not been built."""
    global _ext_module
    if _ext_module is None:
        lib()
        if not os.path.exists(EXT_PATH):
            raise RuntimeError(f"{EXT_PATH} is missing: build it with "
                               "w4a16_int4_weight_sigmoid_gb300.build.build()")
        spec = importlib.util.spec_from_file_location("_chord", EXT_PATH)
        _ext_module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_ext_module)
    return _ext_module


def _check(rc: int):
    if rc != CHORD_OK:
        raise ChordError(rc, lib().chord_last_error_string().decode())


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _check_operands(A, C, K: int, N: int, epilogue: int, a_rows: int, c_rows: int, what: str):
    """Shape and dtype checks the C ABI cannot make (it sees raw pointers):
    A holds a_rows rows of K BF16 values and C holds c_rows rows of N (STORE)
    or N/2 (SiLU*mul) BF16 values.  Raises ValueError before anything runs."""
    for name, t in (("A", A), ("C", C)):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{what}: {name} must be a torch.Tensor")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{what}: {name} must be bfloat16, got {t.dtype}")
    if A.shape[-1] != K:
        raise ValueError(f"{what}: A's last dimension {A.shape[-1]} != K={K}")
    if A.numel() < a_rows * K:
        raise ValueError(f"{what}: A holds {A.numel()} values, needs {a_rows} rows of K={K}")
    ncols = N // 2 if epilogue == CHORD_EPI_SILU_MUL else N
    if C.shape[-1] != ncols:
        raise ValueError(f"{what}: C's last dimension {C.shape[-1]} != {ncols} "
                         f"({'N/2 for SiLU*mul' if epilogue == CHORD_EPI_SILU_MUL else 'N'})")
    if C.numel() < c_rows * ncols:
        raise ValueError(f"{what}: C holds {C.numel()} values, needs {c_rows} rows of {ncols}")


def _check_holds(what: str, *need):
    """Each tensor given as (name, tensor, values) holds at least that many values: the C ABI
    writes or reads them through raw pointers.  Raises ValueError before anything runs."""
    for name, t, n in need:
        if isinstance(t, torch.Tensor) and t.numel() < n:
            raise ValueError(f"{what}: {name} holds {t.numel()} values, needs {n}")


# The current stream's handle without building a torch.cuda.Stream object, which
# takes longer on the host (2.9 us) than the rest of a small call's checks.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _tuning(tuning):
    """None, a chord_tuning, or a path id."""
    if tuning is None:
        return None
    t = tuning if isinstance(tuning, chord_tuning) else chord_tuning(int(tuning), 0, 0, 0)
    return ctypes.byref(t), t


def chord_version() -> int:
    return lib().chord_version()


def chord_debug_force_timeout(enable: bool) -> None:
    """Test hook: later launches of the register-MMA GEMM and of the MXFP4 product withhold
    their work items, so their consumers' waits run out (CHORD_ERR_TIMEOUT, nothing computed)."""
    _check(lib().chord_debug_force_timeout(int(bool(enable))))


def chord_moe_route(logits, bias, topk: int, topk_weights, topk_ids, stream=None):
    M, E = logits.shape
    _check(lib().chord_moe_route(_ptr(logits, torch.float32, "logits"), _ptr(bias, torch.float32, "bias"),
                                 M, E, topk, _ptr(topk_weights, torch.float32, "topk_weights"),
                                 _ptr(topk_ids, torch.int32, "topk_ids"), _stream(stream)))


def chord_moe_align_capacity(M: int, topk: int, E_local: int, block_m: int) -> int:
    return lib().chord_moe_align_capacity(M, topk, E_local, block_m)


def chord_moe_align_workspace_bytes(M: int, topk: int, E_local: int) -> int:
    return lib().chord_moe_align_workspace_bytes(M, topk, E_local)


def chord_moe_align(topk_ids, expert_begin: int, E_local: int, block_m: int, sorted_token_ids,
                    expert_ids, num_tokens_post_padded, expert_counts, expert_offsets,
                    sorted_positions=None, workspace=None, stream=None):
    M, k = topk_ids.shape
    i32 = torch.int32
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().chord_moe_align(
        _ptr(topk_ids, i32, "topk_ids"), M, k, expert_begin, E_local, block_m,
        sorted_token_ids.numel(), _ptr(sorted_token_ids, i32, "sorted_token_ids"),
        _ptr(expert_ids, i32, "expert_ids"), _ptr(num_tokens_post_padded, i32, "ntpp"),
        _ptr(expert_counts, i32, "expert_counts"), _ptr(expert_offsets, i32, "expert_offsets"),
        _ptr(sorted_positions, i32, "sorted_positions"), _ptr(workspace, None, "workspace"),
        ws_bytes, _stream(stream)))


def chord_moe_route_align(logits, bias, topk: int, expert_begin: int, E_local: int, block_m: int,
                          topk_weights, topk_ids, sorted_token_ids, expert_ids, num_tokens_post_padded,
                          expert_counts, expert_offsets, sorted_positions=None, workspace=None,
                          stream=None):
    """chord_moe_route then chord_moe_align in one call (one launch for small M)."""
    M, E_total = logits.shape
    n = M * topk
    _check_holds("chord_moe_route_align", ("bias", bias, E_total), ("topk_weights", topk_weights, n),
                 ("topk_ids", topk_ids, n), ("num_tokens_post_padded", num_tokens_post_padded, 1),
                 ("expert_counts", expert_counts, E_local), ("expert_offsets", expert_offsets, E_local + 1),
                 ("sorted_positions", sorted_positions, n))
    if isinstance(expert_ids, torch.Tensor) and expert_ids.numel() * block_m < sorted_token_ids.numel():
        # fewer blocks than sorted_token_ids has room for: as many as M tokens can fill will do
        blocks = chord_moe_align_capacity(M, topk, E_local, block_m) // max(block_m, 1)
        _check_holds("chord_moe_route_align", ("expert_ids", expert_ids, blocks))
    i32 = torch.int32
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().chord_moe_route_align(
        _ptr(logits, torch.float32, "logits"), _ptr(bias, torch.float32, "bias"), M, E_total, topk,
        expert_begin, E_local, block_m, sorted_token_ids.numel(),
        _ptr(topk_weights, torch.float32, "topk_weights"), _ptr(topk_ids, i32, "topk_ids"),
        _ptr(sorted_token_ids, i32, "sorted_token_ids"), _ptr(expert_ids, i32, "expert_ids"),
        _ptr(num_tokens_post_padded, i32, "ntpp"), _ptr(expert_counts, i32, "expert_counts"),
        _ptr(expert_offsets, i32, "expert_offsets"), _ptr(sorted_positions, i32, "sorted_positions"),
        _ptr(workspace, None, "workspace"), ws_bytes, _stream(stream)))


def chord_moe_align_noalloc(topk_ids, expert_begin: int, E_local: int, block_m: int,
                            sorted_token_ids, expert_ids, num_tokens_post_padded, expert_counts,
                            expert_offsets, sorted_positions=None, stream=None):
    """chord_moe_align without a workspace argument: for callers that cannot
    allocate device memory; its scratch is a static array in the library."""
    M, k = topk_ids.shape
    i32 = torch.int32
    _check(lib().chord_moe_align_noalloc(
        _ptr(topk_ids, i32, "topk_ids"), M, k, expert_begin, E_local, block_m,
        sorted_token_ids.numel(), _ptr(sorted_token_ids, i32, "sorted_token_ids"),
        _ptr(expert_ids, i32, "expert_ids"), _ptr(num_tokens_post_padded, i32, "ntpp"),
        _ptr(expert_counts, i32, "expert_counts"), _ptr(expert_offsets, i32, "expert_offsets"),
        _ptr(sorted_positions, i32, "sorted_positions"), _stream(stream)))


def chord_w4a16_prepack_bytes(E: int, N: int, K: int, group: int = 32) -> int:
    return lib().chord_w4a16_prepack_bytes(E, N, K, group)


def chord_w4a16_prepack(qweight, scales, gate_up: bool, packed, group: int = 32, stream=None):
    E, N, K2 = qweight.shape
    _check(lib().chord_w4a16_prepack(
        _ptr(qweight, torch.uint8, "qweight"), _ptr(scales, None, "scales"), E, N, 2 * K2, group,
        int(gate_up), _ptr(packed, torch.uint8, "packed"), packed.numel(), _stream(stream)))


def chord_w4a16_moe_gemm_workspace_bytes(capacity: int, K: int, a_gather: bool) -> int:
    return lib().chord_w4a16_moe_gemm_workspace_bytes(capacity, K, int(a_gather))


def chord_w4a16_moe_gemm(A, a_gather: bool, packed_w, E_local: int, N: int, K: int, M: int,
                         topk: int, sorted_token_ids, expert_ids, num_tokens_post_padded,
                         expert_counts, expert_offsets, block_m: int, epilogue: int, C, workspace,
                         tuning=None, dev_status=None, stream=None, topk_weights=None):
    """workspace: uint8 tensor of chord_w4a16_moe_gemm_workspace_bytes() bytes, zeroed once
    when allocated (the library keeps its counters zero).  CHORD_EPI_WEIGHTED_ADD: C is a
    float32 [M, N] accumulator the caller initialises, topk_weights float32 [M, topk]."""
    cap = sorted_token_ids.numel()
    if epilogue == CHORD_EPI_WEIGHTED_ADD:
        if not isinstance(C, torch.Tensor) or C.dtype != torch.float32 or C.numel() < M * N:
            raise ValueError("chord_w4a16_moe_gemm: the weighted add needs a float32 C of M x N values")
        if not isinstance(topk_weights, torch.Tensor) or topk_weights.numel() < M * topk:
            raise ValueError("chord_w4a16_moe_gemm: the weighted add needs topk_weights [M, topk]")
        _check_operands(A, A, K, K, CHORD_EPI_STORE, cap, 0, "chord_w4a16_moe_gemm")
    else:
        _check_operands(A, C, K, N, epilogue, M if a_gather else cap, cap, "chord_w4a16_moe_gemm")
    tun = _tuning(tuning)
    _check(lib().chord_w4a16_moe_gemm(
        _ptr(A, None, "A"), int(a_gather), _ptr(packed_w, torch.uint8, "packed_w"), E_local, N, K, M,
        topk, _ptr(sorted_token_ids, torch.int32, "sorted_token_ids"),
        _ptr(expert_ids, torch.int32, "expert_ids"),
        _ptr(num_tokens_post_padded, torch.int32, "num_tokens_post_padded"),
        _ptr(expert_counts, torch.int32, "expert_counts"),
        _ptr(expert_offsets, torch.int32, "expert_offsets"), block_m, sorted_token_ids.numel(),
        epilogue, _ptr(topk_weights, torch.float32, "topk_weights"), _ptr(C, None, "C"),
        tun[0] if tun else None, _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def chord_w4a16_gemm_workspace_bytes(M: int) -> int:
    return lib().chord_w4a16_gemm_workspace_bytes(M)


def chord_w4a16_gemm(A, packed_w, N: int, K: int, epilogue: int, C, workspace, tuning=None,
                     dev_status=None, stream=None):
    """Dense C = A (q*s)^T with a one-expert packed blob; workspace zeroed once when allocated."""
    if A.dim() != 2 or C.dim() != 2 or C.shape[0] != A.shape[0]:
        raise ValueError("chord_w4a16_gemm: A must be [M, K] and C [M, N or N/2] with the same rows")
    _check_operands(A, C, K, N, epilogue, A.shape[0], A.shape[0], "chord_w4a16_gemm")
    tun = _tuning(tuning)
    _check(lib().chord_w4a16_gemm(
        _ptr(A, None, "A"), _ptr(packed_w, torch.uint8, "packed_w"), N, K, A.shape[0], epilogue,
        _ptr(C, None, "C"), tun[0] if tun else None, _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def chord_w4a16_grouped_workspace_bytes(E: int, rows: int) -> int:
    return lib().chord_w4a16_grouped_workspace_bytes(E, rows)


def chord_w4a16_grouped_gemm_contiguous(A, group_rows, packed_w, N: int, K: int, epilogue: int, C, workspace,
                                        expected_m: int = 0, tuning=None, dev_status=None, stream=None):
    """Contiguous layout: A [rows, K], expert groups in order, each padded to 128 rows."""
    if A.dim() != 2:
        raise ValueError("contiguous layout: A must be [rows, K]")
    if C.dim() != 2 or C.shape[0] != A.shape[0]:
        raise ValueError("contiguous layout: C must be [rows, N or N/2] with the rows of A")
    _check_operands(A, C, K, N, epilogue, A.shape[0], A.shape[0], "chord_w4a16_grouped_gemm_contiguous")
    tun = _tuning(tuning)
    _check(lib().chord_w4a16_grouped_gemm_contiguous(
        _ptr(A, None, "A"), A.shape[0], _ptr(group_rows, torch.int32, "group_rows"), group_rows.numel(),
        expected_m, _ptr(packed_w, torch.uint8, "packed_w"), N, K, epilogue, _ptr(C, None, "C"),
        tun[0] if tun else None, _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def chord_w4a16_grouped_gemm_masked(A, group_rows, packed_w, N: int, K: int, epilogue: int, C, workspace,
                                    expected_m: int = 0, tuning=None, dev_status=None, stream=None):
    """Masked layout: A [E, max_m, K], the first group_rows[e] rows of expert e are used."""
    if A.dim() != 3 or group_rows.numel() != A.shape[0]:
        raise ValueError("masked layout: A must be [E, max_m, K] with one group_rows entry per expert")
    if C.dim() != 3 or C.shape[:2] != A.shape[:2]:
        raise ValueError("masked layout: C must be [E, max_m, N or N/2] with the experts and rows of A")
    _check_operands(A, C, K, N, epilogue, A.shape[0] * A.shape[1], A.shape[0] * A.shape[1],
                    "chord_w4a16_grouped_gemm_masked")
    tun = _tuning(tuning)
    _check(lib().chord_w4a16_grouped_gemm_masked(
        _ptr(A, None, "A"), _ptr(group_rows, torch.int32, "group_rows"), A.shape[0], A.shape[1], expected_m,
        _ptr(packed_w, torch.uint8, "packed_w"), N, K, epilogue, _ptr(C, None, "C"),
        tun[0] if tun else None, _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream)))


def chord_moe_sum(y, topk_weights, sorted_positions, out, stream=None):
    M, k = topk_weights.shape
    H = out.shape[1]
    _check(lib().chord_moe_sum(_ptr(y, None, "y"), _ptr(topk_weights, torch.float32, "topk_weights"),
                               _ptr(sorted_positions, torch.int32, "sorted_positions"), M, k, H,
                               _ptr(out, None, "out"), _stream(stream)))


def chord_moe_layer_workspace_bytes(M: int, H: int, I: int, E_local: int, topk: int) -> int:
    return lib().chord_moe_layer_workspace_bytes(M, H, I, E_local, topk)


def chord_moe_layer_plan(M: int, E_total: int, topk: int) -> chord_tuning:
    plan = chord_tuning()
    _check(lib().chord_moe_layer_plan(M, E_total, topk, ctypes.byref(plan)))
    return plan


def chord_moe_layer(x, logits, bias, w13_packed, w2_packed, H: int, I: int, E_total: int,
                    expert_begin: int, E_local: int, topk: int, out, workspace,
                    topk_weights_out=None, topk_ids_out=None, tuning=None, dev_status=None,
                    stream=None):
    M = x.shape[0]
    tun = _tuning(tuning)
    _check(lib().chord_moe_layer(
        _ptr(x, None, "x"), _ptr(logits, torch.float32, "logits"), _ptr(bias, torch.float32, "bias"),
        _ptr(w13_packed, torch.uint8, "w13_packed"), _ptr(w2_packed, torch.uint8, "w2_packed"),
        M, H, I, E_total, expert_begin, E_local, topk, _ptr(out, None, "out"),
        _ptr(topk_weights_out, torch.float32, "topk_weights_out"),
        _ptr(topk_ids_out, torch.int32, "topk_ids_out"), _ptr(workspace, torch.uint8, "workspace"),
        workspace.numel(), tun[0] if tun else None, _ptr(dev_status, torch.int32, "dev_status"),
        _stream(stream)))


# ------------------------------------------- rows in expert order, and MXFP4
# Row matrices are 2-D with unit column stride and any row stride.

def chord_moe_permute(x, sorted_positions, sorted_token_ids, num_tokens_post_padded, topk: int, out, stream=None):
    """out[p(t, j)] = x[t] for every local assignment; padding rows become zeros.
    x [M, H], out [capacity, H] of one type (BF16, FP16, FP32), any row strides."""
    rc = (_ext_module or _ext()).permute(x, sorted_positions, sorted_token_ids, num_tokens_post_padded, topk, out,
                                         None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_moe_permute_backward(dout, sorted_positions, topk: int, dx, stream=None):
    """dx[t] = sum over the local assignments of dout[p(t, j)].  dout [capacity, H], dx [M, H]."""
    rc = (_ext_module or _ext()).permute_backward(dout, sorted_positions, topk, dx,
                                                  None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_moe_unpermute(y, topk_weights, sorted_positions, out, stream=None):
    """out[t] = sum over the local assignments of topk_weights[t, j] * y[p(t, j)].
    y [capacity, H], topk_weights FP32 [M, topk], out [M, H]."""
    rc = (_ext_module or _ext()).unpermute(y, topk_weights, sorted_positions, out,
                                           None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_moe_unpermute_backward(dout, y, topk_weights, sorted_positions, sorted_token_ids, num_tokens_post_padded,
                                 dy, dweights, stream=None):
    """dy[p(t, j)] = topk_weights[t, j] * dout[t], padding rows zeros; dweights[t, j] = <dout[t], y[p(t, j)]>."""
    rc = (_ext_module or _ext()).unpermute_backward(dout, y, topk_weights, sorted_positions, sorted_token_ids,
                                                    num_tokens_post_padded, dy, dweights,
                                                    None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_mxfp4_quantize(x, codes, scales, stream=None):
    """x [rows, K] (BF16, FP16, FP32) -> codes uint8 [rows, K/2], scales uint8 [rows, K/32]."""
    rc = (_ext_module or _ext()).quantize(x, codes, scales, None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_mxfp4_dequantize(codes, scales, out, stream=None):
    """The values of codes and scales, out [rows, K] (BF16, FP16, FP32)."""
    rc = (_ext_module or _ext()).dequantize(codes, scales, out, None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_mxfp4_rows_bytes(capacity: int, K: int) -> int:
    return lib().chord_mxfp4_rows_bytes(capacity, K)


def chord_mxfp4_quantize_rows(x, sorted_positions, topk: int, num_tokens_post_padded, capacity: int, rows,
                              stream=None):
    """Token rows x [M, K] quantised into the product's row operand `rows` (uint8,
    chord_mxfp4_rows_bytes(capacity, K)): token t to its rows sorted_positions[t, :]; with
    sorted_positions None, row r of x to row r below num_tokens_post_padded (topk unused)."""
    rc = (_ext_module or _ext()).quantize_rows(x, sorted_positions, topk, num_tokens_post_padded, capacity, rows,
                                               None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_mxfp4_prepack_bytes(E: int, N: int, K: int) -> int:
    return lib().chord_mxfp4_prepack_bytes(E, N, K)


def chord_mxfp4_prepack(codes, scales, gate_up: bool, packed, stream=None):
    """codes uint8 [E, N, K/2] and scales uint8 [E, N, K/32] -> the product's weight operand."""
    E, N, K2 = codes.shape
    if scales.numel() != E * N * K2 // 16:
        raise ValueError(f"scales must hold {E * N * K2 // 16} values")
    _check(lib().chord_mxfp4_prepack(_ptr(codes, torch.uint8, "codes"), _ptr(scales, torch.uint8, "scales"), E, N,
                                     2 * K2, int(gate_up), _ptr(packed, torch.uint8, "packed"), packed.numel(),
                                     _stream(stream)))


def chord_mxfp4_moe_gemm_workspace_bytes() -> int:
    return lib().chord_mxfp4_moe_gemm_workspace_bytes()


def chord_mxfp4_moe_gemm(rows, packed_w, E_local: int, N: int, K: int, expert_counts, expert_offsets, capacity: int,
                         epilogue: int, C, workspace, dev_status=None, stream=None):
    """C [capacity, N or N/2] BF16 = the experts' product of the quantised rows; workspace: uint8 tensor of
    chord_mxfp4_moe_gemm_workspace_bytes() bytes, zeroed once when allocated."""
    rc = (_ext_module or _ext()).moe_gemm(rows, packed_w, E_local, N, K, expert_counts, expert_offsets, capacity,
                                          epilogue, C, workspace, dev_status,
                                          None if stream is None else _stream(stream))
    if rc:
        _check(rc)

# --------------------------------------- the experts' product in 16 bits

def chord_expert_gemm_workspace_bytes() -> int:
    return lib().chord_expert_gemm_workspace_bytes()


def chord_expert_gemm(x, w, expert_counts, expert_offsets, out, workspace, transpose_w: bool = False, dev_status=None,
                      stream=None):
    """out[r] = w[e] @ x[r] (transpose_w: w[e].T @ x[r]) for every expert e's rows r.  x and out are rows in expert
    order, w [E, N, K], all BF16 or FP16; workspace: uint8 tensor of chord_expert_gemm_workspace_bytes() bytes,
    its first CHORD_EXPERT_GEMM_COUNTER_BYTES zeroed once when allocated."""
    rc = (_ext_module or _ext()).expert_gemm(x, w, expert_counts, expert_offsets, out, workspace, int(transpose_w),
                                             dev_status, None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_expert_wgrad(dout, x, expert_counts, expert_offsets, dw, workspace, dev_status=None, stream=None):
    """dw[e] = dout[rows of e].T @ x[rows of e], zeros for an expert without rows.  dout [capacity, N] and
    x [capacity, K] of one type (BF16, FP16), dw contiguous [E, N, K] of that type or FP32."""
    rc = (_ext_module or _ext()).expert_wgrad(dout, x, expert_counts, expert_offsets, dw, workspace, dev_status,
                                              None if stream is None else _stream(stream))
    if rc:
        _check(rc)


# ------------------------------- rows in 8 bits, and the gated activation

def chord_mxfp8_quantize(x, codes, scales, stream=None):
    """x [rows, K] (BF16, FP16, FP32) -> codes uint8 [rows, K], scales uint8 [rows, K/32]."""
    rc = (_ext_module or _ext()).mxfp8_quantize(x, codes, scales, None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_mxfp8_dequantize(codes, scales, out, stream=None):
    """The values of codes and scales, out [rows, K] (BF16, FP16, FP32)."""
    rc = (_ext_module or _ext()).mxfp8_dequantize(codes, scales, out, None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_mxfp8_permute(codes, scales, sorted_positions, sorted_token_ids, num_tokens_post_padded, topk: int, out,
                        stream=None):
    """The values of token rows codes [M, K] and scales into the aligned expert order, out [capacity, K];
    padding rows become zeros.  (Of sorted_positions [M * topk] only the size is used.)"""
    rc = (_ext_module or _ext()).mxfp8_permute(codes, scales, sorted_positions, sorted_token_ids,
                                               num_tokens_post_padded, topk, out,
                                               None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_swiglu(gu, topk_weights, sorted_token_ids, num_tokens_post_padded, h, codes=None, scales=None, stream=None):
    """h[r] = w silu(gu[r, :I]) gu[r, I:] with the routing weight w of row r's assignment, padding rows zeros.
    gu [capacity, 2I], topk_weights FP32 [M, topk], h [capacity, I] of gu's type.  With codes uint8
    [capacity, 2I] and scales uint8 [capacity, 2I/32], gu is held there in 8 bits."""
    rc = (_ext_module or _ext()).swiglu(gu, topk_weights, sorted_token_ids, num_tokens_post_padded, h, codes, scales,
                                        None if stream is None else _stream(stream))
    if rc:
        _check(rc)


def chord_swiglu_backward(dh, gu, codes, scales, topk_weights, sorted_positions, sorted_token_ids,
                          num_tokens_post_padded, dgu, dweights, h=None, stream=None):
    """The gradients of chord_swiglu: dgu [capacity, 2I] and dweights FP32 [M, topk] from dh [capacity, I] and gu, or
    (gu None) its codes and scales; h [capacity, I]: the forward pass's rows again, of what gu or its codes hold."""
    rc = (_ext_module or _ext()).swiglu_backward(dh, gu, codes, scales, topk_weights, sorted_positions,
                                                 sorted_token_ids, num_tokens_post_padded, dgu, dweights, h,
                                                 None if stream is None else _stream(stream))
    if rc:
        _check(rc)
