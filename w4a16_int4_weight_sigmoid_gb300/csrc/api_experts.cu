// C ABI of the expert-order rows and the MXFP4 operators: argument checks and
// launches.  No entry point allocates memory or synchronises.
#include "api_util.h"
#include "chord_moe.h"
#include "elem.cuh"
#include "kernels.h"

using chord::aligned16;
using chord::cuda_fail;
using chord::fail;

namespace {

cudaStream_t stream_of(void* s) { return static_cast<cudaStream_t>(s); }

int done(cudaError_t e, const char* what) { return e == cudaSuccess ? CHORD_OK : cuda_fail(e, what); }

// The sizes that the row operators share.
int check_rows(int dtype, int M, int topk, int H, size_t capacity) {
  if (!chord::dtype_bytes(dtype)) return fail(CHORD_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (M < 0 || topk < 1 || topk > 32) return fail(CHORD_ERR_INVALID_ARG, "bad M=%d or topk=%d (1 <= topk <= 32)", M, topk);
  if (static_cast<long long>(M) * topk > (1LL << 30)) return fail(CHORD_ERR_INVALID_ARG, "M*topk too large");
  if (H < 1 || H > (1 << 24)) return fail(CHORD_ERR_INVALID_ARG, "row length %d not in [1, 2^24]", H);
  if (capacity > (1u << 30)) return fail(CHORD_ERR_INVALID_ARG, "%zu rows: too many", capacity);
  return CHORD_OK;
}

// One matrix of rows: element-aligned base; a row that is written does not
// overlap the next one (a row that is read may, also with stride 0).
int check_matrix(const char* name, const void* p, int dtype, long long stride, int H, bool written) {
  if (!p) return fail(CHORD_ERR_INVALID_ARG, "null pointer: %s", name);
  if (reinterpret_cast<uintptr_t>(p) % chord::dtype_bytes(dtype))
    return fail(CHORD_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  if (stride < (written ? H : 0))
    return fail(CHORD_ERR_INVALID_ARG, "%s: row stride %lld is too small for rows of %d", name, stride, H);
  return CHORD_OK;
}

int check_mx(const char* what, int K) {
  if (K < 1 || K % 32 != 0 || K > (1 << 24))
    return fail(CHORD_ERR_INVALID_ARG, "%s: K=%d must be a positive multiple of 32 up to 2^24", what, K);
  return CHORD_OK;
}

int check_codes(const uint8_t* codes, const uint8_t* scales) {
  if (!codes || !scales) return fail(CHORD_ERR_INVALID_ARG, "null pointer: codes or scales");
  if (!aligned16(codes)) return fail(CHORD_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  return CHORD_OK;
}

// The sizes and buffers that the 16-bit products share.
int check_product(int dtype, int E, int N, int K, const int32_t* counts, const int32_t* offsets, size_t capacity,
                  const void* ws, size_t ws_bytes) {
  if (dtype != CHORD_DTYPE_BF16 && dtype != CHORD_DTYPE_FP16)
    return fail(CHORD_ERR_INVALID_ARG, "dtype %d: the experts' 16-bit product takes BF16 and FP16", dtype);
  if (E < 1 || E > 1024) return fail(CHORD_ERR_INVALID_ARG, "E_local=%d not in [1, 1024]", E);
  if (N < 8 || N % 8 != 0 || N > (1 << 20) || K < 8 || K % 8 != 0 || K > (1 << 20))
    return fail(CHORD_ERR_INVALID_ARG, "N=%d and K=%d must be positive multiples of 8 up to 2^20", N, K);
  if (capacity > (1u << 30)) return fail(CHORD_ERR_INVALID_ARG, "%zu rows: too many", capacity);
  if (!counts || !offsets) return fail(CHORD_ERR_INVALID_ARG, "null pointer: expert_counts or expert_offsets");
  const size_t need = chord::expert_gemm_workspace_bytes();
  if (!ws || ws_bytes < need)
    return fail(CHORD_ERR_WORKSPACE_TOO_SMALL, "expert product workspace %zu < required %zu", ws_bytes, need);
  if (!aligned16(ws)) return fail(CHORD_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return CHORD_OK;
}
// A matrix that the products read or write in 16-byte parts, rows disjoint
// (the stride of a single row means nothing).
int check_rows16(const char* name, const void* p, int64_t& stride, int width, size_t rows) {
  if (rows == 1) stride = width;
  if (!p) return fail(CHORD_ERR_INVALID_ARG, "null pointer: %s", name);
  if (!aligned16(p)) return fail(CHORD_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (stride < width || stride % 8 != 0 || stride > (1LL << 36))
    return fail(CHORD_ERR_INVALID_ARG, "%s: row stride %lld must be a multiple of 8 from %d to 2^36", name,
                (long long)stride, width);
  return CHORD_OK;
}

}  // namespace

extern "C" {

int chord_moe_permute(const void* x, int dtype, int64_t x_stride, const int32_t* sorted_positions,
                      const int32_t* sorted_token_ids, const int32_t* num_tokens_post_padded, int M, int topk, int H,
                      size_t capacity, void* out, int64_t out_stride, void* stream) {
  int rc = check_rows(dtype, M, topk, H, capacity);
  if (rc || M == 0 || capacity == 0) return rc;
  if ((rc = check_matrix("x", x, dtype, x_stride, H, false))) return rc;
  if ((rc = check_matrix("out", out, dtype, out_stride, H, true))) return rc;
  if (!sorted_positions || !sorted_token_ids || !num_tokens_post_padded)
    return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  return done(chord::moe_permute_launch(x, dtype, x_stride, sorted_positions, sorted_token_ids, num_tokens_post_padded,
                                        M, topk, H, static_cast<int>(capacity), out, out_stride, stream_of(stream)),
              "permute launch");
}

int chord_moe_permute_backward(const void* dout, int dtype, int64_t dout_stride, const int32_t* sorted_positions, int M,
                               int topk, int H, size_t capacity, void* dx, int64_t dx_stride, void* stream) {
  int rc = check_rows(dtype, M, topk, H, capacity);
  if (rc || M == 0) return rc;
  if ((rc = check_matrix("dout", dout, dtype, dout_stride, H, false))) return rc;
  if ((rc = check_matrix("dx", dx, dtype, dx_stride, H, true))) return rc;
  if (!sorted_positions) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  return done(chord::moe_combine_launch(dout, dtype, dout_stride, nullptr, sorted_positions, M, topk, H,
                                        static_cast<int>(capacity), dx, dx_stride, stream_of(stream)),
              "permute_backward launch");
}

int chord_moe_unpermute(const void* y, int dtype, int64_t y_stride, const float* topk_weights,
                        const int32_t* sorted_positions, int M, int topk, int H, size_t capacity, void* out,
                        int64_t out_stride, void* stream) {
  int rc = check_rows(dtype, M, topk, H, capacity);
  if (rc || M == 0) return rc;
  if ((rc = check_matrix("y", y, dtype, y_stride, H, false))) return rc;
  if ((rc = check_matrix("out", out, dtype, out_stride, H, true))) return rc;
  if (!topk_weights || !sorted_positions) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  return done(chord::moe_combine_launch(y, dtype, y_stride, topk_weights, sorted_positions, M, topk, H,
                                        static_cast<int>(capacity), out, out_stride, stream_of(stream)),
              "unpermute launch");
}

int chord_moe_unpermute_backward(const void* dout, const void* y, int dtype, int64_t dout_stride, int64_t y_stride,
                                 const float* topk_weights, const int32_t* sorted_positions,
                                 const int32_t* sorted_token_ids, const int32_t* num_tokens_post_padded, int M,
                                 int topk, int H, size_t capacity, void* dy, int64_t dy_stride, float* dweights,
                                 void* stream) {
  int rc = check_rows(dtype, M, topk, H, capacity);
  if (rc || M == 0) return rc;
  if ((rc = check_matrix("dout", dout, dtype, dout_stride, H, false))) return rc;
  if ((rc = check_matrix("y", y, dtype, y_stride, H, false))) return rc;
  if ((rc = check_matrix("dy", dy, dtype, dy_stride, H, true))) return rc;
  if (!topk_weights || !sorted_positions || !sorted_token_ids || !num_tokens_post_padded || !dweights)
    return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  return done(chord::moe_unpermute_backward_launch(dout, y, dtype, dout_stride, y_stride, topk_weights,
                                                   sorted_positions, sorted_token_ids, num_tokens_post_padded, M, topk,
                                                   H, static_cast<int>(capacity), dy, dy_stride, dweights,
                                                   stream_of(stream)),
              "unpermute_backward launch");
}

int chord_mxfp4_quantize(const void* x, int dtype, int64_t x_stride, int64_t rows, int K, uint8_t* codes,
                         uint8_t* scales, void* stream) {
  if (!chord::dtype_bytes(dtype)) return fail(CHORD_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (rows < 0) return fail(CHORD_ERR_INVALID_ARG, "rows < 0");
  int rc = check_mx("quantize", K);
  if (rc || rows == 0) return rc;
  if ((rc = check_matrix("x", x, dtype, x_stride, K, false))) return rc;
  if (!codes || !scales) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(codes)) return fail(CHORD_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  return done(chord::mxfp4_quantize_launch(x, dtype, x_stride, rows, K, codes, scales, stream_of(stream)),
              "quantize launch");
}

int chord_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, void* out, int dtype,
                           int64_t out_stride, void* stream) {
  if (!chord::dtype_bytes(dtype)) return fail(CHORD_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (rows < 0) return fail(CHORD_ERR_INVALID_ARG, "rows < 0");
  int rc = check_mx("dequantize", K);
  if (rc || rows == 0) return rc;
  if ((rc = check_matrix("out", out, dtype, out_stride, K, true))) return rc;
  if (!codes || !scales) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(codes)) return fail(CHORD_ERR_INVALID_ARG, "codes must be 16-byte aligned");
  return done(chord::mxfp4_dequantize_launch(codes, scales, rows, K, out, dtype, out_stride, stream_of(stream)),
              "dequantize launch");
}

size_t chord_mxfp4_rows_bytes(size_t capacity, int K) {
  if (K < 1 || K % 32 != 0) return 0;
  return chord::mxfp4_rows_bytes(capacity, K);
}

int chord_mxfp4_quantize_rows(const void* x, int dtype, int64_t x_stride, int M, int K,
                              const int32_t* sorted_positions, int topk, const int32_t* num_tokens_post_padded,
                              size_t capacity, void* rows, size_t rows_bytes, void* stream) {
  if (!sorted_positions) topk = 1;   // row r of x is row r of the order
  int rc = check_rows(dtype, M, topk, K, capacity);
  if (rc) return rc;
  if ((rc = check_mx("quantize_rows", K))) return rc;
  if (M == 0 || capacity == 0) return CHORD_OK;
  if ((rc = check_matrix("x", x, dtype, x_stride, K, false))) return rc;
  if (!rows || (!sorted_positions && !num_tokens_post_padded)) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(rows)) return fail(CHORD_ERR_INVALID_ARG, "rows must be 16-byte aligned");
  const size_t need = chord::mxfp4_rows_bytes(capacity, K);
  if (rows_bytes < need) return fail(CHORD_ERR_INVALID_ARG, "rows: %zu bytes < required %zu", rows_bytes, need);
  return done(chord::mxfp4_quantize_rows_launch(x, dtype, x_stride, M, K, sorted_positions, topk,
                                                num_tokens_post_padded, static_cast<int>(capacity),
                                                static_cast<uint8_t*>(rows), stream_of(stream)),
              "quantize_rows launch");
}

size_t chord_mxfp4_prepack_bytes(int E, int N, int K) {
  if (E < 1 || N < 1 || N % 8 != 0 || K < 1 || K % 32 != 0) return 0;
  return chord::mxfp4_prepack_bytes(E, N, K);
}

int chord_mxfp4_prepack(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, int gate_up, void* packed,
                        size_t packed_bytes, void* stream) {
  if (E < 1) return fail(CHORD_ERR_INVALID_ARG, "E=%d < 1", E);
  if (N < 1 || N % 8 != 0) return fail(CHORD_ERR_INVALID_ARG, "N=%d must be a positive multiple of 8", N);
  if (gate_up && N % 16 != 0) return fail(CHORD_ERR_INVALID_ARG, "gate_up needs N %% 16 == 0 (N=%d)", N);
  int rc = check_mx("prepack", K);
  if (rc) return rc;
  if (!codes || !scales || !packed) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(codes) || !aligned16(packed)) return fail(CHORD_ERR_INVALID_ARG, "codes and packed must be 16-byte aligned");
  const size_t need = chord::mxfp4_prepack_bytes(E, N, K);
  if (packed_bytes < need) return fail(CHORD_ERR_INVALID_ARG, "packed_bytes %zu < required %zu", packed_bytes, need);
  return done(chord::mxfp4_prepack_launch(codes, scales, E, N, K, gate_up != 0, static_cast<uint8_t*>(packed),
                                          stream_of(stream)),
              "prepack launch");
}

size_t chord_mxfp4_moe_gemm_workspace_bytes(void) { return chord::mxfp4_gemm_workspace_bytes(); }

int chord_mxfp4_moe_gemm(const void* rows, size_t rows_bytes, const void* packed_w, int E_local, int N, int K,
                         const int32_t* expert_counts, const int32_t* expert_offsets, size_t capacity, int epilogue,
                         chord_bf16* C, void* workspace, size_t ws_bytes, int* dev_status, void* stream) {
  if (E_local < 1 || E_local > 1024) return fail(CHORD_ERR_INVALID_ARG, "E_local=%d not in [1, 1024]", E_local);
  if (N < 1 || N % 8 != 0) return fail(CHORD_ERR_INVALID_ARG, "N=%d must be a positive multiple of 8", N);
  int rc = check_mx("product", K);
  if (rc) return rc;
  if (epilogue != CHORD_EPI_STORE && epilogue != CHORD_EPI_SILU_MUL)
    return fail(CHORD_ERR_INVALID_ARG, "epilogue %d: the MXFP4 product stores or applies SiLU*mul", epilogue);
  if (epilogue == CHORD_EPI_SILU_MUL && N % 16 != 0)
    return fail(CHORD_ERR_INVALID_ARG, "SiLU*mul needs N %% 16 == 0 (N=%d)", N);
  if (capacity > (1u << 30)) return fail(CHORD_ERR_INVALID_ARG, "%zu rows: too many", capacity);
  // item and unit counts fit 32 bits with room
  if ((capacity / 16 + E_local) * (static_cast<size_t>(N) / 256 + 1) > (1u << 30))
    return fail(CHORD_ERR_INVALID_ARG, "%zu rows x N=%d: too large", capacity, N);
  if (capacity == 0) return CHORD_OK;
  if (!rows || !packed_w || !expert_counts || !expert_offsets || !C) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(rows) || !aligned16(packed_w) || !aligned16(C))
    return fail(CHORD_ERR_INVALID_ARG, "rows, packed_w and C must be 16-byte aligned");
  const size_t need = chord::mxfp4_rows_bytes(capacity, K);
  if (rows_bytes < need) return fail(CHORD_ERR_INVALID_ARG, "rows: %zu bytes < required %zu", rows_bytes, need);
  const size_t wneed = chord::mxfp4_gemm_workspace_bytes();
  if (!workspace || ws_bytes < wneed)
    return fail(CHORD_ERR_WORKSPACE_TOO_SMALL, "MXFP4 product workspace %zu < required %zu", ws_bytes, wneed);
  if (!aligned16(workspace)) return fail(CHORD_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  return done(chord::mxfp4_gemm_launch(static_cast<const uint8_t*>(rows), static_cast<const uint8_t*>(packed_w), E_local,
                                       N, K, expert_counts, expert_offsets, static_cast<int>(capacity),
                                       epilogue == CHORD_EPI_SILU_MUL, C, workspace, chord::force_timeout(), dev_status,
                                       stream_of(stream)),
              "MXFP4 product launch");
}

size_t chord_expert_gemm_workspace_bytes(void) { return chord::expert_gemm_workspace_bytes(); }

int chord_expert_gemm(const void* x, int dtype, int64_t x_stride, const void* w, int64_t w_stride,
                      int64_t w_expert_stride, int E_local, int N, int K, int transpose_w,
                      const int32_t* expert_counts, const int32_t* expert_offsets, size_t capacity, void* out,
                      int64_t out_stride, void* workspace, size_t ws_bytes, int* dev_status, void* stream) {
  int rc = check_product(dtype, E_local, N, K, expert_counts, expert_offsets, capacity, workspace, ws_bytes);
  if (rc) return rc;
  // item counts fit 32 bits with room
  if ((capacity / 256 + E_local) * static_cast<size_t>((transpose_w ? K : N) / 256 + 1) > (1u << 30))
    return fail(CHORD_ERR_INVALID_ARG, "%zu rows x N=%d, K=%d: too large", capacity, N, K);
  if (capacity == 0) return CHORD_OK;
  if ((rc = check_rows16("x", x, x_stride, transpose_w ? N : K, capacity))) return rc;
  if ((rc = check_rows16("w", w, w_stride, K, N))) return rc;
  if ((rc = check_rows16("out", out, out_stride, transpose_w ? K : N, capacity))) return rc;
  if (E_local == 1) w_expert_stride = w_stride * N;   // not used
  if (w_expert_stride < 8 || w_expert_stride % 8 != 0 || w_expert_stride > (1LL << 38))
    return fail(CHORD_ERR_INVALID_ARG, "w: expert stride %lld must be a multiple of 8 from 8 to 2^38",
                (long long)w_expert_stride);
  chord::ExpertGemm g{};
  g.x = x, g.ldx = x_stride, g.w = w, g.ldw = w_stride, g.expert_stride = w_expert_stride;
  g.f16 = dtype == CHORD_DTYPE_FP16, g.transposed = transpose_w != 0;
  g.counts = expert_counts, g.offsets = expert_offsets;
  g.E = E_local, g.N = N, g.K = K, g.capacity = static_cast<int>(capacity);
  g.out = out, g.ldo = out_stride, g.ws = workspace, g.test_timeout = chord::force_timeout(), g.status = dev_status;
  return done(chord::expert_gemm_launch(g, stream_of(stream)), "expert product launch");
}

int chord_expert_wgrad(const void* dout, const void* x, int dtype, int64_t dout_stride, int64_t x_stride, int E_local,
                       int N, int K, const int32_t* expert_counts, const int32_t* expert_offsets, size_t capacity,
                       void* dw, int dw_dtype, void* workspace, size_t ws_bytes, int* dev_status, void* stream) {
  int rc = check_product(dtype, E_local, N, K, expert_counts, expert_offsets, capacity, workspace, ws_bytes);
  if (rc) return rc;
  if (dw_dtype != dtype && dw_dtype != CHORD_DTYPE_FP32)
    return fail(CHORD_ERR_INVALID_ARG, "dw_dtype %d must be dtype or FP32", dw_dtype);
  const size_t tiles = (static_cast<size_t>(N) / 256 + 1) * (K / 256 + 1);
  if (tiles * E_local > (1u << 30)) return fail(CHORD_ERR_INVALID_ARG, "%d experts x N=%d, K=%d: too large", E_local, N, K);
  if (!dw) return fail(CHORD_ERR_INVALID_ARG, "null pointer: dw");
  if (!aligned16(dw)) return fail(CHORD_ERR_INVALID_ARG, "dw must be 16-byte aligned");
  if (capacity == 0)
    return done(cudaMemsetAsync(dw, 0, static_cast<size_t>(E_local) * N * K * chord::dtype_bytes(dw_dtype),
                                stream_of(stream)),
                "weight gradient of no rows");
  if ((rc = check_rows16("dout", dout, dout_stride, N, capacity))) return rc;
  if ((rc = check_rows16("x", x, x_stride, K, capacity))) return rc;
  chord::ExpertWgrad g{};
  g.dout = dout, g.ldd = dout_stride, g.x = x, g.ldx = x_stride;
  g.f16 = dtype == CHORD_DTYPE_FP16, g.f32 = dw_dtype == CHORD_DTYPE_FP32;
  g.counts = expert_counts, g.offsets = expert_offsets;
  g.E = E_local, g.N = N, g.K = K, g.capacity = static_cast<int>(capacity);
  g.dw = dw, g.ws = workspace, g.test_timeout = chord::force_timeout(), g.status = dev_status;
  return done(chord::expert_wgrad_launch(g, stream_of(stream)), "weight gradient launch");
}

int chord_mxfp8_quantize(const void* x, int dtype, int64_t x_stride, int64_t rows, int K, uint8_t* codes,
                         uint8_t* scales, void* stream) {
  if (!chord::dtype_bytes(dtype)) return fail(CHORD_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (rows < 0) return fail(CHORD_ERR_INVALID_ARG, "rows < 0");
  int rc = check_mx("quantize", K);
  if (rc || rows == 0) return rc;
  if ((rc = check_matrix("x", x, dtype, x_stride, K, false))) return rc;
  if ((rc = check_codes(codes, scales))) return rc;
  return done(chord::mxfp8_quantize_launch(x, dtype, x_stride, rows, K, codes, scales, stream_of(stream)),
              "quantize launch");
}

int chord_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int K, void* out, int dtype,
                           int64_t out_stride, void* stream) {
  if (!chord::dtype_bytes(dtype)) return fail(CHORD_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (rows < 0) return fail(CHORD_ERR_INVALID_ARG, "rows < 0");
  int rc = check_mx("dequantize", K);
  if (rc || rows == 0) return rc;
  if ((rc = check_matrix("out", out, dtype, out_stride, K, true))) return rc;
  if ((rc = check_codes(codes, scales))) return rc;
  return done(chord::mxfp8_dequantize_launch(codes, scales, rows, K, out, dtype, out_stride, stream_of(stream)),
              "dequantize launch");
}

int chord_mxfp8_permute(const uint8_t* codes, const uint8_t* scales, const int32_t* sorted_token_ids,
                        const int32_t* num_tokens_post_padded, int M, int topk, int K, size_t capacity, void* out,
                        int dtype, int64_t out_stride, void* stream) {
  int rc = check_rows(dtype, M, topk, K, capacity);
  if (rc) return rc;
  if ((rc = check_mx("permute", K))) return rc;
  if (M == 0 || capacity == 0) return CHORD_OK;
  if ((rc = check_matrix("out", out, dtype, out_stride, K, true))) return rc;
  if ((rc = check_codes(codes, scales))) return rc;
  if (!sorted_token_ids || !num_tokens_post_padded) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  return done(chord::mxfp8_permute_launch(codes, scales, K, sorted_token_ids, num_tokens_post_padded, M, topk,
                                          static_cast<int>(capacity), out, dtype, out_stride, stream_of(stream)),
              "permute launch");
}

int chord_swiglu(const void* gu, int dtype, int64_t gu_stride, const float* topk_weights,
                 const int32_t* sorted_token_ids, const int32_t* num_tokens_post_padded, int M, int topk, int I,
                 size_t capacity, void* h, int64_t h_stride, uint8_t* codes, uint8_t* scales, void* stream) {
  int rc = check_rows(dtype, M, topk, I, capacity);
  if (rc) return rc;
  if (I > (1 << 23)) return fail(CHORD_ERR_INVALID_ARG, "I=%d > 2^23", I);
  const bool keep = codes || scales;
  if (keep && I % 32 != 0) return fail(CHORD_ERR_INVALID_ARG, "I=%d must be a multiple of 32 to be held in 8 bits", I);
  if (M == 0 || capacity == 0) return CHORD_OK;
  if ((rc = check_matrix("gu", gu, dtype, gu_stride, 2 * I, false))) return rc;
  if ((rc = check_matrix("h", h, dtype, h_stride, I, true))) return rc;
  if (keep && (rc = check_codes(codes, scales))) return rc;
  if (!topk_weights || !sorted_token_ids || !num_tokens_post_padded) return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  chord::Swiglu s{};
  s.gu = gu, s.w = topk_weights, s.sorted = sorted_token_ids, s.ntpp = num_tokens_post_padded;
  s.h = h, s.codes = codes, s.scales = scales, s.ldg = gu_stride, s.ldh = h_stride;
  s.rows = static_cast<int>(capacity), s.I = I, s.assignments = M * topk;
  return done(chord::swiglu_launch(s, dtype, false, stream_of(stream)), "swiglu launch");
}

int chord_swiglu_backward(const void* dh, int dtype, int64_t dh_stride, const void* gu, int64_t gu_stride,
                          const uint8_t* codes, const uint8_t* scales, const float* topk_weights,
                          const int32_t* sorted_positions, const int32_t* sorted_token_ids,
                          const int32_t* num_tokens_post_padded, int M, int topk, int I, size_t capacity, void* dgu,
                          int64_t dgu_stride, float* dweights, void* h, int64_t h_stride, void* stream) {
  int rc = check_rows(dtype, M, topk, I, capacity);
  if (rc) return rc;
  if (I > (1 << 23)) return fail(CHORD_ERR_INVALID_ARG, "I=%d > 2^23", I);
  const bool keep = codes || scales;
  if (keep && gu) return fail(CHORD_ERR_INVALID_ARG, "gu and its codes: one of them");
  if (keep && I % 32 != 0) return fail(CHORD_ERR_INVALID_ARG, "I=%d must be a multiple of 32 to be held in 8 bits", I);
  if (M == 0) return CHORD_OK;
  if (!dweights) return fail(CHORD_ERR_INVALID_ARG, "null pointer: dweights");
  if (capacity == 0)
    return done(cudaMemsetAsync(dweights, 0, sizeof(float) * M * topk, stream_of(stream)), "gradient of no rows");
  if ((rc = check_matrix("dh", dh, dtype, dh_stride, I, false))) return rc;
  if (keep ? (rc = check_codes(codes, scales)) : (rc = check_matrix("gu", gu, dtype, gu_stride, 2 * I, false))) return rc;
  if ((rc = check_matrix("dgu", dgu, dtype, dgu_stride, 2 * I, true))) return rc;
  if (h && (rc = check_matrix("h", h, dtype, h_stride, I, true))) return rc;
  if (!topk_weights || !sorted_positions || !sorted_token_ids || !num_tokens_post_padded)
    return fail(CHORD_ERR_INVALID_ARG, "null pointer");
  chord::Swiglu s{};
  s.gu = gu, s.dh = dh, s.w = topk_weights, s.sorted = sorted_token_ids, s.ntpp = num_tokens_post_padded;
  s.pos = sorted_positions, s.h = h, s.dgu = dgu, s.dw = dweights;
  s.codes = const_cast<uint8_t*>(codes), s.scales = const_cast<uint8_t*>(scales);   // (read only)
  s.ldg = gu_stride, s.ldh = h_stride, s.ldd = dh_stride, s.ldo = dgu_stride;
  s.rows = static_cast<int>(capacity), s.I = I, s.assignments = M * topk;
  return done(chord::swiglu_launch(s, dtype, true, stream_of(stream)), "swiglu backward launch");
}

}  // extern "C"
