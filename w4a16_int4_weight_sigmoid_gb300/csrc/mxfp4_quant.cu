// MXFP4 quantisation: values to 4-bit blocks and back, token rows straight
// into the experts' product's operand (with the permutation into expert
// order), and the weights' repacking.
//
// A thread holds 8 consecutive values (one 16-byte load for 16-bit types);
// four threads hold a block of 32, whose largest magnitude takes two
// shuffles.  The maximum is taken on the bit patterns of |x| (ordered like
// the values, infinities and NaNs above all finite ones), and the scale is a
// power of two, so x / scale and its rounding to E2M1 are exact operations.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "mxfp4.cuh"

namespace chord {
namespace {

constexpr int kThreads = 256;

// Eight consecutive values as FP32; V elements per access (V divides 8).
template <typename T, int V>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8 / V; ++i) {
    const Vec<T, V> x = reinterpret_cast<const Vec<T, V>*>(p)[i];
#pragma unroll
    for (int e = 0; e < V; ++e) v[i * V + e] = to_f32(x.e[e]);
  }
}

// This thread's 8 codes and the scale code of the block that it shares with
// the other lanes of its group of four.  All lanes of the warp call it.
__device__ __forceinline__ uint32_t quantize8(float (&v)[8], uint32_t& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  scale = mx_scale_code(m);
  const float inv = mx_inverse_scale(scale);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = scale == 255u ? 0.f : v[i] * inv;
  return e2m1x8(v);
}

// ---------------------------------------------------------------- row-major
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T* __restrict__ x, long long ldx, long long rows,
                                                            int K, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  const int g = blockIdx.x * kThreads + threadIdx.x;   // group of 8 values of the row
  const bool in = g < K / 8;
  for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
    float v[8] = {};
    if (in) load8<T, V>(x + r * ldx + 8 * g, v);
    uint32_t scale;
    const uint32_t q = quantize8(v, scale);
    if (in) {
      reinterpret_cast<uint32_t*>(codes + r * (K / 2))[g] = q;
      if ((g & 3) == 0) scales[r * (K / kMxBlock) + g / 4] = static_cast<uint8_t>(scale);
    }
  }
}

// E2M1 code -> value: an FP32 number whose exponent and mantissa come
// straight from the three magnitude bits, times 2^126 (subnormal 0.5
// included), then the block's scale.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, long long rows,
                                                              int K, T* __restrict__ out, long long ldo) {
  const int g = blockIdx.x * kThreads + threadIdx.x;
  if (g >= K / 8) return;
  for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
    const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(codes + r * (K / 2)) + g);
    const uint32_t code = __ldg(scales + r * (K / kMxBlock) + g / 4);
    const float scale = code == 255u ? __uint_as_float(0x7FC00000u)
                                     : code == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(code << 23);
    T* dst = out + r * ldo + 8 * g;
#pragma unroll
    for (int i = 0; i < 8 / V; ++i) {
      Vec<T, V> o;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const uint32_t n = (q >> (4 * (i * V + e))) & 15u;
        const float mag = __uint_as_float((n & 7u) << 22) * __uint_as_float(253u << 23);
        from_f32(o.e[e], (n & 8u ? -mag : mag) * scale);
      }
      reinterpret_cast<Vec<T, V>*>(dst)[i] = o;
    }
  }
}

// ------------------------------------------------------- the product's rows
// Token rows into the operand layout: token t to its rows pos[t, :] (pos
// given), or row r to row r below the padded total (pos NULL).  Each token
// is read and quantised once, whatever the number of its experts.  Padding
// rows are not written: the product computes each row from itself alone and
// stores no padding row.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const T* __restrict__ x, long long ldx, int M, int K,
                                                                 const int32_t* __restrict__ pos, int topk,
                                                                 const int32_t* __restrict__ ntpp, int rows,
                                                                 uint8_t* __restrict__ out) {
  const int g = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
  const size_t padded = mx_rows_padded(rows);
  uint8_t* out_scales = out + static_cast<size_t>(mx_units(K)) * padded * kMxRowBytes;
  const bool in_unit = g < mx_units(K) * (kMxUnitK / 8), in = g < K / 8;
  const int unit = g / (kMxUnitK / 8), chunk = (g / 4) % kMxRowScales;
  const int n = pos ? M : min(min(__ldg(ntpp), rows), M);
  for (int t = blockIdx.y; t < n; t += gridDim.y) {
    int p = -1;
    if (pos) {
      if (lane < topk) p = __ldg(pos + static_cast<long long>(t) * topk + lane);
      if (p >= rows) p = -1;
    } else if (lane == 0) {
      p = t;
    }
    uint32_t left = __ballot_sync(0xffffffffu, p >= 0);
    if (!left) continue;
    float v[8] = {};
    if (in) load8<T, V>(x + t * ldx + 8 * g, v);
    uint32_t scale;
    const uint32_t q = quantize8(v, scale);
    for (; left; left &= left - 1) {
      const size_t r = __shfl_sync(0xffffffffu, p, __ffs(left) - 1);
      if (in_unit) {
        reinterpret_cast<uint32_t*>(out + mx_chunk_offset(unit, padded, r, chunk))[g & 3] = q;
        if ((g & 3) == 0) out_scales[(unit * padded + r) * kMxRowScales + chunk] = static_cast<uint8_t>(scale);
      }
    }
  }
}

// ------------------------------------------------------------------ weights
struct MxHeader {
  uint32_t magic, version;
  int32_t E, N, K, flags;
};

// Thread = one block of 32 values (16 B and one scale byte) of one tile row.
__global__ void mx_prepack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int E, int N,
                                  int K, int gate_up, uint8_t* __restrict__ out, MxHeader h) {
  const int units = mx_units(K), tiles = mx_tiles(N);
  const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (id < 64) reinterpret_cast<uint32_t*>(out)[id] = id < sizeof(h) / 4 ? reinterpret_cast<const uint32_t*>(&h)[id] : 0u;
  if (id >= static_cast<long long>(E) * tiles * units * kMxTileRows * kMxRowScales) return;
  const int c = static_cast<int>(id % kMxRowScales);
  const int r = static_cast<int>(id / kMxRowScales % kMxTileRows);
  const long long unit_id = id / (kMxRowScales * kMxTileRows);
  const int u = static_cast<int>(unit_id % units), tile = static_cast<int>(unit_id / units % tiles);
  const long long e = unit_id / units / tiles;
  int n = kMxTileRows * tile + r;
  if (gate_up) {
    const int i = (kMxTileRows / 2) * tile + 16 * (r / 32) + r % 16;
    n = i < N / 2 ? i + (r % 32 / 16) * (N / 2) : N;
  }
  const int block = u * kMxRowScales + c;
  uint4 q = make_uint4(0, 0, 0, 0);
  uint8_t s = 0;
  if (n < N && block < K / kMxBlock) {
    const long long at = (e * N + n) * (K / kMxBlock) + block;
    q = reinterpret_cast<const uint4*>(codes)[at];
    s = scales[at];
  }
  uint8_t* dst = out + kPackHeaderBytes + unit_id * kMxUnitBytes;
  *reinterpret_cast<uint4*>(dst + r * kMxRowBytes + 16 * (c ^ (r & 7))) = q;
  dst[kMxTileBytes + (c / 4) * 512 + (r % 32) * 16 + (r / 32) * 4 + c % 4] = s;
}

template <typename T>
cudaError_t quantize_t(const void* x, long long ldx, long long rows, int K, uint8_t* codes, uint8_t* scales,
                       cudaStream_t st) {
  const dim3 grid((K / 8 + kThreads - 1) / kThreads, static_cast<unsigned>(std::min<long long>(rows, 65535)));
  constexpr int kV = 16 / sizeof(T);
  if (row_access_bytes(x, ldx, K, sizeof(T)) == 16)
    quantize_kernel<T, kV><<<grid, kThreads, 0, st>>>(static_cast<const T*>(x), ldx, rows, K, codes, scales);
  else
    quantize_kernel<T, 1><<<grid, kThreads, 0, st>>>(static_cast<const T*>(x), ldx, rows, K, codes, scales);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, long long rows, int K, void* out, long long ldo,
                         cudaStream_t st) {
  const dim3 grid((K / 8 + kThreads - 1) / kThreads, static_cast<unsigned>(std::min<long long>(rows, 65535)));
  constexpr int kV = 16 / sizeof(T);
  if (row_access_bytes(out, ldo, K, sizeof(T)) == 16)
    dequantize_kernel<T, kV><<<grid, kThreads, 0, st>>>(codes, scales, rows, K, static_cast<T*>(out), ldo);
  else
    dequantize_kernel<T, 1><<<grid, kThreads, 0, st>>>(codes, scales, rows, K, static_cast<T*>(out), ldo);
  return cudaGetLastError();
}

template <typename T>
cudaError_t quantize_rows_t(const void* x, long long ldx, int M, int K, const int32_t* pos, int topk,
                            const int32_t* ntpp, int rows, uint8_t* out, cudaStream_t st) {
  const dim3 grid((mx_units(K) * (kMxUnitK / 8) + kThreads - 1) / kThreads, std::min(M, 65535));
  constexpr int kV = 16 / sizeof(T);
  if (row_access_bytes(x, ldx, K, sizeof(T)) == 16)
    quantize_rows_kernel<T, kV><<<grid, kThreads, 0, st>>>(static_cast<const T*>(x), ldx, M, K, pos, topk, ntpp, rows,
                                                           out);
  else
    quantize_rows_kernel<T, 1><<<grid, kThreads, 0, st>>>(static_cast<const T*>(x), ldx, M, K, pos, topk, ntpp, rows,
                                                          out);
  return cudaGetLastError();
}

}  // namespace

cudaError_t mxfp4_quantize_launch(const void* x, int dtype, long long ldx, long long rows, int K, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t st) {
  if (dtype == CHORD_DTYPE_BF16) return quantize_t<Bf16>(x, ldx, rows, K, codes, scales, st);
  if (dtype == CHORD_DTYPE_FP16) return quantize_t<Fp16>(x, ldx, rows, K, codes, scales, st);
  return quantize_t<float>(x, ldx, rows, K, codes, scales, st);
}

cudaError_t mxfp4_dequantize_launch(const uint8_t* codes, const uint8_t* scales, long long rows, int K, void* out,
                                    int dtype, long long ldo, cudaStream_t st) {
  if (dtype == CHORD_DTYPE_BF16) return dequantize_t<Bf16>(codes, scales, rows, K, out, ldo, st);
  if (dtype == CHORD_DTYPE_FP16) return dequantize_t<Fp16>(codes, scales, rows, K, out, ldo, st);
  return dequantize_t<float>(codes, scales, rows, K, out, ldo, st);
}

cudaError_t mxfp4_quantize_rows_launch(const void* x, int dtype, long long ldx, int M, int K, const int32_t* pos,
                                       int topk, const int32_t* ntpp, int rows, uint8_t* out, cudaStream_t st) {
  if (dtype == CHORD_DTYPE_BF16) return quantize_rows_t<Bf16>(x, ldx, M, K, pos, topk, ntpp, rows, out, st);
  if (dtype == CHORD_DTYPE_FP16) return quantize_rows_t<Fp16>(x, ldx, M, K, pos, topk, ntpp, rows, out, st);
  return quantize_rows_t<float>(x, ldx, M, K, pos, topk, ntpp, rows, out, st);
}

size_t mxfp4_prepack_bytes(int E, int N, int K) {
  return kPackHeaderBytes + static_cast<size_t>(E) * mx_tiles(N) * mx_units(K) * kMxUnitBytes;
}

size_t mxfp4_rows_bytes(size_t rows, int K) {
  return static_cast<size_t>(mx_units(K)) * mx_rows_padded(rows) * (kMxRowBytes + kMxRowScales);
}

cudaError_t mxfp4_prepack_launch(const uint8_t* codes, const uint8_t* scales, int E, int N, int K, bool gate_up,
                                 uint8_t* out, cudaStream_t st) {
  const MxHeader h{kMxMagic, kMxVersion, E, N, K, gate_up ? 1 : 0};
  const long long threads = static_cast<long long>(E) * mx_tiles(N) * mx_units(K) * kMxTileRows * kMxRowScales;
  mx_prepack_kernel<<<static_cast<unsigned>((threads + 255) / 256), 256, 0, st>>>(codes, scales, E, N, K,
                                                                                  gate_up ? 1 : 0, out, h);
  return cudaGetLastError();
}

}  // namespace chord
