// MXFP4 quantisation: values to 4-bit blocks and back, token rows straight
// into the experts' product's operand (with the permutation into expert
// order), and the weights' repacking.
//
// A thread holds a whole block: 32 consecutive values (two 32-byte loads for
// 16-bit types), so the block's maximum needs no other lane, its codes are
// one 16-byte store, and what a row costs beside its values (positions,
// addresses) is paid by half the threads that a block shared by two needs.
// The maximum is taken on |x| with NaNs above all (16-bit types two to a
// register), and the scale is a power of two, so x / scale and its rounding
// to E2M1 are exact operations.
// Bound by memory.  Measured, 8192 x 7168 BF16: quantise 22.9 us, dequantise
// 24.0 us (148 MB each: 6.5 and 6.2 TB/s of 6.7 that a copy reaches); rows into
// expert order on 48 of 384 experts 20.6 us (108 MB), on all of 8 experts, two
// copies of each token, 29.3 us (179 MB).
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "mxfp4.cuh"

namespace chord {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
// CTAs per SM that the kernels are compiled for, and the grid in such waves,
// each CTA walking on to its next row.  8192 x 7168 BF16: dequantising took
// 25.0 us with two waves, 23.9 with four, 34 with a CTA for every row;
// rows into expert order (8 ranks' share) 19.8 us with two, 21.0 with four.
template <typename T>
constexpr int kCtas = sizeof(T) == 4 ? 5 : 8;
constexpr int kWaves = 4, kRowWaves = 2;
constexpr int kRun = kMxBlock;   // values per thread

// kRun consecutive values as 32-bit words; kWide: 32-byte aligned.
template <typename T>
struct Run {
  static constexpr int kWords = kRun * sizeof(T) / 4;
  union {
    uint32_t w[kWords];
    T e[kRun];
    Chunk<32> c[kWords / 8];
  };
};
template <bool kWide, typename T>
__device__ __forceinline__ void load_run(const T* p, Run<T>& r) {
  if constexpr (kWide) {
#pragma unroll
    for (int i = 0; i < Run<T>::kWords / 8; ++i) load_chunk<32>(reinterpret_cast<const uint8_t*>(p) + 32 * i, r.c[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      Chunk<sizeof(T)> c;
      load_chunk<sizeof(T)>(p + i, c);
      if constexpr (sizeof(T) == 4) r.w[i] = c.w[0];
      else r.w[i / 2] = i & 1 ? r.w[i / 2] | (c.w[0] << 16) : c.w[0];
    }
  }
}

// Bits of the largest |x| as FP32; a NaN's where there is one.
__device__ __forceinline__ uint32_t run_max(const Run<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) m = max(m, r.w[i] & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, Bf16) {
  asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, Fp16) {
  asm("max.NaN.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
template <typename T>
__device__ __forceinline__ uint32_t run_max(const Run<T>& r) {
  uint32_t m = r.w[0];
#pragma unroll
  for (int i = 1; i < Run<T>::kWords; ++i) m = max_abs2(m, r.w[i], T{});
  T t;
  t.v = static_cast<uint16_t>(max(m & 0x7FFFu, (m >> 16) & 0x7FFFu));
  return __float_as_uint(to_f32(t));
}

// Codes of eight values (words r.w[n..]) times 2^(127 - code).  The product
// is exact wherever it is not far below the smallest midpoint, in the input's
// own type for the 16-bit ones.
__device__ __forceinline__ uint32_t scaled_codes(const Run<float>& r, int n, uint32_t code) {
  const float inv = mx_inverse_scale(code);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r.e[n + i] * inv;
  return e2m1x8(v);
}
__device__ __forceinline__ uint32_t scaled_codes(const Run<Bf16>& r, int n, uint32_t code) {
  const uint32_t inv = min(254u, 254u - code) * 0x00800080u;   // the exponent field of both halves
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p) : "r"(r.w[n / 2 + i]), "r"(inv));
    v[2 * i] = __uint_as_float(p << 16);
    v[2 * i + 1] = __uint_as_float(p & 0xFFFF0000u);
  }
  return e2m1x8(v);
}
__device__ __forceinline__ uint32_t scaled_codes(const Run<Fp16>& r, int n, uint32_t code) {
  // 127 - code is -13 .. 26 for FP16's range: two factors within FP16's own
  const int k = 127 - static_cast<int>(code), k0 = min(k, 15), k1 = min(k - k0, 15);
  const uint32_t f0 = static_cast<uint32_t>(max(k0 + 15, 1)) * 0x04000400u;
  const uint32_t f1 = static_cast<uint32_t>(k1 + 15) * 0x04000400u;
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(r.w[n / 2 + i]), "r"(f0));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[i]) : "r"(f1));
  }
  return e2m1x8_from_f16(h);
}

// The 32 codes of a block and its scale code.
template <typename T>
__device__ __forceinline__ uint4 quantize_run(const Run<T>& r, uint32_t& scale) {
  scale = mx_scale_code(run_max(r));
  uint4 q = make_uint4(scaled_codes(r, 0, scale), scaled_codes(r, 8, scale), scaled_codes(r, 16, scale),
                       scaled_codes(r, 24, scale));
  if (scale == 255u) q = make_uint4(0, 0, 0, 0);   // an infinity or a NaN in the block
  return q;
}

// ---------------------------------------------------------------- row-major
// A thread's block g of rows r, r + step, ..., two at a time so that the
// second's loads are in flight while the first is worked on.  2^cols_log2
// threads of a CTA lie along the row and the rest on other rows, so short rows
// leave no threads idle.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtas<T>) quantize_kernel(const T* x, long long ldx, long long rows, int K,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales, int cols_log2) {
  const int g = (blockIdx.x << cols_log2) + (threadIdx.x & ((1 << cols_log2) - 1)), per = kThreads >> cols_log2;
  const long long first = static_cast<long long>(blockIdx.y) * per + (threadIdx.x >> cols_log2), step = gridDim.y * per;
  const bool in = g < K / kRun;
  grid_dep_wait();
  grid_dep_launch();
  auto load = [&](long long r, Run<T>& v) {
    if (in && r < rows) load_run<kWide>(x + r * ldx + kRun * g, v);
  };
  auto store = [&](long long r, const Run<T>& v) {
    uint32_t scale;
    if (in && r < rows) {
      const uint4 q = quantize_run(v, scale);
      reinterpret_cast<uint4*>(codes + r * (K / 2))[g] = q;
      scales[r * (K / kMxBlock) + g] = static_cast<uint8_t>(scale);
    }
  };
  for (long long r = first; r < rows; r += 2 * step) {
    Run<T> v0{}, v1{};
    load(r, v0);
    load(r + step, v1);
    store(r, v0);
    store(r + step, v1);
  }
}

template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtas<T>) dequantize_kernel(const uint8_t* codes,
                                                              const uint8_t* scales, long long rows,
                                                              int K, T* __restrict__ out, long long ldo, int cols_log2) {
  const int g = (blockIdx.x << cols_log2) + (threadIdx.x & ((1 << cols_log2) - 1)), per = kThreads >> cols_log2;
  const long long first = static_cast<long long>(blockIdx.y) * per + (threadIdx.x >> cols_log2), step = gridDim.y * per;
  grid_dep_wait();
  grid_dep_launch();
  if (g >= K / kRun) return;
  constexpr int kRows = 2;   // rows in flight
  for (long long r = first; r < rows; r += kRows * step) {
    Chunk<16> q[kRows];
    uint32_t code[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const long long row = r + j * step;
      if (row < rows) {
        load_chunk<16>(codes + row * (K / 2) + 16 * g, q[j]);
        asm volatile("ld.global.u8 %0, [%1];" : "=r"(code[j]) : "l"(scales + row * (K / kMxBlock) + g));
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const long long row = r + j * step;
      if (row >= rows) break;
      // 2^(code - 127): code 0 is subnormal, 255 is NaN
      const float scale =
          __uint_as_float(code[j] == 255u ? 0x7FC00000u : code[j] == 0u ? 0x00400000u : code[j] << 23);
      T* dst = out + row * ldo + kRun * g;
      constexpr int kPart = 32 / sizeof(T);   // values per 32-byte store
#pragma unroll
      for (int c = 0; c < kRun / kPart; ++c) {
        float f[kPart];
#pragma unroll
        for (int w = 0; w < kPart / 8; ++w) {
          uint32_t h[4];
          e2m1x8_to_f16(q[j].w[c * (kPart / 8) + w], h);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f[8 * w + i] = __half2float(__ushort_as_half(static_cast<uint16_t>(h[i / 2] >> (16 * (i & 1))))) * scale;
        }
        if constexpr (kWide) {
          Chunk<32> o;
          f32_chunk<T, 32>(o, f);
          store_chunk<32>(dst + kPart * c, o);
        } else {
#pragma unroll
          for (int i = 0; i < kPart; ++i) from_f32(dst[kPart * c + i], f[i]);
        }
      }
    }
  }
}

// ------------------------------------------------------- the product's rows
// Token rows into the operand layout: token t to its rows pos[t, :] (pos
// given), or row r to row r below the padded total (pos NULL).  Each token
// is read and quantised once, whatever the number of its experts; the next
// token's positions are fetched meanwhile.  Padding rows are not written: the
// product computes each row from itself alone and stores no padding row.
// A programmatic launch: the product that follows starts while this ends.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtas<T>) quantize_rows_kernel(const T* x, long long ldx, int M, int K,
                                                                 const int32_t* pos, int topk, const int32_t* ntpp,
                                                                 int rows, uint8_t* __restrict__ out, int wpt_log2) {
  // 2^wpt_log2 warps (1, 2 or 4) of a CTA share a token
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tokens = kWarps >> wpt_log2;
  const int g = ((blockIdx.x << wpt_log2) + (warp & ((1 << wpt_log2) - 1))) * 32 + lane;
  const int units = mx_units(K);
  uint8_t* out_scales = out + units * mx_rows_padded(rows) * kMxRowBytes;
  const bool in_unit = g < units * (kMxUnitK / kRun), in = g < K / kRun;
  const int unit = g / kMxRowScales, chunk = g % kMxRowScales;
  grid_dep_wait();
  grid_dep_launch();
  const int n = pos ? M : min(min(ld_ca(ntpp), rows), M);
  auto position = [&](int t) {
    int p = -1;
    if (t < n) {
      if (!pos) p = lane == 0 ? t : -1;
      else if (lane < topk) p = ld_ca(pos + static_cast<long long>(t) * topk + lane);
    }
    return p < rows ? p : -1;
  };
  // two tokens alternate, so that the next one's values and the positions of
  // the one after it are in flight
  // this thread's place in a row of slab 0; a slab and a row further on
  uint8_t* out_g = out + static_cast<size_t>(unit) * kMxSlabRows * kMxRowBytes;
  uint8_t* scale_g = out_scales + static_cast<size_t>(unit) * kMxSlabRows * kMxRowScales + chunk;
  const uint32_t slab_rows = units * kMxSlabRows;
  auto load = [&](int p, Run<T>& v, int t) {
    if (!in) v = Run<T>{};   // K's padding
    const uint32_t left = __ballot_sync(0xffffffffu, p >= 0);
    if (left && in) load_run<kWide>(x + t * ldx + kRun * g, v);
    return left;
  };
  auto store = [&](int p, uint32_t left, const Run<T>& v) {
    if (!left) return;
    uint32_t scale;
    const uint4 q = quantize_run(v, scale);
    for (; left; left &= left - 1) {
      const uint32_t r = __shfl_sync(0xffffffffu, p, __ffs(left) - 1);
      if (in_unit) {
        const size_t at = static_cast<size_t>(r / kMxSlabRows) * slab_rows + r % kMxSlabRows;
        *reinterpret_cast<uint4*>(out_g + at * kMxRowBytes + 16 * (chunk ^ (r & 7))) = q;
        scale_g[at * kMxRowScales] = static_cast<uint8_t>(scale);
      }
    }
  };
  const int step = gridDim.y * tokens, t_first = blockIdx.y * tokens + (warp >> wpt_log2);
  Run<T> v0, v1;
  int p0 = position(t_first), p1 = position(t_first + step);
  uint32_t left0 = load(p0, v0, t_first);
  for (int t = t_first; t < n; t += 2 * step) {
    const int p2 = position(t + 2 * step), p3 = position(t + 3 * step);
    const uint32_t left1 = load(p1, v1, t + step);
    store(p0, left0, v0);
    left0 = load(p2, v0, t + 2 * step);
    store(p1, left1, v1);
    p0 = p2;
    p1 = p3;
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
  const long long pair_tiles = min(2, tiles - tile / 2 * 2);
  const long long place = (e * tiles + tile / 2 * 2) * units + u * pair_tiles + tile % 2;
  uint8_t* dst = out + kPackHeaderBytes + place * kMxUnitBytes;
  *reinterpret_cast<uint4*>(dst + r * kMxRowBytes + 16 * (c ^ (r & 7))) = q;
  dst[kMxTileBytes + (c / 4) * 512 + (r % 32) * 16 + (r / 32) * 4 + c % 4] = s;
}

template <typename T>
dim3 grid_for(int columns, long long rows, int waves) {
  const long long most = std::max(1LL, static_cast<long long>(waves) * kCtas<T> * sm_count() / columns);
  return dim3(columns, static_cast<unsigned>(std::min({rows, most, 65535LL})));
}

// log2 of the threads along a row of K / 32 blocks.
int row_threads_log2(int K) {
  int n = 0;
  while ((1 << n) < kThreads && (1 << n) < K / kRun) ++n;
  return n;
}

template <typename T>
cudaError_t quantize_t(const void* x, long long ldx, long long rows, int K, uint8_t* codes, uint8_t* scales,
                       cudaStream_t st) {
  const bool wide = row_access_bytes(x, ldx, K, sizeof(T), 32) == 32;
  const int log2 = row_threads_log2(K), cols = 1 << log2, per = kThreads >> log2;
  return launch_kernel(wide ? quantize_kernel<T, true> : quantize_kernel<T, false>,
                       grid_for<T>((K / kRun + cols - 1) / cols, (rows + per - 1) / per, kWaves), dim3(kThreads), 0,
                       st, true, static_cast<const T*>(x), ldx, rows, K, codes, scales, log2);
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, long long rows, int K, void* out, long long ldo,
                         cudaStream_t st) {
  const bool wide = row_access_bytes(out, ldo, K, sizeof(T), 32) == 32;
  const int log2 = row_threads_log2(K), cols = 1 << log2, per = kThreads >> log2;
  return launch_kernel(wide ? dequantize_kernel<T, true> : dequantize_kernel<T, false>,
                       grid_for<T>((K / kRun + cols - 1) / cols, (rows + per - 1) / per, kWaves), dim3(kThreads), 0,
                       st, true, codes, scales, rows, K, static_cast<T*>(out), ldo, log2);
}

template <typename T>
cudaError_t quantize_rows_t(const void* x, long long ldx, int M, int K, const int32_t* pos, int topk,
                            const int32_t* ntpp, int rows, uint8_t* out, cudaStream_t st) {
  const bool wide = row_access_bytes(x, ldx, K, sizeof(T), 32) == 32;
  const int warps = (mx_units(K) * kMxRowScales + 31) / 32, wpt = warps >= 3 ? 4 : warps, per = kWarps / wpt;
  return launch_kernel(wide ? quantize_rows_kernel<T, true> : quantize_rows_kernel<T, false>,
                       grid_for<T>((warps + wpt - 1) / wpt, (M + per - 1) / per, kRowWaves), dim3(kThreads), 0, st,
                       true, static_cast<const T*>(x), ldx, M, K, pos, topk, ntpp, rows, out, wpt / 2);
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
