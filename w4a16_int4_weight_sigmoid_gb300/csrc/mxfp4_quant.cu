// MXFP4 quantisation: values to 4-bit blocks and back, token rows straight
// into the experts' product's operand (with the permutation into expert
// order), and the weights' repacking.
//
// A thread holds 16 consecutive values (one 32-byte load for 16-bit types);
// two threads hold a block of 32, whose largest magnitude takes one shuffle.
// The maximum is taken on the bit patterns of |x| (ordered like the values,
// infinities and NaNs above all finite ones; 16-bit types two to a register),
// and the scale is a power of two, so x / scale and its rounding to E2M1 are
// exact operations.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"
#include "mxfp4.cuh"

namespace chord {
namespace {

constexpr int kThreads = 128;
// CTAs per SM that the kernels are compiled for, and the grid in such waves,
// each CTA walking on to its next row: dequantising 8192 x 7168 took 27.4 us
// with one wave, 25.5 with two, 24.4 with four, 34.2 with a CTA for every row.
template <typename T>
constexpr int kCtas = sizeof(T) == 4 ? 8 : 12;
constexpr int kWaves = 4;
constexpr int kRun = 16;   // values per thread

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

// Bits of the largest |x| as FP32.
__device__ __forceinline__ uint32_t run_max(const Run<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) m = max(m, r.w[i] & 0x7FFFFFFFu);
  return m;
}
template <typename T>
__device__ __forceinline__ uint32_t run_max(const Run<T>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < Run<T>::kWords; ++i) m = __vmaxu2(m, r.w[i] & 0x7FFF7FFFu);
  T t;
  t.v = static_cast<uint16_t>(max(m & 0xFFFFu, m >> 16));
  return __float_as_uint(to_f32(t));
}

// This thread's 16 codes and the scale code of the block that it shares with
// its neighbour lane.  All lanes of the warp call it.
template <typename T>
__device__ __forceinline__ uint2 quantize_run(const Run<T>& r, uint32_t& scale) {
  uint32_t m = run_max(r);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  scale = mx_scale_code(m);
  const float inv = scale == 255u ? 0.f : mx_inverse_scale(scale);
  float v[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) v[i] = to_f32(r.e[i]) * inv;
  uint2 q = make_uint2(e2m1x8(v), e2m1x8(v + 8));
  if (scale == 255u) q = make_uint2(0, 0);   // an infinity or a NaN in the block
  return q;
}

// ---------------------------------------------------------------- row-major
// CTA column: a run of each thread; rows blockIdx.y, + gridDim.y, ..., two at
// a time so that the second's loads are in flight while the first is worked on.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtas<T>) quantize_kernel(const T* x, long long ldx, long long rows, int K,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  const int g = blockIdx.x * kThreads + threadIdx.x;
  const bool in = g < K / kRun;
  grid_dep_wait();
  grid_dep_launch();
  auto load = [&](long long r, Run<T>& v) {
    v = Run<T>{};
    if (in && r < rows) load_run<kWide>(x + r * ldx + kRun * g, v);
  };
  auto store = [&](long long r, const Run<T>& v) {
    uint32_t scale;
    const uint2 q = quantize_run(v, scale);
    if (in && r < rows) {
      reinterpret_cast<uint2*>(codes + r * (K / 2))[g] = q;
      if ((g & 1) == 0) scales[r * (K / kMxBlock) + g / 2] = static_cast<uint8_t>(scale);
    }
  };
  for (long long r = blockIdx.y; r < rows; r += 2 * gridDim.y) {
    Run<T> v0, v1;
    load(r, v0);
    load(r + gridDim.y, v1);
    store(r, v0);
    store(r + gridDim.y, v1);
  }
}

template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtas<T>) dequantize_kernel(const uint8_t* codes,
                                                              const uint8_t* scales, long long rows,
                                                              int K, T* __restrict__ out, long long ldo) {
  const int g = blockIdx.x * kThreads + threadIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  if (g >= K / kRun) return;
  constexpr int kRows = 4;   // rows in flight
  for (long long r = blockIdx.y; r < rows; r += kRows * gridDim.y) {
    uint2 q[kRows];
    uint32_t code[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const long long row = r + static_cast<long long>(j) * gridDim.y;
      if (row < rows) {
        Chunk<8> c;
        load_chunk<8>(codes + row * (K / 2) + 8 * g, c);
        q[j] = make_uint2(c.w[0], c.w[1]);
        asm volatile("ld.global.u8 %0, [%1];" : "=r"(code[j]) : "l"(scales + row * (K / kMxBlock) + g / 2));
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const long long row = r + static_cast<long long>(j) * gridDim.y;
      if (row >= rows) break;
      // 2^(code - 127): code 0 is subnormal, 255 is NaN
      const float scale =
          __uint_as_float(code[j] == 255u ? 0x7FC00000u : code[j] == 0u ? 0x00400000u : code[j] << 23);
      uint32_t h[8];
      e2m1x8_to_f16(q[j].x, *reinterpret_cast<uint32_t(*)[4]>(h));
      e2m1x8_to_f16(q[j].y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
      Run<T> o;
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        from_f32(o.e[i], __half2float(__ushort_as_half(static_cast<uint16_t>(h[i / 2] >> (16 * (i & 1))))) * scale);
      T* dst = out + row * ldo + kRun * g;
      if (kWide) {
#pragma unroll
        for (int i = 0; i < Run<T>::kWords / 8; ++i) store_chunk<32>(reinterpret_cast<uint8_t*>(dst) + 32 * i, o.c[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kRun; ++i) dst[i] = o.e[i];
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
                                                                 int rows, uint8_t* __restrict__ out) {
  const int g = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
  const int units = mx_units(K);
  uint8_t* out_scales = out + units * mx_rows_padded(rows) * kMxRowBytes;
  const bool in_unit = g < units * (kMxUnitK / kRun), in = g < K / kRun;
  const int unit = g / (kMxUnitK / kRun), chunk = (g / 2) % kMxRowScales;
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
  auto load = [&](int p, Run<T>& v, int t) {
    v = Run<T>{};
    const uint32_t left = __ballot_sync(0xffffffffu, p >= 0);
    if (left && in) load_run<kWide>(x + t * ldx + kRun * g, v);
    return left;
  };
  auto store = [&](int p, uint32_t left, const Run<T>& v) {
    if (!left) return;
    uint32_t scale;
    const uint2 q = quantize_run(v, scale);
    for (; left; left &= left - 1) {
      const uint32_t r = __shfl_sync(0xffffffffu, p, __ffs(left) - 1);
      if (in_unit) {
        const size_t at = mx_row_place(unit, units, r);
        reinterpret_cast<uint2*>(out + at * kMxRowBytes + 16 * (chunk ^ (r & 7)))[g & 1] = q;
        if ((g & 1) == 0) out_scales[at * kMxRowScales + chunk] = static_cast<uint8_t>(scale);
      }
    }
  };
  const int step = gridDim.y;
  Run<T> v0, v1;
  int p0 = position(blockIdx.y), p1 = position(blockIdx.y + step);
  uint32_t left0 = load(p0, v0, blockIdx.y);
  for (int t = blockIdx.y; t < n; t += 2 * step) {
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
dim3 grid_for(int columns, long long rows) {
  static int sms = 0;
  if (!sms) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, 0);
  const long long most = std::max(1LL, static_cast<long long>(kWaves) * kCtas<T> * sms / columns);
  return dim3(columns, static_cast<unsigned>(std::min({rows, most, 65535LL})));
}

template <typename T>
cudaError_t quantize_t(const void* x, long long ldx, long long rows, int K, uint8_t* codes, uint8_t* scales,
                       cudaStream_t st) {
  const bool wide = row_access_bytes(x, ldx, K, sizeof(T), 32) == 32;
  return launch_kernel(wide ? quantize_kernel<T, true> : quantize_kernel<T, false>,
                       grid_for<T>((K / kRun + kThreads - 1) / kThreads, rows), dim3(kThreads), 0, st, true,
                       static_cast<const T*>(x), ldx, rows, K, codes, scales);
}

template <typename T>
cudaError_t dequantize_t(const uint8_t* codes, const uint8_t* scales, long long rows, int K, void* out, long long ldo,
                         cudaStream_t st) {
  const bool wide = row_access_bytes(out, ldo, K, sizeof(T), 32) == 32;
  return launch_kernel(wide ? dequantize_kernel<T, true> : dequantize_kernel<T, false>,
                       grid_for<T>((K / kRun + kThreads - 1) / kThreads, rows), dim3(kThreads), 0, st, true, codes,
                       scales, rows, K, static_cast<T*>(out), ldo);
}

template <typename T>
cudaError_t quantize_rows_t(const void* x, long long ldx, int M, int K, const int32_t* pos, int topk,
                            const int32_t* ntpp, int rows, uint8_t* out, cudaStream_t st) {
  const bool wide = row_access_bytes(x, ldx, K, sizeof(T), 32) == 32;
  return launch_kernel(wide ? quantize_rows_kernel<T, true> : quantize_rows_kernel<T, false>,
                       grid_for<T>((mx_units(K) * (kMxUnitK / kRun) + kThreads - 1) / kThreads, M), dim3(kThreads), 0,
                       st, true, static_cast<const T*>(x), ldx, M, K, pos, topk, ntpp, rows, out);
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
