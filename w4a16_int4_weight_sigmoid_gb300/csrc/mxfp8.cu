// Rows held in 8 bits (MXFP8), for activations that a backward pass reads again:
//   quantize    codes and scales of rows; see mxfp8.cuh for the scale
//   dequantize  the rows that they stand for
//   permute     the same, token rows straight into the aligned expert order:
//               out[r] = row of token sorted_token_ids[r] / topk, zeros in
//               padding rows
// Bound by memory: each value is read and written once, a thread takes up to
// 32 bytes of the wider side at a time; a block's largest magnitude takes one
// exchange between two lanes (16-bit types) or two among four.  permute reads
// a token's codes once for each of its local rows (one byte a value against
// the two that it writes, and mostly from L2, where quantize left them).
#include "kernels.h"
#include "mxfp8.cuh"

namespace chord {
namespace {

struct Mx8Args {
  const void* x;          // quantize
  void* out;              // the others
  long long ld;           // row stride of x or out, in elements
  const uint8_t* codes_in;
  const uint8_t* scales_in;
  uint8_t* codes;
  uint8_t* scales;
  const int32_t* sorted;  // permute
  const int32_t* ntpp;
  long long rows;
  int K, topk, assignments, lanes;
};

constexpr int kUnroll = 4;

template <typename T, int B>
__global__ void __launch_bounds__(kRowThreads) mxfp8_quantize_kernel(Mx8Args a) {
  constexpr int kN = B / sizeof(T);
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % a.lanes, per = kRowThreads / a.lanes;
  const long long step = static_cast<long long>(gridDim.x) * per;
  const int chunks = a.K / kN;
  // (the row of a warp is the same for all its lanes, and so are its turns)
  for (long long r = static_cast<long long>(blockIdx.x) * per + threadIdx.x / a.lanes; r < a.rows; r += step) {
    const T* x = static_cast<const T*>(a.x) + r * a.ld;
    for (int c0 = lane; c0 - (lane & 31) < chunks; c0 += kUnroll * a.lanes) {
      Chunk<B> v[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        v[i] = Chunk<B>{};
        if (c0 + i * a.lanes < chunks) load_chunk<B>(x + (c0 + i * a.lanes) * kN, v[i]);
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + i * a.lanes;
        if (i > 0 && c - (lane & 31) >= chunks) break;
        const uint32_t s = block_scale(block_top<T, B>(v[i]));
        if (c >= chunks) continue;
        float f[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) f[j] = chunk_f32<T, B>(v[i], j);
        uint32_t code[kN < 4 ? 1 : kN / 4];
        to_codes<kN>(f, s, code);
        store_codes<kN>(a.codes + r * a.K + c * kN, code);
        if ((c * kN) % kMx8Block == 0) a.scales[r * (a.K / kMx8Block) + c * kN / kMx8Block] = static_cast<uint8_t>(s);
      }
    }
  }
}

// The values in T, rounded once.  The largest E4M3 steps can round past FP16's
// largest value, which a finite block then keeps.
template <typename T, int B>
__device__ __forceinline__ void typed_values(const uint32_t (&code)[B / sizeof(T) < 4 ? 1 : B / sizeof(T) / 4],
                                             uint32_t s, Chunk<B>& v) {
  constexpr int kN = B / sizeof(T);
  float f[kN];
  from_codes<kN>(code, scale_value(s), f);
  if constexpr (std::is_same_v<T, Fp16>) {
    if (s != 255)
#pragma unroll
      for (int i = 0; i < kN; ++i) f[i] = fminf(fmaxf(f[i], -65504.f), 65504.f);
  }
  f32_chunk<T, B>(v, f);
}

template <typename T, int B, bool kPermute>
__global__ void __launch_bounds__(kRowThreads) mxfp8_dequantize_kernel(Mx8Args a) {
  constexpr int kN = B / sizeof(T);
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % a.lanes, per = kRowThreads / a.lanes;
  const long long step = static_cast<long long>(gridDim.x) * per;
  const int chunks = a.K / kN;
  const long long rows = kPermute ? min(a.rows, static_cast<long long>(ld_ca(a.ntpp))) : a.rows;
  for (long long r = static_cast<long long>(blockIdx.x) * per + threadIdx.x / a.lanes; r < rows; r += step) {
    long long from = r;
    bool filled = true;
    if constexpr (kPermute) {
      const int f = ld_ca(a.sorted + r);
      filled = f >= 0 && f < a.assignments;
      from = filled ? f / a.topk : 0;
    }
    const uint8_t* codes = a.codes_in + from * a.K;
    const uint8_t* scales = a.scales_in + from * (a.K / kMx8Block);
    T* out = static_cast<T*>(a.out) + r * a.ld;
    for (int c0 = lane; c0 < chunks; c0 += kUnroll * a.lanes) {
      uint32_t code[kUnroll][kN < 4 ? 1 : kN / 4], scale[kUnroll];
      if (filled) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int c = min(c0 + i * a.lanes, chunks - 1);
          load_codes<kN>(codes + c * kN, code[i]);
          scale[i] = load_scale(scales + c * kN / kMx8Block);
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + i * a.lanes;
        if (c >= chunks) break;
        Chunk<B> v{};
        if (filled) typed_values<T, B>(code[i], scale[i], v);
        store_chunk<B>(out + c * kN, v);
      }
    }
  }
}

template <typename T, int B>
cudaError_t launch(const Mx8Args& args, int what, cudaStream_t st) {
  Mx8Args a = args;
  a.lanes = row_lanes(a.rows, a.K / static_cast<int>(B / sizeof(T)), kUnroll);
  const long long per = kRowThreads / a.lanes, want = (a.rows + per - 1) / per, most = 32LL * sm_count();
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  auto kern = what == 0 ? mxfp8_quantize_kernel<T, B>
              : what == 1 ? mxfp8_dequantize_kernel<T, B, false>
                          : mxfp8_dequantize_kernel<T, B, true>;
  return launch_kernel(kern, grid, dim3(kRowThreads), 0, st, true, a);
}
template <typename T>
cudaError_t launch(const Mx8Args& a, int what, cudaStream_t st) {
  const int b = row_access_bytes(what == 0 ? a.x : a.out, a.ld, a.K, sizeof(T), 32);
  switch (b) {
    case 32: return launch<T, 32>(a, what, st);
    case 16: return launch<T, 16>(a, what, st);
    case 8: return launch<T, 8>(a, what, st);
    case 4: return launch<T, 4>(a, what, st);
    default:
      if constexpr (sizeof(T) == 2) return launch<T, 2>(a, what, st);
      return cudaErrorInvalidValue;   // (elements are aligned)
  }
}
cudaError_t launch(const Mx8Args& a, int dtype, int what, cudaStream_t st) {
  switch (dtype) {
    case CHORD_DTYPE_BF16: return launch<Bf16>(a, what, st);
    case CHORD_DTYPE_FP16: return launch<Fp16>(a, what, st);
    default: return launch<float>(a, what, st);
  }
}

}  // namespace

cudaError_t mxfp8_quantize_launch(const void* x, int dtype, long long ldx, long long rows, int K, uint8_t* codes,
                                  uint8_t* scales, cudaStream_t st) {
  Mx8Args a{};
  a.x = x, a.ld = ldx, a.rows = rows, a.K = K, a.codes = codes, a.scales = scales;
  return launch(a, dtype, 0, st);
}
cudaError_t mxfp8_dequantize_launch(const uint8_t* codes, const uint8_t* scales, long long rows, int K, void* out,
                                    int dtype, long long ldo, cudaStream_t st) {
  Mx8Args a{};
  a.codes_in = codes, a.scales_in = scales, a.rows = rows, a.K = K, a.out = out, a.ld = ldo;
  return launch(a, dtype, 1, st);
}
cudaError_t mxfp8_permute_launch(const uint8_t* codes, const uint8_t* scales, int K, const int32_t* sorted,
                                 const int32_t* ntpp, int M, int topk, int rows, void* out, int dtype, long long ldo,
                                 cudaStream_t st) {
  Mx8Args a{};
  a.codes_in = codes, a.scales_in = scales, a.rows = rows, a.K = K, a.out = out, a.ld = ldo;
  a.sorted = sorted, a.ntpp = ntpp, a.topk = topk, a.assignments = M * topk;
  return launch(a, dtype, 2, st);
}

}  // namespace chord
