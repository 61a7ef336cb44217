// The gated activation between an expert's two products, with the routing
// weight w of the row's assignment on it, over rows in the aligned expert
// order (gate = gu[r, :I], up = gu[r, I:]):
//   forward   h = w silu(gate) up; optionally gu held in 8 bits (MXFP8)
//   backward  dgate = w dh up (s + silu (1 - s)), s = sigmoid(gate)
//             dup = w dh silu(gate)
//             dweight = sum_i dh silu(gate) up
//             h again, where gu comes from its 8 bits
// With w here, the second product's rows are summed back to tokens without
// weights, and its output is not needed for the weights' gradient:
// <dout, W2 h> = <W2^T dout, h>.
// All bound by memory: one pass over the rows, up to 32 bytes an access, a row
// to one warp or more (row_lanes); 1 - s is formed from the exponential of
// -|gate| as s is, so neither loses digits near 1.  dweight is added up in
// FP32 in an order fixed by the call's sizes.
#include "kernels.h"
#include "mxfp8.cuh"

namespace chord {
namespace {

struct SwigluArgs {
  const void* gu;          // [rows, 2 I]; backward: NULL with codes
  const void* dh;          // backward
  const float* w;          // [assignments]
  const int32_t* sorted;
  const int32_t* ntpp;
  const int32_t* pos;      // backward
  void* h;                 // backward: NULL where not asked for
  void* dgu;               // backward
  uint8_t* codes;          // forward: written where not NULL; backward: read
  uint8_t* scales;
  float* dw;               // backward
  long long ldg, ldh, ldd, ldo;   // strides of gu, h, dh, dgu
  int rows, I, assignments, lanes;
};

// s = sigmoid(g) and 1 - s.
template <bool kPrecise>
__device__ __forceinline__ void sigmoids(float g, float& s, float& rest) {
  const float t = kPrecise ? expf(-fabsf(g)) : __expf(-fabsf(g));   // at most 1
  const float d = kPrecise ? 1.f / (1.f + t) : __fdividef(1.f, 1.f + t);
  s = g < 0.f ? t * d : d;
  rest = g < 0.f ? d : t * d;
}

// Chunks of a row that a thread has in flight.
constexpr int kUnroll = 2;

template <typename T, int B, bool kKeep>
__global__ void __launch_bounds__(kRowThreads) swiglu_kernel(SwigluArgs a) {
  constexpr int kN = B / sizeof(T);
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x % a.lanes, per = kRowThreads / a.lanes, step = gridDim.x * per;
  const int chunks = a.I / kN, total = min(a.rows, ld_ca(a.ntpp));
  // (the row of a warp is the same for all its lanes)
  for (int r = blockIdx.x * per + threadIdx.x / a.lanes; r < total; r += step) {
    const int f = ld_ca(a.sorted + r);
    const bool filled = f >= 0 && f < a.assignments;
    const float w = filled ? ld_ca(a.w + f) : 0.f;
    const T* gu = static_cast<const T*>(a.gu) + r * a.ldg;
    T* h = static_cast<T*>(a.h) + r * a.ldh;
    for (int c0 = lane; c0 - (lane & 31) < chunks; c0 += kUnroll * a.lanes) {
      Chunk<B> gs[kUnroll], us[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + i * a.lanes;
        gs[i] = us[i] = Chunk<B>{};
        if (c < chunks && filled) {
          load_chunk<B>(gu + c * kN, gs[i]);
          load_chunk<B>(gu + a.I + c * kN, us[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + i * a.lanes;
        if (i > 0 && c - (lane & 31) >= chunks) break;
        const Chunk<B>&g = gs[i], &u = us[i];
        float fg[kN], fu[kN], fo[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) fg[j] = chunk_f32<T, B>(g, j), fu[j] = chunk_f32<T, B>(u, j);
        if constexpr (kKeep) {
          const uint32_t sg = block_scale(block_top<T, B>(g)), su = block_scale(block_top<T, B>(u));
          uint32_t code[kN < 4 ? 1 : kN / 4];
          if (c < chunks) {
            uint8_t* codes = a.codes + static_cast<long long>(r) * 2 * a.I + c * kN;
            to_codes<kN>(fg, sg, code);
            store_codes<kN>(codes, code);
            to_codes<kN>(fu, su, code);
            store_codes<kN>(codes + a.I, code);
            if ((c * kN) % kMx8Block == 0) {
              uint8_t* scales = a.scales + static_cast<long long>(r) * (2 * a.I / kMx8Block) + c * kN / kMx8Block;
              scales[0] = static_cast<uint8_t>(sg);
              scales[a.I / kMx8Block] = static_cast<uint8_t>(su);
            }
          }
        }
        if (c >= chunks) continue;
        Chunk<B> o{};
        if (filled) {
#pragma unroll
          for (int j = 0; j < kN; ++j) {
            float s, rest;
            sigmoids<sizeof(T) == 4>(fg[j], s, rest);
            fo[j] = w * (fg[j] * s) * fu[j];
          }
          f32_chunk<T, B>(o, fo);
        }
        store_chunk<B>(h + c * kN, o);
      }
    }
  }
}

template <typename T, int B, bool kKeep>
__global__ void __launch_bounds__(kRowThreads) swiglu_backward_kernel(SwigluArgs a) {
  constexpr int kN = B / sizeof(T), kW = kN < 4 ? 1 : kN / 4;
  __shared__ float sums[kRowThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  // assignments without a row here
  for (int f = blockIdx.x * kRowThreads + threadIdx.x; f < a.assignments; f += gridDim.x * kRowThreads) {
    const int p = ld_ca(a.pos + f);
    if (p < 0 || p >= a.rows) a.dw[f] = 0.f;
  }
  const int lane = threadIdx.x % a.lanes, per = kRowThreads / a.lanes, step = gridDim.x * per;
  const int chunks = a.I / kN, total = min(a.rows, ld_ca(a.ntpp));
  for (int r0 = blockIdx.x * per; r0 < total; r0 += step) {   // (the same for all threads)
    const int r = r0 + threadIdx.x / a.lanes;
    const int f = r < total ? ld_ca(a.sorted + r) : -1;
    const bool filled = f >= 0 && f < a.assignments;
    const float w = filled ? ld_ca(a.w + f) : 0.f;
    const long long row = r;
    float sum = 0.f;
    for (int c0 = r < total ? lane : chunks; c0 < chunks; c0 += kUnroll * a.lanes) {
      Chunk<B> ds[kUnroll], xs[kKeep ? 1 : kUnroll], ys[kKeep ? 1 : kUnroll];
      uint32_t cg[kKeep ? kUnroll : 1][kW], cu[kKeep ? kUnroll : 1][kW], sg[kUnroll], su[kUnroll];
      if (filled) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int c = min(c0 + i * a.lanes, chunks - 1);
          load_chunk<B>(static_cast<const T*>(a.dh) + row * a.ldd + c * kN, ds[i]);
          if constexpr (kKeep) {
            const uint8_t* codes = a.codes + row * 2 * a.I + c * kN;
            const uint8_t* scales = a.scales + row * (2 * a.I / kMx8Block) + c * kN / kMx8Block;
            load_codes<kN>(codes, cg[i]);
            load_codes<kN>(codes + a.I, cu[i]);
            sg[i] = load_scale(scales);
            su[i] = load_scale(scales + a.I / kMx8Block);
          } else {
            const T* gu = static_cast<const T*>(a.gu) + row * a.ldg + c * kN;
            load_chunk<B>(gu, xs[i]);
            load_chunk<B>(gu + a.I, ys[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int c = c0 + i * a.lanes;
        if (c >= chunks) break;
        Chunk<B> x{}, y{}, o{};
        if (filled) {
          float fg[kN], fu[kN], oh[kN];
          if constexpr (kKeep) {
            from_codes<kN>(cg[i], scale_value(sg[i]), fg);
            from_codes<kN>(cu[i], scale_value(su[i]), fu);
          } else {
#pragma unroll
            for (int j = 0; j < kN; ++j) fg[j] = chunk_f32<T, B>(xs[i], j), fu[j] = chunk_f32<T, B>(ys[i], j);
          }
#pragma unroll
          for (int j = 0; j < kN; ++j) {
            float s, rest;
            sigmoids<sizeof(T) == 4>(fg[j], s, rest);
            const float silu = fg[j] * s, dh = chunk_f32<T, B>(ds[i], j), wd = w * dh, up = fu[j];
            sum += dh * silu * up;
            oh[j] = w * silu * up;
            fg[j] = wd * up * (s + silu * rest);
            fu[j] = wd * silu;
          }
          f32_chunk<T, B>(x, fg);
          f32_chunk<T, B>(y, fu);
          f32_chunk<T, B>(o, oh);
        }
        T* dgu = static_cast<T*>(a.dgu) + row * a.ldo + c * kN;
        store_chunk<B>(dgu, x);
        store_chunk<B>(dgu + a.I, y);
        if (a.h) store_chunk<B>(static_cast<T*>(a.h) + row * a.ldh + c * kN, o);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (a.lanes > 32) {
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) sums[warp] = sum;
      __syncthreads();
      if (lane == 0)
        for (int i = 1; i < a.lanes / 32; ++i) sum += sums[warp + i];
      __syncthreads();
    }
    if (lane == 0 && filled) a.dw[f] = sum;
  }
}

template <typename T, int B>
cudaError_t launch(const SwigluArgs& args, bool backward, cudaStream_t st) {
  SwigluArgs a = args;
  a.lanes = row_lanes(a.rows, a.I / static_cast<int>(B / sizeof(T)), kUnroll);
  const long long per = kRowThreads / a.lanes, want = (a.rows + per - 1) / per, most = 32LL * sm_count();
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  auto kern = backward ? (a.codes ? swiglu_backward_kernel<T, B, true> : swiglu_backward_kernel<T, B, false>)
                       : (a.codes ? swiglu_kernel<T, B, true> : swiglu_kernel<T, B, false>);
  return launch_kernel(kern, grid, dim3(kRowThreads), 0, st, true, a);
}
// The widest access that all matrices of the call allow.
template <typename T>
cudaError_t launch(const SwigluArgs& a, bool backward, cudaStream_t st) {
  int b = 32;
  auto allow = [&](const void* p, long long ld) { b = std::min(b, p ? row_access_bytes(p, ld, a.I, sizeof(T), 32) : 32); };
  allow(a.gu, a.ldg), allow(a.h, a.ldh), allow(a.dh, a.ldd), allow(a.dgu, a.ldo);
  switch (b) {
    case 32: return launch<T, 32>(a, backward, st);
    case 16: return launch<T, 16>(a, backward, st);
    case 8: return launch<T, 8>(a, backward, st);
    case 4: return launch<T, 4>(a, backward, st);
    default:
      if constexpr (sizeof(T) == 2) return launch<T, 2>(a, backward, st);
      return cudaErrorInvalidValue;   // (elements are aligned)
  }
}
cudaError_t launch(const SwigluArgs& a, int dtype, bool backward, cudaStream_t st) {
  switch (dtype) {
    case CHORD_DTYPE_BF16: return launch<Bf16>(a, backward, st);
    case CHORD_DTYPE_FP16: return launch<Fp16>(a, backward, st);
    default: return launch<float>(a, backward, st);
  }
}

}  // namespace

cudaError_t swiglu_launch(const Swiglu& s, int dtype, bool backward, cudaStream_t st) {
  SwigluArgs a{};
  a.gu = s.gu, a.dh = s.dh, a.w = s.w, a.sorted = s.sorted, a.ntpp = s.ntpp, a.pos = s.pos;
  a.h = s.h, a.dgu = s.dgu, a.codes = s.codes, a.scales = s.scales, a.dw = s.dw;
  a.ldg = s.ldg, a.ldh = s.ldh, a.ldd = s.ldd, a.ldo = s.ldo;
  a.rows = s.rows, a.I = s.I, a.assignments = s.assignments;
  return launch(a, dtype, backward, st);
}

}  // namespace chord
