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
// All bound by memory: one pass over the rows, a row to one warp or more
// (row_lanes).  dweight is added up in FP32 in an order fixed by the call's
// sizes.  Accesses of up to 32 bytes forward and 16 backward, where a value
// needs twice the registers: compiled for three and four CTAs per SM (16384
// rows, I = 2048 BF16, held in 8 bits: forward 45 us against 50 uncapped,
// backward 59 against 84 and, with 32 bytes, 64).  What a pass moves then goes
// at 5.7 to 6.0 TB/s of the 6.8 of a copy; loading a step ahead, or half the
// instructions (two values in one FP32 operation), changed nothing.
#include <cfloat>
#include <utility>

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

// Two gates: silu(g) = max(g, 0) - |g| t / (1 + t) with t = exp(-|g|), which
// loses no digits on either side, and sigmoid(g).  For 16-bit types t is the
// square of exp2(-|g| log2(e) / 2), which stays a normal number where t does
// not, and the fast reciprocal's operand lies in [1, 2].  At the ends silu has its
// limits, infinity and 0: the |g| that t = 0 multiplies is a number there.
template <bool kPrecise>
__device__ __forceinline__ void gates(float2 g, float2& silu, float2& s) {
  const float2 size = make_float2(fabsf(g.x), fabsf(g.y));
  float2 t, d;
  if (kPrecise) {
    t = make_float2(expf(-size.x), expf(-size.y));
    d = make_float2(1.f / (1.f + t.x), 1.f / (1.f + t.y));
  } else {
    const float2 half = mul2(size, make_float2(-0.72134752f, -0.72134752f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(half.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(half.y));
    t = mul2(t, t);
    d = add2(t, make_float2(1.f, 1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d.y) : "f"(d.y));
  }
  const float2 q = mul2(t, d);                              // sigmoid(-|g|)
  silu = fma2(make_float2(-fminf(size.x, FLT_MAX), -fminf(size.y, FLT_MAX)), q,
              make_float2(fmaxf(g.x, 0.f), fmaxf(g.y, 0.f)));
  s = make_float2(g.x < 0.f ? q.x : d.x, g.y < 0.f ? q.y : d.y);
}
// Values i and i + 1 of an array of kN (one: 0 for the second).
template <int kN>
__device__ __forceinline__ float2 two(const float (&f)[kN], int i) {
  return make_float2(f[i], i + 1 < kN ? f[i + 1] : 0.f);
}
template <int kN>
__device__ __forceinline__ void set(float (&f)[kN], int i, float2 v) {
  f[i] = v.x;
  if (i + 1 < kN) f[i + 1] = v.y;
}

// Chunks of a row that a thread has in flight.
constexpr int kUnroll = 2;

template <typename T, int B, bool kKeep>
__global__ void __launch_bounds__(kRowThreads, 3) swiglu_kernel(SwigluArgs a) {
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
          for (int j = 0; j < kN; j += 2) {
            float2 silu, s;
            gates<sizeof(T) == 4>(two(fg, j), silu, s);
            set(fo, j, mul2(mul2(silu, make_float2(w, w)), two(fu, j)));
          }
          f32_chunk<T, B>(o, fo);
        }
        store_chunk<B>(h + c * kN, o);
      }
    }
  }
}

template <typename T, int B, bool kKeep>
__global__ void __launch_bounds__(kRowThreads, 4) swiglu_backward_kernel(SwigluArgs a) {
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
    float2 sum = make_float2(0.f, 0.f);
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
          float dh[kN];
#pragma unroll
          for (int j = 0; j < kN; ++j) dh[j] = chunk_f32<T, B>(ds[i], j);
#pragma unroll
          for (int j = 0; j < kN; j += 2) {
            const float2 ww = make_float2(w, w), d = two(dh, j), up = two(fu, j);
            float2 silu, s;
            gates<sizeof(T) == 4>(two(fg, j), silu, s);
            const float2 act = mul2(silu, up), wd = mul2(ww, d);
            // 1 - s is off by 2^-25, silu times that by less than the slope's own rounding times |gate|; it is 0
            // from a gate of 18 on, where silu's size does not matter (but for an infinity)
            const float2 slope =
                fma2(make_float2(fminf(silu.x, 64.f), fminf(silu.y, 64.f)), make_float2(1.f - s.x, 1.f - s.y), s);
            sum = fma2(d, act, sum);
            set(oh, j, mul2(mul2(silu, ww), up));       // as in the forward pass, whose bits it has
            set(fg, j, mul2(mul2(wd, up), slope));
            set(fu, j, mul2(wd, silu));
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
    float all = sum.x + sum.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (a.lanes > 32) {
      const int warp = threadIdx.x >> 5;
      if ((threadIdx.x & 31) == 0) sums[warp] = all;
      __syncthreads();
      if (lane == 0)
        for (int i = 1; i < a.lanes / 32; ++i) all += sums[warp + i];
      __syncthreads();
    }
    if (lane == 0 && filled) a.dw[f] = all;
  }
}

template <typename T, int B, bool kBackward>
cudaError_t launch(const SwigluArgs& args, cudaStream_t st) {
  SwigluArgs a = args;
  a.lanes = row_lanes(a.rows, a.I / static_cast<int>(B / sizeof(T)), kUnroll);
  const long long per = kRowThreads / a.lanes, want = (a.rows + per - 1) / per, most = 8LL * sm_count();
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  void (*kern)(SwigluArgs);
  if constexpr (kBackward) kern = a.codes ? swiglu_backward_kernel<T, B, true> : swiglu_backward_kernel<T, B, false>;
  else kern = a.codes ? swiglu_kernel<T, B, true> : swiglu_kernel<T, B, false>;
  return launch_kernel(kern, grid, dim3(kRowThreads), 0, st, true, a);
}
// The widest access that all matrices of the call allow.
template <typename T, bool kBackward>
cudaError_t launch(const SwigluArgs& a, cudaStream_t st) {
  int b = kBackward ? 16 : 32;
  for (auto [p, ld] : {std::pair{a.gu, a.ldg}, {a.h, a.ldh}, {a.dh, a.ldd}, {a.dgu, a.ldo}})
    if (p) b = std::min(b, row_access_bytes(p, ld, a.I, sizeof(T), 32));
  switch (b) {
    case 32:
      if constexpr (!kBackward) return launch<T, 32, kBackward>(a, st);
    case 16: return launch<T, 16, kBackward>(a, st);
    case 8: return launch<T, 8, kBackward>(a, st);
    case 4: return launch<T, 4, kBackward>(a, st);
    default:
      if constexpr (sizeof(T) == 2) return launch<T, 2, kBackward>(a, st);
      return cudaErrorInvalidValue;   // (elements are aligned)
  }
}
template <bool kBackward>
cudaError_t launch(const SwigluArgs& a, int dtype, cudaStream_t st) {
  switch (dtype) {
    case CHORD_DTYPE_BF16: return launch<Bf16, kBackward>(a, st);
    case CHORD_DTYPE_FP16: return launch<Fp16, kBackward>(a, st);
    default: return launch<float, kBackward>(a, st);
  }
}

}  // namespace

cudaError_t swiglu_launch(const Swiglu& s, int dtype, bool backward, cudaStream_t st) {
  SwigluArgs a{};
  a.gu = s.gu, a.dh = s.dh, a.w = s.w, a.sorted = s.sorted, a.ntpp = s.ntpp, a.pos = s.pos;
  a.h = s.h, a.dgu = s.dgu, a.codes = s.codes, a.scales = s.scales, a.dw = s.dw;
  a.ldg = s.ldg, a.ldh = s.ldh, a.ldd = s.ldd, a.ldo = s.ldo;
  a.rows = s.rows, a.I = s.I, a.assignments = s.assignments;
  return backward ? launch<true>(a, dtype, st) : launch<false>(a, dtype, st);
}

}  // namespace chord
