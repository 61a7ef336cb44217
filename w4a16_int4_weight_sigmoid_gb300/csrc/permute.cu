// Token rows into the aligned expert order and back, and the gradient of
// both.  p(t, j) = sorted_positions[t * topk + j] is the row of assignment
// (t, j), or negative when its expert is not local:
//   permute            out[p(t, j)] = x[t]; padding rows are zeros
//   permute_backward   dx[t] = sum_j dout[p(t, j)]
//   unpermute          out[t] = sum_j w[t, j] y[p(t, j)]
//   unpermute_backward dy[p(t, j)] = w[t, j] dout[t]; padding rows are zeros;
//                      dw[t, j] = <dout[t], y[p(t, j)]>, 0 where not local
// All four move rows and do next to no arithmetic, so they are bound by
// memory: every kernel is token-major, which reads a token's row once
// whatever the number of its experts.  Sums are FP32 in increasing j (the
// weight gradient: FP32 in a fixed tree), each result rounded once, so
// results do not depend on the launch.
//
// Rows are moved in accesses of V elements.  V is 16 bytes where every base,
// row stride and row length allows it; otherwise the largest power of two
// they share, down to one element.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"

namespace chord {
namespace {

constexpr int kMaxTopk = 32;

struct RowArgs {
  const void* x;            // token rows [M, H]
  const void* y;            // expert rows [capacity, H]
  const float* w;           // [M, topk]
  const int32_t* pos;       // [M * topk]
  const int32_t* sorted;    // [capacity]
  const int32_t* ntpp;
  void* out;                // rows written
  float* dw;                // [M, topk]
  long long ldx, ldy, ldo;
  int M, topk, H, rows;     // rows: capacity of the expert order
};

// ------------------------------------------------------------ padding rows
// Zeros in the padding rows (sorted >= M * topk) of the aligned order: CTA b
// of nb takes every nb-th run of kPadRows rows below the padded total.
constexpr int kPadRows = 16;

template <typename T, int V>
__device__ __forceinline__ void zero_padding(const RowArgs& a, int b, int nb) {
  const int n = min(__ldg(a.ntpp), a.rows), sentinel = a.M * a.topk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  Vec<T, V> z;
#pragma unroll
  for (int i = 0; i < V; ++i) from_f32(z.e[i], 0.f);
  for (int r0 = b * kPadRows; r0 < n; r0 += nb * kPadRows)
    for (int r = r0 + warp; r < min(n, r0 + kPadRows); r += warps) {
      if (__ldg(a.sorted + r) < sentinel) continue;
      auto* dst = reinterpret_cast<Vec<T, V>*>(static_cast<T*>(a.out) + r * a.ldo);
      for (int c = lane; c < a.H / V; c += 32) dst[c] = z;
    }
}

// ----------------------------------------------------------------- permute
// CTA (t, chunk) below the padding CTAs: VPT accesses of each thread of
// token t's row are loaded, then stored to each of its rows.
template <typename T, int V, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS) permute_kernel(RowArgs a, int pad_ctas) {
  if (static_cast<int>(blockIdx.x) < pad_ctas) {
    if (blockIdx.y == 0) zero_padding<T, V>(a, blockIdx.x, pad_ctas);
    return;
  }
  const int t = blockIdx.x - pad_ctas, lane = threadIdx.x & 31;
  int p = -1;
  if (lane < a.topk) p = __ldg(a.pos + static_cast<long long>(t) * a.topk + lane);
  if (p >= a.rows) p = -1;
  const uint32_t local = __ballot_sync(0xffffffffu, p >= 0);
  if (!local) return;
  const int nv = a.H / V, c0 = blockIdx.y * THREADS * VPT + threadIdx.x;
  const auto* src = reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(a.x) + t * a.ldx);
  Vec<T, V> v[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (c0 + i * THREADS < nv) v[i] = src[c0 + i * THREADS];
  for (uint32_t left = local; left; left &= left - 1) {
    const long long row = __shfl_sync(0xffffffffu, p, __ffs(left) - 1);
    auto* dst = reinterpret_cast<Vec<T, V>*>(static_cast<T*>(a.out) + row * a.ldo);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (c0 + i * THREADS < nv) dst[c0 + i * THREADS] = v[i];
  }
}

// ---------------------------------------------------- weighted sum of rows
// CTA (t, chunk): VPT accesses per thread of the token's local rows, ROWS
// rows in flight, added in increasing j.
template <typename T, int V, int VPT, int THREADS, bool kWeighted>
__global__ void __launch_bounds__(THREADS) combine_kernel(RowArgs a) {
  constexpr int kRows = VPT >= 4 ? 2 : 4;
  __shared__ int s_pos[kMaxTopk];
  __shared__ float s_w[kMaxTopk];
  __shared__ int s_n;
  const int t = blockIdx.x, tid = threadIdx.x;
  if (tid < 32) {
    int p = -1;
    float wj = 1.f;
    if (tid < a.topk) {
      const long long o = static_cast<long long>(t) * a.topk + tid;
      p = __ldg(a.pos + o);
      if (kWeighted) wj = __ldg(a.w + o);
    }
    if (p >= a.rows) p = -1;
    const uint32_t local = __ballot_sync(0xffffffffu, p >= 0);
    if (p >= 0) {
      const int k = __popc(local & ((1u << tid) - 1u));
      s_pos[k] = p;
      s_w[k] = wj;
    }
    if (tid == 0) s_n = __popc(local);
  }
  __syncthreads();
  const int n = s_n, nv = a.H / V, c0 = blockIdx.y * THREADS * VPT + tid;
  float acc[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) acc[i][e] = 0.f;
  for (int j0 = 0; j0 < n; j0 += kRows) {
    Vec<T, V> v[kRows][VPT];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (j0 + r < n) {
        const auto* src = reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(a.y) + s_pos[j0 + r] * a.ldy);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (c0 + i * THREADS < nv) v[r][i] = src[c0 + i * THREADS];
      }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (j0 + r < n) {
        const float wj = s_w[j0 + r];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (c0 + i * THREADS < nv)
#pragma unroll
            for (int e = 0; e < V; ++e)
              acc[i][e] = kWeighted ? fmaf(wj, to_f32(v[r][i].e[e]), acc[i][e]) : acc[i][e] + to_f32(v[r][i].e[e]);
      }
  }
  auto* dst = reinterpret_cast<Vec<T, V>*>(static_cast<T*>(a.out) + t * a.ldo);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (c0 + i * THREADS < nv) {
      Vec<T, V> o;
#pragma unroll
      for (int e = 0; e < V; ++e) from_f32(o.e[e], acc[i][e]);
      dst[c0 + i * THREADS] = o;
    }
}

// ------------------------------------------------- gradient of the weighted sum
// CTA (t, s) below the padding CTAs: assignments j = s, s + S, ... of token t
// (S = gridDim.y).  One pass over dout[t] and y[p] gives both dy[p] and the
// dot product; dout[t] comes from L1 for every j after the first.
template <typename T, int V, int THREADS>
__global__ void __launch_bounds__(THREADS) unpermute_backward_kernel(RowArgs a, int pad_ctas) {
  if (static_cast<int>(blockIdx.x) < pad_ctas) {
    if (blockIdx.y == 0) zero_padding<T, V>(a, blockIdx.x, pad_ctas);
    return;
  }
  constexpr int kUnroll = 4;
  __shared__ float s_part[kMaxTopk][THREADS / 32];
  const int t = blockIdx.x - pad_ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nv = a.H / V;
  const auto* g = reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(a.x) + t * a.ldx);
  for (int j = blockIdx.y; j < a.topk; j += gridDim.y) {
    const long long f = static_cast<long long>(t) * a.topk + j;
    const int p = __ldg(a.pos + f);
    float dot = 0.f;
    if (p >= 0 && p < a.rows) {
      const float wj = __ldg(a.w + f);
      const auto* y = reinterpret_cast<const Vec<T, V>*>(static_cast<const T*>(a.y) + p * a.ldy);
      auto* dy = reinterpret_cast<Vec<T, V>*>(static_cast<T*>(a.out) + p * a.ldo);
      for (int c0 = tid; c0 < nv; c0 += kUnroll * THREADS) {
        Vec<T, V> vg[kUnroll], vy[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
          if (c0 + i * THREADS < nv) {
            vg[i] = g[c0 + i * THREADS];
            vy[i] = y[c0 + i * THREADS];
          }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
          if (c0 + i * THREADS < nv) {
            Vec<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float gv = to_f32(vg[i].e[e]);
              dot = fmaf(gv, to_f32(vy[i].e[e]), dot);
              from_f32(o.e[e], wj * gv);
            }
            dy[c0 + i * THREADS] = o;
          }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_part[j][warp] = dot;
  }
  __syncthreads();
  for (int j = blockIdx.y + tid * gridDim.y; j < a.topk; j += THREADS * gridDim.y) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) sum += s_part[j][i];
    a.dw[static_cast<long long>(t) * a.topk + j] = sum;
  }
}

int sm_count() {
  static int sms[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if (!sms[dev]) cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
  return sms[dev] > 0 ? sms[dev] : 1;
}

constexpr int kThreads = 128;

// CTAs for the padding rows: enough for every run, at most one per SM.
int padding_ctas(int rows) { return std::min((rows + kPadRows - 1) / kPadRows, sm_count()); }

enum class Op { kPermute, kPermuteBackward, kUnpermute, kUnpermuteBackward };

template <typename T, int V>
cudaError_t launch_rows(Op op, const RowArgs& a, cudaStream_t st) {
  const int nv = a.H / V;
  // accesses per thread: a whole row per CTA where there are at least four
  // CTAs per SM, otherwise smaller chunks
  auto chunks = [&](int vpt) { return (nv + kThreads * vpt - 1) / (kThreads * vpt); };
  int vpt = 8;
  while (vpt > 1 && static_cast<long long>(a.M) * chunks(vpt) < 4LL * sm_count()) vpt /= 2;
  if (op == Op::kPermute) {
    const int pad = padding_ctas(a.rows);
    const dim3 grid(a.M + pad, chunks(vpt));
    switch (vpt) {
      case 8: permute_kernel<T, V, 8, kThreads><<<grid, kThreads, 0, st>>>(a, pad); break;
      case 4: permute_kernel<T, V, 4, kThreads><<<grid, kThreads, 0, st>>>(a, pad); break;
      case 2: permute_kernel<T, V, 2, kThreads><<<grid, kThreads, 0, st>>>(a, pad); break;
      default: permute_kernel<T, V, 1, kThreads><<<grid, kThreads, 0, st>>>(a, pad);
    }
  } else if (op == Op::kUnpermuteBackward) {
    const int pad = padding_ctas(a.rows);
    int split = 1;
    while (split < a.topk && static_cast<long long>(a.M) * split < 4LL * sm_count()) split *= 2;
    unpermute_backward_kernel<T, V, kThreads><<<dim3(a.M + pad, std::min(split, a.topk)), kThreads, 0, st>>>(a, pad);
  } else {
    const dim3 grid(a.M, chunks(vpt));
    const bool w = op == Op::kUnpermute;
    switch (vpt) {
      case 8:
        if (w) combine_kernel<T, V, 8, kThreads, true><<<grid, kThreads, 0, st>>>(a);
        else combine_kernel<T, V, 8, kThreads, false><<<grid, kThreads, 0, st>>>(a);
        break;
      case 4:
        if (w) combine_kernel<T, V, 4, kThreads, true><<<grid, kThreads, 0, st>>>(a);
        else combine_kernel<T, V, 4, kThreads, false><<<grid, kThreads, 0, st>>>(a);
        break;
      case 2:
        if (w) combine_kernel<T, V, 2, kThreads, true><<<grid, kThreads, 0, st>>>(a);
        else combine_kernel<T, V, 2, kThreads, false><<<grid, kThreads, 0, st>>>(a);
        break;
      default:
        if (w) combine_kernel<T, V, 1, kThreads, true><<<grid, kThreads, 0, st>>>(a);
        else combine_kernel<T, V, 1, kThreads, false><<<grid, kThreads, 0, st>>>(a);
    }
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_access(Op op, const RowArgs& a, int bytes, cudaStream_t st) {
  constexpr int kE = sizeof(T);
  switch (bytes / kE) {
    case 16 / kE: return launch_rows<T, 16 / kE>(op, a, st);
    case 8 / kE: return launch_rows<T, 8 / kE>(op, a, st);
    case 4 / kE: return launch_rows<T, 4 / kE>(op, a, st);
    default: return launch_rows<T, 1>(op, a, st);
  }
}

cudaError_t launch_dtype(Op op, const RowArgs& a, int dtype, cudaStream_t st) {
  const size_t es = dtype_bytes(dtype);
  int bytes = row_access_bytes(a.out, a.ldo, a.H, es);
  if (a.x) bytes = std::min(bytes, row_access_bytes(a.x, a.ldx, a.H, es));
  if (a.y) bytes = std::min(bytes, row_access_bytes(a.y, a.ldy, a.H, es));
  if (dtype == CHORD_DTYPE_BF16) return launch_access<Bf16>(op, a, bytes, st);
  if (dtype == CHORD_DTYPE_FP16) return launch_access<Fp16>(op, a, bytes, st);
  return launch_access<float>(op, a, bytes, st);
}

}  // namespace

cudaError_t moe_permute_launch(const void* x, int dtype, long long ldx, const int32_t* pos, const int32_t* sorted,
                               const int32_t* ntpp, int M, int topk, int H, int rows, void* out, long long ldo,
                               cudaStream_t st) {
  RowArgs a{};
  a.x = x, a.ldx = ldx, a.pos = pos, a.sorted = sorted, a.ntpp = ntpp, a.out = out, a.ldo = ldo;
  a.M = M, a.topk = topk, a.H = H, a.rows = rows;
  return launch_dtype(Op::kPermute, a, dtype, st);
}

cudaError_t moe_combine_launch(const void* y, int dtype, long long ldy, const float* w, const int32_t* pos, int M,
                               int topk, int H, int rows, void* out, long long ldo, cudaStream_t st) {
  RowArgs a{};
  a.y = y, a.ldy = ldy, a.w = w, a.pos = pos, a.out = out, a.ldo = ldo;
  a.M = M, a.topk = topk, a.H = H, a.rows = rows;
  return launch_dtype(w ? Op::kUnpermute : Op::kPermuteBackward, a, dtype, st);
}

cudaError_t moe_unpermute_backward_launch(const void* dout, const void* y, int dtype, long long ldd, long long ldy,
                                          const float* w, const int32_t* pos, const int32_t* sorted,
                                          const int32_t* ntpp, int M, int topk, int H, int rows, void* dy,
                                          long long ldo, float* dw, cudaStream_t st) {
  RowArgs a{};
  a.x = dout, a.ldx = ldd, a.y = y, a.ldy = ldy, a.w = w, a.pos = pos, a.sorted = sorted, a.ntpp = ntpp;
  a.out = dy, a.ldo = ldo, a.dw = dw, a.M = M, a.topk = topk, a.H = H, a.rows = rows;
  return launch_dtype(Op::kUnpermuteBackward, a, dtype, st);
}

}  // namespace chord
