// The experts' product in 16 bits for a handful of rows (decoding one token or
// two): out[r, n] = sum_k x[r, k] W[e(r), n, k] as dot products, without the
// tensor cores.
//
// Bound by the weights' bytes, each used for one or two rows, and at this size
// by what comes before and after them: the kernel on pairs of SMs takes about
// 5 us until its first weights arrive and 3 to add up the parts of an item.
// Here 16-byte loads go out as soon as the counts are known, and partial sums
// meet in shared memory only (the smallest calls 3.5 us against 7; one token's
// 59 MB 14.8 against 16.4).
//   * Work: the weight rows of all experts that have rows, in runs of one
//     expert, of a length that gives every CTA about one;
//   * sixteen warps form 1 to 16 groups, so that a group's warps share K in
//     steps of 256; a lane holds its 8 values of x and walks over 32 of the
//     group's weight rows, eight loads at a time.  (Fewer sums a lane and two
//     sets of loads, or rows by bulk copies through shared memory, were slower:
//     15.6 to 16.2 us);
//   * the lanes' sums of 32 rows are added and spread over the lanes by 31
//     shuffles; a group's warps meet in shared memory.
// Two rows of x are taken at once; an expert with more takes several passes over
// its weights (from L2).  Sums are FP32 in an order fixed by N, K and the counts.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"

namespace chord {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kStep = 256;             // of K: 8 values a lane
constexpr int kFlight = 8;             // weight rows whose loads go out together
constexpr int kGroupRun = 32;          // weight rows of a run for each group, at most
constexpr int kMaxRows = 2;            // rows of x at once
constexpr int kMaxExperts = 1024;

struct GemvArgs {
  const uint16_t* x;
  const uint16_t* w;
  const int32_t* counts;
  const int32_t* offsets;
  uint16_t* out;
  int* status;
  long long ldx, ldw, expert_stride, ldo;
  int E, N, K, capacity;
  int groups_log2;       // 16 warps in groups of as many as share K
};

template <typename T>
__device__ __forceinline__ void unpack(const Chunk<16>& c, float2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(chunk_f32<T, 16>(c, 2 * i), chunk_f32<T, 16>(c, 2 * i + 1));
}

// 32 values a lane -> lane l has the sum over the lanes of value l: at each
// step a lane keeps half of its values and adds what its partner had of them.
__device__ __forceinline__ float spread_sums(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 16; half; half >>= 1) {
    const bool upper = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, half);
    }
  }
  return v[0];
}

// One run: weight rows w .. of `count`, times kRows rows of x, to `out`.
template <typename T, int kRows>
__device__ __forceinline__ void run_rows(const GemvArgs& a, const uint16_t* w, const uint16_t* x, uint16_t* out,
                                         int count, float* sums) {
  constexpr int kBatch = 32 / kRows;   // weight rows of a group at once
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = 1 << a.groups_log2, share = kWarps >> a.groups_log2;
  const int group = warp / share, part = warp % share;
  const int longest = kGroupRun << a.groups_log2;
  for (int b0 = group * kBatch; b0 < count; b0 += groups * kBatch) {
    float acc[32];                     // [weight row][row of x]
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = 0.f;
    for (int k0 = part * kStep; k0 < a.K; k0 += share * kStep) {
      const int k = k0 + 8 * lane;
      const bool in = k < a.K;         // (K is a multiple of 8)
      float2 xf[kRows][4];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        Chunk<16> c{};
        if (in) load_chunk<16>(x + r * a.ldx + k, c);
        unpack<T>(c, xf[r]);
      }
#pragma unroll
      for (int i0 = 0; i0 < kBatch; i0 += kFlight) {
        if (b0 + i0 >= count) break;
        Chunk<16> c[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          c[i] = Chunk<16>{};
          if (in && b0 + i0 + i < count) load_chunk<16>(w + (b0 + i0 + i) * a.ldw + k, c[i]);
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          float2 wf[4];
          unpack<T>(c[i], wf);
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            float2 s = mul2(wf[0], xf[r][0]);
#pragma unroll
            for (int j = 1; j < 4; ++j) s = fma2(wf[j], xf[r][j], s);
            acc[(i0 + i) * kRows + r] += s.x + s.y;
          }
        }
      }
    }
    sums[(part * longest + b0) * kRows + lane] = spread_sums(acc);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < count * kRows; i += kThreads) {
    float s = 0.f;
    for (int v = 0; v < share; ++v) s += sums[v * longest * kRows + i];
    T t;
    from_f32(t, s);
    out[(i % kRows) * a.ldo + i / kRows] = t.v;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) expert_gemv_kernel(const GemvArgs a) {
  __shared__ int list[kMaxExperts];    // experts with rows
  __shared__ float sums[kWarps * kGroupRun * kMaxRows];
  __shared__ int warp_count[kWarps], bad_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) bad_s = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  // the experts with rows, in order
  int total = 0;
  for (int e0 = 0; e0 < a.E; e0 += kThreads) {
    const int e = e0 + tid;
    int cnt = 0;
    if (e < a.E) {
      cnt = ld_ca(a.counts + e);
      const int off = ld_ca(a.offsets + e), next = ld_ca(a.offsets + e + 1);
      // Experts that end before the next one begins have disjoint rows.
      if (cnt < 0 || off < 0 || cnt > a.capacity || off > a.capacity - cnt || off + cnt > next) bad_s = 1;
    }
    const uint32_t with = __ballot_sync(0xffffffffu, cnt > 0);
    if (lane == 0) warp_count[warp] = __popc(with);
    __syncthreads();
    int before = total;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      const int c = warp_count[v];
      before += v < warp ? c : 0;
      total += c;
    }
    if (cnt > 0) list[before + __popc(with & ((1u << lane) - 1u))] = e;
    __syncthreads();
  }
  if (bad_s) {
    if (tid == 0) set_status(a.status, CHORD_ERR_INVALID_ARG);
    return;
  }
  if (total == 0) return;
  // runs of a length that gives every CTA about one, or the longest
  const int longest = kGroupRun << a.groups_log2;
  const int per_expert = max(static_cast<int>(gridDim.x) / total, (a.N + longest - 1) / longest);
  const int length = (a.N + per_expert - 1) / per_expert;
  const int runs = (a.N + length - 1) / length;
  for (long long i = blockIdx.x; i < static_cast<long long>(total) * runs; i += gridDim.x) {
    const int place = static_cast<int>(i / runs), n0 = static_cast<int>(i - static_cast<long long>(place) * runs) * length;
    const int e = list[place], cnt = ld_ca(a.counts + e), count = min(length, a.N - n0);
    const long long row0 = ld_ca(a.offsets + e);
    const uint16_t* w = a.w + e * a.expert_stride + n0 * a.ldw;
    const uint16_t* x = a.x + row0 * a.ldx;
    uint16_t* out = a.out + row0 * a.ldo + n0;
    int r = 0;
    for (; r + 2 <= cnt; r += 2) run_rows<T, 2>(a, w, x + r * a.ldx, out + r * a.ldo, count, sums);
    if (r < cnt) run_rows<T, 1>(a, w, x + r * a.ldx, out + r * a.ldo, count, sums);
  }
}

}  // namespace

namespace {
// Groups for a K: 16 warps over the steps of 256.
int groups_log2(int K) {
  int g = 4;
  while (g > 0 && (kWarps >> g) * kStep < K) --g;
  return g;
}
}  // namespace

// The host knows the capacity, not the counts: at most kFewRows rows, about
// eight to an expert as an aligned order pads them, and no more experts' runs
// than there are CTAs.  Measured against the kernel on pairs of SMs, both ways:
// one token of 8 of 384 experts, K 7168, N 512 14.8 us against 16.4, K 256, N
// 7168 7.9 / 9.0; of 2 of 8 experts, K 4096, N 1536 6.3 / 9.4; of one of 16, K
// and N 1024 3.5 / 7.1; four tokens of 2 of 8 experts, K and N 512 4.4 / 6.0.
// Past it: two tokens of 8 of 384, K 7168, N 512 (two runs a CTA) 26.3 / 24.8;
// one token of 8 of 48, N 4096 (seven) 82.6 / 71.4; sixteen tokens of 2 of 8, K
// 4096, N 1536 (eight rows an expert) 50.7 / 21.0.
constexpr int kFewRows = 128;
bool expert_gemv_serves(const ExpertGemm& g) {
  if (g.capacity > kFewRows || g.capacity > 8 * g.E) return false;
  const int longest = kGroupRun << groups_log2(g.K), runs = (g.N + longest - 1) / longest;
  const int experts = std::min(g.E, (g.capacity + 7) / 8);
  return static_cast<long long>(experts) * runs <= sm_count();
}

cudaError_t expert_gemv_launch(const ExpertGemm& g, cudaStream_t st) {
  GemvArgs a{};
  a.x = static_cast<const uint16_t*>(g.x), a.w = static_cast<const uint16_t*>(g.w);
  a.counts = g.counts, a.offsets = g.offsets, a.out = static_cast<uint16_t*>(g.out), a.status = g.status;
  a.ldx = g.ldx, a.ldw = g.ldw, a.expert_stride = g.expert_stride, a.ldo = g.ldo;
  a.E = g.E, a.N = g.N, a.K = g.K, a.capacity = g.capacity;
  a.groups_log2 = groups_log2(g.K);
  return launch_kernel(g.f16 ? expert_gemv_kernel<Fp16> : expert_gemv_kernel<Bf16>, dim3(sm_count()), dim3(kThreads), 0,
                       st, true, a);
}

}  // namespace chord
