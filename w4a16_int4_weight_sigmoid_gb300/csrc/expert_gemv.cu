// The experts' product in 16 bits for a handful of rows (decoding one token or
// two): out[r, n] = sum_k x[r, k] W[e(r), n, k], without the pairs of SMs.
//
// Bound by the weights' bytes, each used for a few rows, and at this size by
// what comes before and after them: the kernel on pairs of SMs takes about 5 us
// until its first weights arrive and 3 to add up the parts of an item.  Here
// 16-byte loads go out as soon as the counts are known, and partial sums meet in
// shared memory only (the smallest calls 3.5 us against 6.5; one token's 59 MB
// 14.8 against 16.4).
//   * Work: up to eight rows of x of one expert, and of its weight rows a run, of
//     a length that gives every CTA about the same number of runs.  An expert's
//     further rows are further work, for which its weights come from L2;
//   * sixteen warps form 1 to 16 groups, so that a group's warps share K in
//     steps of 256 and meet in shared memory;
//   * one row: dot products.  A lane holds its 8 values of x and walks over 32 of
//     the group's weight rows, eight loads at a time; the lanes' sums of 32 rows
//     are added and spread over the lanes by 31 shuffles.  (Fewer sums a lane and
//     two sets of loads, or rows by bulk copies through shared memory, were
//     slower: 15.6 to 16.2 us);
//   * two to eight rows: a warp's MMAs (m16n8k16) on fragments loaded straight
//     from global memory.  Dot products for two rows at once took 24 us for 16
//     experts of 8 rows each, 83 for 128 rows unevenly on 16 experts (K and N 1024;
//     here 9.2 and 12.5).  For one row the MMAs are faster with long K and N (one
//     token 13.8 against 14.8) and slower with few weights (K 7168, N 64 6.1 / 4.8,
//     K and N 1024 4.0 / 3.6).
// Sums are FP32 in an order that N, K and the counts fix.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.h"

namespace chord {
namespace {

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kStep = 256;             // of K: 8 values a lane
constexpr int kFlight = 8;             // weight rows whose loads go out together
constexpr int kGroupRun = 32;          // weight rows of a run for each group, at most
constexpr int kMaxRows = 8;            // rows of x at once
constexpr int kFewRows = 128;          // largest capacity

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

// A run's sums, [warp of a group][weight row][row of x] with room for kRows of the
// last, added up to `out`.
template <typename T, int kRows>
__device__ __forceinline__ void store_run(const GemvArgs& a, uint16_t* out, int count, int rows, const float* sums) {
  const int share = kWarps >> a.groups_log2, longest = kGroupRun << a.groups_log2;
  __syncthreads();
  for (int i = threadIdx.x; i < count * kRows; i += kThreads) {
    float s = 0.f;
    for (int v = 0; v < share; ++v) s += sums[v * longest * kRows + i];
    T t;
    from_f32(t, s);
    if (i % kRows < rows) out[(i % kRows) * a.ldo + i / kRows] = t.v;
  }
  __syncthreads();
}

// One run: weight rows w .. of `count`, times one row of x, to `out`.
template <typename T>
__device__ __forceinline__ void run_one(const GemvArgs& a, const uint16_t* w, const uint16_t* x, uint16_t* out,
                                        int count, float* sums) {
  constexpr int kBatch = 32;           // weight rows of a group at once
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = 1 << a.groups_log2, share = kWarps >> a.groups_log2;
  const int group = warp / share, part = warp % share;
  const int longest = kGroupRun << a.groups_log2;
  for (int b0 = group * kBatch; b0 < count; b0 += groups * kBatch) {
    float acc[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) acc[i] = 0.f;
    for (int k0 = part * kStep; k0 < a.K; k0 += share * kStep) {
      const int k = k0 + 8 * lane;
      const bool in = k < a.K;         // (K is a multiple of 8)
      float2 xf[4];
      Chunk<16> xc{};
      if (in) load_chunk<16>(x + k, xc);
      unpack<T>(xc, xf);
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
          float2 s = mul2(wf[0], xf[0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) s = fma2(wf[j], xf[j], s);
          acc[i0 + i] += s.x + s.y;
        }
      }
    }
    sums[part * longest + b0 + lane] = spread_sums(acc);
  }
  store_run<T, 1>(a, out, count, 1, sums);
}

// D += A B: 16 weight rows, 16 of K, 8 rows of x.
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if constexpr (std::is_same_v<T, Fp16>)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same for up to eight rows of x.  Lane 4 g + t loads 16 bytes of weight rows g and g + 8 and of row g of x, from
// 8 t of the 32 values of K on: its words are the fragments of two steps, with K
// in another order, the same on both sides.
template <typename T>
__device__ __forceinline__ void run_eight(const GemvArgs& a, const uint16_t* w, const uint16_t* x, uint16_t* out,
                                          int count, int rows, float* sums) {
  constexpr int kTiles = 2, kSteps = 4;    // of 16 weight rows; of 32 of K whose loads go out together
  const int warp = threadIdx.x >> 5, g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  const int groups = 1 << a.groups_log2, share = kWarps >> a.groups_log2;
  const int group = warp / share, part = warp % share;
  const int longest = kGroupRun << a.groups_log2;
  for (int b0 = group * 16 * kTiles; b0 < count; b0 += groups * 16 * kTiles) {
    float acc[kTiles][4] = {};
    for (int k0 = part * kStep; k0 < a.K; k0 += share * kStep) {
#pragma unroll
      for (int h = 0; h < kStep; h += 32 * kSteps) {
        if (k0 + h >= a.K) break;
        Chunk<16> xs[kSteps], ws[kSteps][2 * kTiles];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int k = k0 + h + 32 * i + 8 * t;
          xs[i] = Chunk<16>{};
          if (k < a.K && g < rows) load_chunk<16>(x + g * a.ldx + k, xs[i]);
#pragma unroll
          for (int j = 0; j < 2 * kTiles; ++j) {
            const int n = b0 + 8 * j + g;
            ws[i][j] = Chunk<16>{};
            if (k < a.K && n < count) load_chunk<16>(w + n * a.ldw + k, ws[i][j]);
          }
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int q = 0; q < 4; q += 2)
              mma_16816<T>(acc[j], ws[i][2 * j].w[q], ws[i][2 * j + 1].w[q], ws[i][2 * j].w[q + 1],
                           ws[i][2 * j + 1].w[q + 1], xs[i].w[q], xs[i].w[q + 1]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2 * kTiles; ++j)
      *reinterpret_cast<float2*>(&sums[(part * longest + b0 + 8 * j + g) * kMaxRows + 2 * t]) =
          make_float2(acc[j / 2][2 * (j & 1)], acc[j / 2][2 * (j & 1) + 1]);
  }
  store_run<T, kMaxRows>(a, out, count, rows, sums);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) expert_gemv_kernel(const GemvArgs a) {
  __shared__ int list[kFewRows];       // (expert, first row) of each group of rows
  __shared__ __align__(8) float sums[kWarps * kGroupRun * kMaxRows];
  __shared__ int warp_count[kWarps], bad_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) bad_s = 0;
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  // the groups of rows, experts in order
  int total = 0;
  for (int e0 = 0; e0 < a.E; e0 += kThreads) {
    const int e = e0 + tid;
    int cnt = 0;
    if (e < a.E) {
      cnt = ld_ca(a.counts + e);
      const int off = ld_ca(a.offsets + e), next = ld_ca(a.offsets + e + 1);
      // Experts that end before the next one begins have disjoint rows.
      if (cnt < 0 || off < 0 || cnt > a.capacity || off > a.capacity - cnt || off + cnt > next) bad_s = 1, cnt = 0;
    }
    const int mine = (cnt + kMaxRows - 1) / kMaxRows;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    if (lane == 31) warp_count[warp] = upto;
    __syncthreads();
    int place = total + upto - mine;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      const int c = warp_count[v];
      place += v < warp ? c : 0;
      total += c;
    }
    // (an order of disjoint rows has no more groups than the list; another one is not computed)
    for (int r = 0; r < cnt && place < kFewRows; r += kMaxRows, ++place) list[place] = e << 8 | r;
    __syncthreads();
  }
  if (bad_s) {
    if (tid == 0) set_status(a.status, CHORD_ERR_INVALID_ARG);
    return;
  }
  if (total == 0) return;
  // runs of a length that gives every CTA about the same number, as few as the longest run allows
  const int longest = kGroupRun << a.groups_log2, least = (a.N + longest - 1) / longest;
  const int grid = gridDim.x, turns = (total * least + grid - 1) / grid;   // (total <= 128, least <= 2^15)
  const int per_group = max(min(turns * grid / total, a.N), least);
  const int length = (a.N + per_group - 1) / per_group;
  const int runs = (a.N + length - 1) / length;
  for (int i = blockIdx.x; i < total * runs; i += grid) {
    const int place = i / runs, n0 = (i - place * runs) * length;
    const int e = list[place] >> 8, r = list[place] & 255;
    const int rows = min(kMaxRows, ld_ca(a.counts + e) - r), count = min(length, a.N - n0);
    const long long row = static_cast<long long>(ld_ca(a.offsets + e)) + r;
    const uint16_t* w = a.w + e * a.expert_stride + n0 * a.ldw;
    const uint16_t* x = a.x + row * a.ldx;
    uint16_t* out = a.out + row * a.ldo + n0;
    if (rows == 1) run_one<T>(a, w, x, out, count, sums);
    else run_eight<T>(a, w, x, out, count, rows, sums);
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
// eight to an expert as an order aligned to 8 pads them, and no more experts' runs
// than there are CTAs.  (An order aligned to 16 has 128 rows for one token's 8
// experts, one aligned to 32 or more is past kFewRows: the pairs then.)  Measured
// against the kernel on pairs of SMs, both ways: one token of 8 of 384 experts, K
// 7168, N 512 14.8 us against 16.4, K 256, N 7168 7.7 / 9.0; of 2 of 8 experts, K
// 4096, N 1536 6.8 / 9.4; of one of 16, K and N 1024 3.6 / 6.5; four tokens of 2 of
// 8 experts, K and N 512 4.5 / 5.5.  Orders without padding that the capacity does
// not tell from these, K and N 1024: 128 rows on 16 experts, 8 each 9.2 / 10.1, all
// in one 6.6 / 7.6, uneven (40 to 1) 12.5 / 9.5; one row on each of 128 experts 49.5
// / 43.2; K 2048, N 512, two on each of 64 27.5 / 24.6.  Past it: two tokens of 8 of
// 384, K 7168, N 512 (two runs a CTA) 26.3 / 24.8; one token of 8 of 48, N 4096
// (seven) 82.6 / 71.4.
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
