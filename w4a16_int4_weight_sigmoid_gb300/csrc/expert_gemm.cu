// The experts' product in 16 bits and its gradients, on pairs of SMs:
//   product      out[r, n] = sum_k x[r, k] W[e(r), n, k]
//   transposed   out[r, k] = sum_n x[r, n] W[e(r), n, k]     (the rows' gradient)
//   gradient     dW[e, n, k] = sum_{r of e} dout[r, n] x[r, k]
// over rows in expert order: expert e's rows are counts[e] rows from
// offsets[e] on, of any number, read on the device.
//
// Design on sm_103a (one persistent CTA per SM, two to a cluster):
//   * the MMA is M = 256 over the pair (cta_group::2).  M is the weights' side
//     (product: 256 weight rows times up to 256 of an expert's rows, a
//     multiple of 32; gradient: 256 x 256 of an expert's dW), so an expert of
//     few rows costs 32 columns, not 256 rows;
//   * each CTA loads half of A and half of B per 64 of the contraction, 32 KB
//     at most for 512 cycles of MMA; one CTA alone would need 48;
//   * the transposed product reads the same weights with their M index
//     contiguous, and the gradient reads both operands so: only the TMA boxes
//     and the descriptors differ;
//   * an item is one output tile; clusters take items in turn, so that those
//     at work at one time share weights and rows in L2.  With few rows (up to
//     kSplitTok to a tile) the items that do not divide evenly among the
//     clusters come first and are cut along the contraction, a part to a
//     cluster; the CTA that arrives last at its half of an item adds the parts
//     in order, so results do not depend on timing;
//   * a product's stage of the ring holds 128 of the contraction: with few rows
//     a stage's hand-offs, not its bytes, set the pace (one token, 64 to a stage:
//     18.6 us against 17.3; many rows 612 against 600);
//   * one warp per CTA loads, one (of the leading CTA) issues MMAs, one decodes
//     items for the others, eight store finished tiles from one accumulator
//     while the next is filled;
//   * product tiles have weights in lanes and rows in columns: stmatrix.trans
//     turns them so that rows are stored 16 bytes per lane.  Gradient tiles
//     leave by TMA, which stops at the edges of dW;
//   * the gradient's contraction ends inside a box of 64 rows.  What lies
//     behind an expert's last row may be anything (another expert's, NaN), so
//     a warp of the leading CTA has up to 15 rows of both operands filled with
//     zeros in both CTAs' shared memory before the MMAs of a last box run; MMAs
//     that would see no row at all are left out.
// Rows of a product's B that are not the expert's give columns that are not
// stored, so they need no zeroing.
// Every mbarrier wait is bounded; see mxfp4_gemm.cu.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"

namespace chord {
namespace {

enum Mode { kProduct, kTransposed, kGradient, kGradient32 };   // the last: dW in FP32
constexpr bool is_gradient(Mode m) { return m >= kGradient; }

constexpr int kMaxTok = 256;           // largest row tile (columns of the accumulator)
constexpr int kTileM = 256;            // of the pair
constexpr int kStageK = 64;
constexpr int kABytes = 128 * kStageK * 2;
template <Mode kMode>
constexpr int kSubs = is_gradient(kMode) ? 1 : 2;  // steps of 64 of the contraction in a stage
constexpr int kSplitTok = 64;          // largest row tile of items that are cut
constexpr int kSlotFloats = kSplitTok * 128;       // one CTA's part of an item that is cut
constexpr int kMaxCtas = 160;
static_assert(kMaxCtas * sizeof(int) <= CHORD_EXPERT_GEMM_COUNTER_BYTES, "a counter for each CTA");
// Stages of 128 that cutting has to save to pay for adding the parts up, and
// that a part has at least.
constexpr int kSplitSaves = 6, kSplitLeast = 4;
constexpr int kBlockBytes = 64 * kStageK * 2;      // 64 contiguous M or N values x 64 of the contraction
constexpr int kMaxStages = 10, kMaxAcc = 8;
__host__ __device__ constexpr int stage_bytes(int tok) { return kABytes + tok / 2 * kStageK * 2; }
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kItemWarp = 2;
// Two zeroing warps of the leading CTA take items in turn.  Both CTAs' last box
// completes on a barrier of theirs.  Then they start copies from behind the
// tensor's end, which fill with zeros, to the same rows of both CTAs; these
// complete on the stage's barrier, for which the MMAs wait anyway, so that nothing
// but completed copies has to be seen from the other CTA.  (Zeros stored by threads
// of the CTA that holds them need a release at cluster scope, 0.8 us, zeros stored
// into the other CTA a fence: 170 rows an expert 571 and 541 us, 341 rows 836 and
// 835; here 533 and 757.)
constexpr int kZeroWarp0 = 3, kZeroWarp1 = kEpiWarp0 + kEpiWarps;
constexpr int kThreads = 32 * (kZeroWarp1 + 1);
// Where a dW passes through DRAM and its tiles have one box, what the clusters
// store sets the pace, and they drift apart: dW's lines then reach DRAM in a worse
// order.  A fence at cluster scope for each such box (two in FP32: twice the bytes)
// slows the zeroing warps to about that pace and keeps the clusters in step: 48
// experts of 4096 x 7168 with 43 rows each 494 us without, 431 with it, FP32 960
// and 916; 48 of 2048 x 2048 75.5 / 72.0.  Where dW nearly fits in L2 (129 MB) it
// only takes time: 128 MB 25.9 without, 26.4 with it, 192 MB 35.7 / 35.4, 256 MB
// 46.4 / 45.9, FP32 of 256 MB 49.6 / 49.6.
constexpr size_t kPacedBytes = size_t{256} << 20;
constexpr int kItemSlots = 8;
// Barriers in one array, so that each is initialised by a thread of its own (one
// thread for all took 0.15 us of every launch).
constexpr int kEmptyBar = kMaxStages, kTfullBar = kEmptyBar + kMaxStages, kTemptyBar = kTfullBar + kMaxAcc,
              kItemFullBar = kTemptyBar + kMaxAcc, kItemEmptyBar = kItemFullBar + kItemSlots,
              kDoneBar = kItemEmptyBar + kItemSlots, kTailBar = kDoneBar + 1, kBars = kTailBar + 2 * kMaxStages;
constexpr int kMaxExperts = 1024;
constexpr int kTmemCols = 512;
constexpr int kGroupTiles = 8;         // row tiles that are taken together
// Up to this many experts are taken in descending order of their rows, and
// dealt forth and back, so that experts of uneven popularity leave the clusters
// about evenly busy.
constexpr int kMaxSorted = 256;
// An epilogue warp's staging: product 32 tokens x 32 weights (rows of 80
// bytes spread over the banks); gradient 32 rows of 128 bytes (twice that, at
// the cost of a stage of the ring, gained 1.5 % where an expert's rows are few
// and lost 4 % where they are many).
constexpr int kOutPitch = 80;
template <Mode kMode>
constexpr int kOutBytes = is_gradient(kMode) ? 32 * 128 : 32 * kOutPitch;
constexpr int kStageBudget = 6 * stage_bytes(kMaxTok);
// The tensor cores cut products off toward zero where they enter a sum, about two
// bits below FP32's last place: n products of one sign come out up to n 2^-26 too
// small (FP16 6.4e-9 n, at worst 9.3e-9 n; BF16, whose products have fewer bits,
// 1e-9 n at 16384 and 6e-9 n at 2^20), products of both signs far less.  An FP32
// gradient is therefore added up, rounding to nearest, from parts of at most this
// many boxes (768 rows: 4.2e-6 in FP16 and 3.5e-7 in BF16 for one sign, where one
// sum of 16384 rows is 1e-4 and 1.9e-5 off).  In 16 bits the result's own rounding is
// larger up to n = 2^15 (FP16, 2^-11) and 2^18 (BF16, 2^-8) at the least.
constexpr int kExactBoxes = 12;
template <Mode kMode>
constexpr int kSmemBytes = kStageBudget + kEpiWarps * kOutBytes<kMode> + 1024;
static_assert(kMaxStages * stage_bytes(32) <= kStageBudget, "stage budget");
static_assert(kSmemBytes<kProduct> + (kMaxExperts + 1) * 4 + 2048 <= 232448, "shared memory budget");
static_assert(kSmemBytes<kGradient> + 1536 <= 232448, "shared memory budget");
static_assert(kBars <= kThreads, "a thread for each barrier");
static_assert(3 * kThreads >= kMaxExperts, "three experts per thread at most");

struct Args {
  const int32_t* counts;
  const int32_t* offsets;
  uint16_t* out;         // product
  long long ldo;
  int* status;
  int* split_cnt;        // [CTAs] parts arrived, zero between launches
  float* partial;        // [CTAs][rows / 4][128 weights][4]
  int E, capacity;
  int m, k;              // product: weights' side of the output, contraction; gradient: N, K
  int m_tiles, n_tiles;  // tiles of 256
  int paced;             // (gradient)
  int test_timeout;      // test of the timeout path: no item is handed out, waits for one are short
};
// The product's B boxes (rows of x) have the height of half a row tile: one
// map for each multiple of 16.  A gradient's b[0] has 64 rows, its b[3] to b[7]
// have 1, 2, 4, 8 and 16, for zeros.
struct Maps {
  CUtensorMap a, b[8], out;
};

struct alignas(16) Seg {
  int e, row0, rows, m0;   // expert; its rows of this item (gradient: all of them); first weight row
  int n0, cols;            // gradient: first column of dW; product: the part's item.  Columns of the accumulator
  int u0, u1;              // of the contraction, in steps of 64; u1 < 0: the end of the work
};

// a / b for a >= 0, b > 0.  A launch's first instructions are fetched as they
// run, and an integer division is three times as many as this one of small
// numbers (the correction makes up for a quotient that is one off).
__device__ __forceinline__ int quick_div(int a, int b) {
  if (a >= 1 << 22) return a / b;
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  q -= q * b > a;
  q += (q + 1) * b <= a;
  return q;
}
// Whether a gradient's last box of an expert passes through a zeroing warp.
__device__ __forceinline__ bool zeroed(const Args& a, int rows) {
  return (rows & 15) || (a.paced && rows > 0 && rows <= kStageK);
}
__device__ __forceinline__ int up32(int v) { return (v + 31) & ~31; }
__device__ __forceinline__ int row_tiles(int cnt) { return (cnt + kMaxTok - 1) / kMaxTok; }
// Rows of an expert's row tiles: equal to within the rounding to 32.
__device__ __forceinline__ int tile_rows(int cnt, int n) { return up32(n > 1 ? (cnt + n - 1) / n : cnt); }

// The items in the order in which they are dealt, `e` the expert's place.
//   product: experts in order; per expert groups of kGroupTiles row tiles; per
//   group the weight tiles; per weight tile the group's row tiles
//   gradient: experts in order; per expert tiles of N, per tile tiles of K
template <Mode kMode>
__device__ __forceinline__ Seg decode(const Args& a, const int* prefix, const uint8_t* order, int item, int& e) {
  const int lane = threadIdx.x & 31;
  Seg s{};
  if constexpr (is_gradient(kMode)) {
    const int per = a.m_tiles * a.n_tiles;
    e = quick_div(item, per);
    const int local = item - e * per, mt = quick_div(local, a.n_tiles);
    s.m0 = mt * kTileM;
    s.n0 = (local - mt * a.n_tiles) * kMaxTok;
    s.cols = min(kMaxTok, up32(a.k - s.n0));
    s.e = order ? order[e] : e;
    s.row0 = ld_ca(a.offsets + s.e);
    s.rows = ld_ca(a.counts + s.e);
    s.u1 = (s.rows + kStageK - 1) / kStageK;
  } else {
    // the largest e with prefix[e] <= item (items only grow)
    auto past = [&](int at) { return __ballot_sync(0xffffffffu, at > a.E || prefix[at] > item); };
    uint32_t found = past(e + 1 + lane);
    if (!found) {                      // further on: the 32nd of the experts, then the expert
      const int block = (a.E + 31) / 32;
      static_assert(kMaxExperts <= 32 * 32, "two steps of 32");
      e = block * (__ffs(past(min(block * (lane + 1), a.E))) - 1);
      found = past(e + 1 + lane);
    }
    e += __ffs(found) - 1;
    s.e = order ? order[e] : e;
    const int cnt = ld_ca(a.counts + s.e);
    int local = item - prefix[e], rt = 0;
    s.row0 = ld_ca(a.offsets + s.e);
    s.rows = cnt;
    if (cnt > kMaxTok) {
      const int n = row_tiles(cnt), per = tile_rows(cnt, n);
      const int group = local / (kGroupTiles * a.m_tiles);
      local -= group * kGroupTiles * a.m_tiles;
      const int width = min(kGroupTiles, n - group * kGroupTiles);
      const int mt = local / width;
      rt = group * kGroupTiles + local - mt * width;
      local = mt;
      s.row0 += rt * per;
      s.rows = min(per, cnt - rt * per);
    }
    s.m0 = local * kTileM;
    s.cols = up32(s.rows);
    s.u1 = (a.k + kStageK - 1) / kStageK;
  }
  return s;
}

struct ItemRing {
  uint64_t *full, *empty;
  const Seg* slots;
  uint32_t polls;
  int slot, ph;
  // The next item: false at the end of the work or on a timeout.  All lanes
  // of the calling warp take it; lane 0 releases the slot.
  __device__ __forceinline__ bool next(Seg& s, bool& ok, int* status) {
    ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], ph, status, polls));
    if (!ok) return false;
    const int4* src = reinterpret_cast<const int4*>(&slots[slot]);
    const int4 lo = src[0], hi = src[1];
    s.e = lo.x, s.row0 = lo.y, s.rows = lo.z, s.m0 = lo.w;
    s.n0 = hi.x, s.cols = hi.y, s.u0 = hi.z, s.u1 = hi.w;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[slot]);
    if (++slot == kItemSlots) slot = 0, ph ^= 1;
    return s.u1 >= 0;
  }
};

// The sum over the lanes up to this one.
__device__ __forceinline__ int scan_warp(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four 8 x 8 matrices of 16-bit values, transposed (as in mxfp4_gemm.cu).
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Up to 32 rows of a finished product tile: this warp's accumulators of its 32
// weights (lo: 0-15 of the lane quarter, hi: 16-31), `n` rows at `out`, from
// column `col0` on.
template <bool kF16>
__device__ __forceinline__ void store_rows(const Args& a, const uint32_t (&lo)[16], const uint32_t (&hi)[16],
                                           uint16_t* out, uint32_t stage_s, int col0, int lane, int n) {
  // lane 8 i + c: row c of its group of 8, weights 8 (i & 1) on
  const uint32_t dst = stage_s + ((lane & 7) + 8 * (lane >> 4)) * kOutPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
  for (int p = 0; p < 2; ++p) {   // rows 16 p .. 16 p + 15
    uint32_t l[4], h[4];          // [group of 8 rows][weights 0-7, 8-15]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * p + 2 * i;
      l[i] = pack2<kF16>(__uint_as_float(lo[r]), __uint_as_float(lo[r + 1]));
      h[i] = pack2<kF16>(__uint_as_float(hi[r]), __uint_as_float(hi[r + 1]));
    }
    stmatrix_x4_trans(dst + 16 * p * kOutPitch, l[0], l[1], l[2], l[3]);
    stmatrix_x4_trans(dst + 16 * p * kOutPitch + 32, h[0], h[1], h[2], h[3]);
  }
  __syncwarp();
  const int part = lane & 3, col = col0 + 8 * part;   // four lanes per row
  uint4 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w)
                 : "r"(stage_s + ((lane >> 2) + 8 * j) * kOutPitch + 16 * part)
                 : "memory");
  if (col < a.m) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = (lane >> 2) + 8 * j;
      if (row < n) *reinterpret_cast<uint4*>(out + row * a.ldo + col) = v[j];
    }
  }
  __syncwarp();
}

// Whether `ok` holds in all threads of the epilogue warps.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "n"(32 * kEpiWarps)
      : "memory");
  return r != 0;
}

// The sum of an item's parts (of CTAs first, first + 2, ...) in order, for this
// lane's weight and the rows c0 .. c0 + 3 and, where `both`, the four after
// them, to `out` (the item's first row and this lane's column).  Six parts' loads
// are in flight; parts past the last are loaded again, not added.
template <bool kF16>
__device__ __forceinline__ void add_parts(const float* partial, int first, int parts, int c0, int rows, uint16_t* out,
                                          long long ldo, bool in) {
  float f[8] = {};
  for (int p0 = 0; p0 < parts; p0 += 6) {
    float4 x[6][2];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const float* src = partial + static_cast<size_t>(first + 2 * min(p0 + i, parts - 1)) * kSlotFloats + c0 * 128;
      x[i][0] = ld_cg_f4(src);
      x[i][1] = ld_cg_f4(src + (c0 + 4 < rows ? 512 : 0));
    }
#pragma unroll
    for (int i = 0; i < 6; ++i)
      if (p0 + i < parts)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          f[4 * c] += x[i][c].x, f[4 * c + 1] += x[i][c].y;
          f[4 * c + 2] += x[i][c].z, f[4 * c + 3] += x[i][c].w;
        }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (in && c0 + i < rows) out[(c0 + i) * ldo] = static_cast<uint16_t>(pack2<kF16>(f[i], 0.f));
}

template <Mode kMode, bool kF16>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    expert_gemm_kernel(const __grid_constant__ Maps maps, const Args a) {
  constexpr bool kGrad = is_gradient(kMode), kF32 = kMode == kGradient32;
  constexpr bool kMnA = kMode != kProduct, kMnB = kGrad;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kBars];
  uint64_t *full = bars, *empty = bars + kEmptyBar, *tfull = bars + kTfullBar, *tempty = bars + kTemptyBar;
  uint64_t *item_full = bars + kItemFullBar, *item_empty = bars + kItemEmptyBar, *done_bar = bars + kDoneBar;
  uint64_t* tail = bars + kTailBar;      // [zeroing warp][stage], of the leading CTA
  __shared__ Seg item_slots[kItemSlots];
  __shared__ uint32_t tmem_base_s;
  __shared__ int prefix[kGrad ? 1 : kMaxExperts + 1];
  __shared__ uint8_t order_s[kMaxSorted];
  __shared__ int warp_sum[kThreads / 32], warp_max[kThreads / 32];
  __shared__ int last_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;

  if (tid < kBars) {
    int count = 1;
    if (tid < kEmptyBar || tid >= kTailBar) count = 2;               // of the leading CTA: each CTA's bytes, or zeros
    if (tid >= kTemptyBar && tid < kItemFullBar) count = 2 * kEpiWarps;   // of the leading CTA
    if (tid >= kItemEmptyBar && tid < kDoneBar) count = 1 + (rank == 0 ? (kGrad ? 3 : 1) : 0) + kEpiWarps;
    mbar_init(&bars[tid], count);
    fence_mbar_init();
  }
  __syncwarp();
  cluster_arrive();   // the barriers are there
  if (warp == 1) tmem_alloc_pair(&tmem_base_s, kTmemCols);
  // programmatic launch: nothing above touches global memory
  grid_dep_wait();
  grid_dep_launch();

  // The order is checked, and for a product the first item of each expert and
  // the largest row tile are found: thread i covers experts [i * per, (i + 1) * per).
  const int per = 1 + (a.E > kThreads) + (a.E > 2 * kThreads);
  int mine = 0, most = 32, bad = 0, cnt = 0;
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e >= a.E) break;
    cnt = ld_ca(a.counts + e);
    const int off = ld_ca(a.offsets + e), next = ld_ca(a.offsets + e + 1);
    // Experts that end before the next one begins have disjoint rows.
    if (cnt < 0 || off < 0 || cnt > a.capacity || off > a.capacity - cnt || off + cnt > next) bad = 1, cnt = 0;
    if constexpr (!kGrad) {
      prefix[e] = mine;
      if (cnt > 0) {
        const int n = row_tiles(cnt);
        mine += a.m_tiles * n;
        most = max(most, tile_rows(cnt, n));
      }
    }
  }
  // (scratch: the staging that the epilogue will use)
  int* cnt_s = reinterpret_cast<int*>(smem_raw + (smem0 - smem_u32(smem_raw)) + kStageBudget);
  if (a.E <= kMaxSorted && tid < kMaxSorted) cnt_s[tid] = tid < a.E ? cnt : -1;
  int inc = kGrad ? 0 : scan_warp(mine);
  most = __reduce_max_sync(0xffffffffu, bad ? 1 << 16 : most);
  if (lane == 31) {
    warp_sum[warp] = inc;
    warp_max[warp] = most;
  }
  __syncthreads();
  int tok = __reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? warp_max[lane] : 0);
  const bool order_ok = tok < 1 << 16;   // else nothing is computed
  if (!order_ok && tid == 0) set_status(a.status, CHORD_ERR_INVALID_ARG);
  // With few rows in every tile a product's items take the same time, and
  // a gradient of one round has no order (6.33 -> 6.01 us at 8 experts of
  // 72 x 1192).
  const bool sorted = a.E > 1 && a.E <= kMaxSorted &&
                      (kGrad ? a.E * a.m_tiles * a.n_tiles > clusters : tok > kSplitTok);
  if (sorted) {
    if (tid < a.E) {
      int place = 0;
      for (int i = 0; i < a.E; i += 4) {
        const int4 c = *reinterpret_cast<const int4*>(cnt_s + i);
        place += (c.x > cnt || (c.x == cnt && i < tid)) + (c.y > cnt || (c.y == cnt && i + 1 < tid)) +
                 (c.z > cnt || (c.z == cnt && i + 2 < tid)) + (c.w > cnt || (c.w == cnt && i + 3 < tid));
      }
      order_s[place] = static_cast<uint8_t>(tid);
      cnt_s[kMaxSorted + place] = mine;
    }
    __syncthreads();
    if constexpr (!kGrad) {
      mine = tid < a.E ? cnt_s[kMaxSorted + tid] : 0;
      if (tid < a.E) prefix[tid] = 0;
      inc = scan_warp(mine);
      if (lane == 31) warp_sum[warp] = inc;
      __syncthreads();
    }
  }
  if constexpr (!kGrad) {
    const int sum = scan_warp(lane < kThreads / 32 ? warp_sum[lane] : 0);
    const int run = inc - mine + (warp ? __shfl_sync(0xffffffffu, sum, warp - 1) : 0);
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int e = tid * per + i;
      if (e >= a.E) break;
      prefix[e] += run;
    }
    if (tid == kThreads - 1) prefix[a.E] = run + mine;   // the last thread ends at the total
  }
  const uint8_t* order = sorted ? order_s : nullptr;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_wait();                        // the peer's barriers are there
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, tmem_base_s, 0);
  if (kGrad) tok = kMaxTok;
  tok = order_ok ? tok : 32;
  const int items = !order_ok ? 0 : kGrad ? a.E * a.m_tiles * a.n_tiles : prefix[a.E];
  constexpr int subs = kSubs<kMode>;
  const int sub_bytes = stage_bytes(tok), stage = subs * sub_bytes;
  const int n_stages = min(kMaxStages, kStageBudget / stage);
  // The items that are cut, and their parts: cluster i has part i % parts of
  // item i / parts, then whole items like all others.
  int cut = 0, parts = 0;
  if constexpr (!kGrad) {
    const int units = (a.k + 2 * kStageK - 1) / (2 * kStageK);   // stages
    if (tok <= kSplitTok) {
      cut = items - quick_div(items, clusters) * clusters;
      if (cut > 0) parts = min(quick_div(clusters, cut), units / kSplitLeast);
      if (parts < 2 || units - quick_div(units + parts - 1, parts) < kSplitSaves) cut = parts = 0;
    }
  }
  const int n_acc = min(kMaxAcc, kTmemCols / tok);
  ItemRing ring{item_full, item_empty, item_slots, a.test_timeout ? kTestWaitPolls : kWaitPolls, 0, 0};
  Seg w;
  bool ok = true;

  if (warp == 0) {
    // ----------------------------------------------------------------- loads
    // The whole warp runs the loop, one elected lane issues.  Both CTAs' bytes
    // count on barriers of the leading CTA: the stage's, or for a gradient's last
    // box the zeroing warp's.
    const uint32_t full0 = cluster_addr(&full[0], 0), tail0 = cluster_addr(&tail[0], 0);
    int it = 0, st = 0, ph = 0, turn = 0;
    while (ring.next(w, ok, a.status)) {
      const int half = w.cols >> 1;
      const CUtensorMap* mb = &maps.b[kGrad ? 0 : (half >> 4) - 1];
      const uint32_t bytes = kABytes + (kGrad ? 2 * kBlockBytes : half * kStageK * 2);
      const int m = w.m0 + 128 * static_cast<int>(rank);
      const int n = kGrad ? w.n0 + half * static_cast<int>(rank) : w.row0 + half * static_cast<int>(rank);
      for (int u0 = w.u0; u0 < w.u1; u0 += subs, ++it) {
        if (it >= n_stages && !(ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1, a.status)))) break;
        uint32_t dst = smem0 + st * stage, bar = full0 + 8 * st;
        const int here = min(subs, w.u1 - u0);
        const int left = w.rows - u0 * kStageK;            // (gradient)
        if (kGrad && left <= kStageK && zeroed(a, w.rows)) {
          bar = tail0 + 8 * (turn * kMaxStages + st);
          turn ^= 1;
        }
        mbar_arrive_expect_tx_cluster_elect(bar, here * bytes);
        for (int u = u0; u < u0 + here; ++u, dst += sub_bytes) {
          const int k0 = u * kStageK;
          if constexpr (kMode == kProduct) {
            tma_pair_3d_elect(dst, &maps.a, k0, m, w.e, bar);
            tma_pair_2d_elect(dst + kABytes, mb, k0, n, bar);
          } else if constexpr (kMode == kTransposed) {
            tma_pair_3d_elect(dst, &maps.a, m, k0, w.e, bar);
            tma_pair_3d_elect(dst + kBlockBytes, &maps.a, m + 64, k0, w.e, bar);
            tma_pair_2d_elect(dst + kABytes, mb, k0, n, bar);
          } else {
            const int row = w.row0 + k0;
            tma_pair_2d_elect(dst, &maps.a, m, row, bar);
            tma_pair_2d_elect(dst + kBlockBytes, &maps.a, m + 64, row, bar);
            tma_pair_2d_elect(dst + kABytes, mb, n, row, bar);
            tma_pair_2d_elect(dst + kABytes + kBlockBytes, mb, n + 64, row, bar);
          }
        }
        if (++st == n_stages) st = 0, ph ^= 1;
      }
      if (!ok) break;
    }
    // Every copy lands before a CTA can exit: the leading CTA waits for both
    // CTAs' bytes (the cluster barrier below holds the other).
    if (rank == 0)
      for (int j = max(0, it - n_stages); j < it; ++j)
        ok = mbar_wait(&full[j % n_stages], (j / n_stages) & 1, a.status) && ok;
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------------ MMAs
    int st = 0, ph = 0, acc = 0, use = 0;
    bool issued = false;
    while (ring.next(w, ok, a.status)) {
      const uint32_t d = tmem_base + acc * tok;
      const uint32_t idesc = idesc_pair(!kF16, kMnA, kMnB, w.cols);
      uint32_t accumulate = 0;
      if (use >= 1) ok = __all_sync(0xffffffffu, mbar_wait(&tempty[acc], (use - 1) & 1, a.status));
      tc_fence_after();
      for (int u0 = w.u0; ok && u0 < w.u1; u0 += subs) {
        const int left = w.rows - u0 * kStageK;            // (gradient)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&full[st], ph, a.status)))) break;
        tc_fence_after();
        // 16 of the contraction: 32 bytes on in a row, or 16 rows of 128 bytes
        constexpr int kStepA = kMnA ? 128 : 2, kStepB = kMnB ? 128 : 2;
        uint32_t sa = smem0 + st * stage;
        for (int u = u0; u < min(u0 + subs, w.u1); ++u, sa += sub_bytes) {
          const uint32_t sb = sa + kABytes;
          const uint64_t da = kMnA ? sw128_mnmajor_desc(sa, kBlockBytes) : sw128_kmajor_desc(sa);
          const uint64_t db = kMnB ? sw128_mnmajor_desc(sb, kBlockBytes) : sw128_kmajor_desc(sb);
          const int steps = kGrad ? (min(left, kStageK) + 15) / 16 : 4;
          if (!kGrad || steps == 4) {
            tc_pair_mma4_elect<kStepA, kStepB>(d, da, db, idesc, accumulate);
          } else {
            for (int i = 0; i < steps; ++i)
              tc_pair_mma_elect(d, da + i * kStepA, db + i * kStepB, idesc, accumulate | (i > 0));
          }
          accumulate = 1;
        }
        tc_pair_commit_elect(&empty[st]);
        issued = true;
        if (++st == n_stages) st = 0, ph ^= 1;
      }
      if (!ok) break;
      tc_pair_commit_elect(&tfull[acc]);
      if (++acc == n_acc) acc = 0, ++use;
    }
    // all issued MMAs complete before TMEM can be freed
    if (issued) {
      tc_commit_pair_local_elect(done_bar);
      ok = mbar_wait(done_bar, 0, a.status) && ok;
    }
  } else if (warp == kItemWarp) {
    // ----------------------------------------------------------------- items
    int slot = 0, ph = 0, e = 0;
    bool part = cluster < cut * parts;
    int item = part ? quick_div(cluster, parts) : cut + cluster, round = cut;
    int boxes = 0, piece = 0;            // of an FP32 gradient's item, and of each of its parts
    Seg s{};
    for (bool first = true, more = !a.test_timeout; more;) {
      if (kF32 && s.u1 < boxes) {        // the item's next part
        s.u0 = s.u1;
        s.u1 = min(boxes, s.u0 + piece);
      } else if ((more = item < items)) {
        s = decode<kMode>(a, prefix, order, item, e);
        if (part) {
          // whole stages of two steps, the last one short where their number is odd
          const int units = (s.u1 + 1) / 2, p = cluster - item * parts;
          s.u0 = 2 * quick_div(p * units, parts);
          s.u1 = min(s.u1, 2 * quick_div((p + 1) * units, parts));
          s.n0 = item;
        }
        boxes = s.u1;
        if (kF32 && boxes > kExactBoxes) {
          const int n = (boxes + kExactBoxes - 1) / kExactBoxes;
          s.u1 = piece = (boxes + n - 1) / n;
        }
        if (!part) round += clusters;
        item = round + cluster;
        // forth and back over items of falling size
        if (sorted && quick_div(round, clusters) & 1) item = round + clusters - 1 - cluster;
        part = false;
      } else {
        s.u1 = -1;
      }
      if (!first && !(ok = __all_sync(0xffffffffu, mbar_wait_backoff(&item_empty[slot], ph ^ 1, a.status)))) break;
      if (lane == 0) {
        item_slots[slot] = s;
        mbar_arrive(&item_full[slot]);   // release: the item is visible to the waiters
      }
      if (++slot == kItemSlots) slot = 0, ph ^= 1, first = false;
    }
  } else if (kGrad && rank == 0 && (warp == kZeroWarp0 || warp == kZeroWarp1)) {
    // ------------------------------------------- rows behind an expert's last
    const uint32_t full0 = cluster_addr(&full[0], 0);
    const int mine = warp == kZeroWarp1;   // boxes are handed to the two warps in turn
    int st = 0, turn = 0;
    uint32_t tail_ph = 0;                // of this warp's barriers: one turns when its stage holds a box for it
    while (ring.next(w, ok, a.status)) {
      st = (st + w.u1 - w.u0) % n_stages;
      if (!zeroed(a, w.rows) || (kF32 && w.u1 * kStageK < w.rows)) continue;
      turn ^= 1;
      if (turn == mine) continue;        // the other warp's: turn was its number
      // Every phase of a warp's barriers is waited for, in order.
      const int at = (st ? st : n_stages) - 1;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&tail[mine * kMaxStages + at], (tail_ph >> at) & 1, a.status)))) break;
      tail_ph ^= 1u << at;
      if (a.paced && w.rows <= kStageK)
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) fence_cluster();
      // n rows from `last` on of the four blocks of 64 values: 16 rows where the box
      // has them (no MMA reads the ones past n; 170 rows an expert 544 us without, 533
      // with it), else once or twice the largest power of two, from both ends
      const int last = w.rows % kStageK, n = -last & 15;
      const int log = last <= kStageK - 16 ? 4 : 31 - __clz(n), h = n ? 1 << log : 0;
      const int copies = n ? n > h ? 8 : 4 : 0;
      const uint32_t base = smem0 + at * stage + last * 128;
      // both CTAs' arrivals and bytes; a release, for the boxes that were waited for
      mbar_arrive_expect_tx_elect(&full[at], copies * h * 128);
      mbar_arrive_expect_tx_elect(&full[at], copies * h * 128);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < copies)
          tma_pair_2d_both_elect(base + (i & 3) * kBlockBytes + (i >> 2) * (n - h) * 128, &maps.b[3 + log], 0, a.capacity,
                                 full0 + 8 * at);
    }
  } else if (warp >= kEpiWarp0 && warp < kEpiWarp0 + kEpiWarps) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3, t = (warp - kEpiWarp0) / 4;   // TMEM lane quarter; which of the column chunks
    const uint32_t out_stage = smem0 + kStageBudget + (warp - kEpiWarp0) * kOutBytes<kMode>;
    const uint32_t tempty0 = cluster_addr(&tempty[0], 0);
    const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
    int acc = 0, use = 0;
    // A wait that ran out ends a warp; at an item that is cut, whose handling
    // has barriers, the epilogue warps end together.
    bool part = !kGrad && cluster < cut * parts;
    while (true) {
      const bool on = ring.next(w, ok, a.status);
      bool go = on && (ok = __all_sync(0xffffffffu, mbar_wait(&tfull[acc], use & 1, a.status)));
      if (part && !a.test_timeout) go = epilogue_all(go);
      if (!go) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + acc * tok + lanes;
      const int m = w.m0 + 128 * static_cast<int>(rank) + 32 * q;
      if (!kGrad && part) {
        // this CTA's part, four rows of a weight together
        float* mine_p = a.partial + static_cast<size_t>(blockIdx.x) * kSlotFloats + (32 * q + lane) * 4;
        for (int c0 = 32 * t; c0 < w.rows; c0 += 64) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c0, v);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            if (c0 + c < w.rows)
              *reinterpret_cast<uint4*>(mine_p + (c0 + c) * 128) = make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        }
      } else if constexpr (!kGrad) {
        // the next 32 rows' accumulators are on their way while these go out
        uint32_t next[2][16];
        auto load = [&](int c0) {
          tmem_ld_16x256b_x4(taddr + c0, next[0]);
          tmem_ld_16x256b_x4(taddr + c0 + (16u << 16), next[1]);
        };
        uint16_t* out = a.out + w.row0 * a.ldo;
        if (32 * t < w.rows) load(32 * t);
#pragma unroll 1
        for (int c0 = 32 * t; c0 < w.rows; c0 += 64) {
          tmem_ld_wait();
          uint32_t v[2][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[0][i] = next[0][i], v[1][i] = next[1][i];
          if (c0 + 64 < w.rows) load(c0 + 64);
          store_rows<kF16>(a, v[0], v[1], out + c0 * a.ldo, out_stage, m, lane, w.rows - c0);
        }
      } else {
        // chunks of 128 bytes of dW's rows leave by TMA, 16-byte parts swizzled
        // with the row; 32 columns at a time, the next ones on their way
        constexpr int width = kF32 ? 32 : 64;
        const uint32_t dst = out_stage + lane * 128;
        uint32_t next[32];
        auto load = [&](int c) {
          if (w.rows > 0 && c < w.cols) {
            tmem_ld_32x32b_x32(taddr + c, next);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) next[i] = 0;
          }
        };
        load(width * t);
        if (kF32 && w.u0 > 0 && lane == 0) bulk_wait_all();   // the item's parts before are there to be added to
        // dW passes through L2 once (left to it, the lines went to DRAM in an
        // order that took 452 us where this takes 431: 48 experts of 4096 x 7168,
        // 43 rows each; 128 MB 28.8 / 25.0, 64 MB 15.7 / 14.8).  A dW that fits in
        // L2 and is read at once comes back more slowly: the call and a sum over
        // 64 MB 28.7 us left to L2, 30.8 here; 256 MB 126.5 / 123.9.  Parts are
        // added to where they lie
        const uint64_t policy = kF32 && w.u1 * kStageK < w.rows ? policy_evict_normal() : policy_evict_first();
#pragma unroll 1
        for (int c0 = width * t; c0 < w.cols; c0 += 2 * width) {
#pragma unroll
          for (int half = 0; half < width / 32; ++half) {
            uint32_t v[32];
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = next[i];
            load(half + 1 < width / 32 ? c0 + 32 : c0 + 2 * width);
            if (half == 0) {
              if (lane == 0) bulk_wait_read();                // the last store has read its staging
              __syncwarp();
            }
            if constexpr (kF32) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                st_shared_v4(dst + ((j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  p[i] = pack2<kF16>(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
                st_shared_v4(dst + (((j + 4 * half) ^ (lane & 7)) << 4), p[0], p[1], p[2], p[3]);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && m < a.m && w.n0 + c0 < a.k) {
            if (kF32 && w.u0 > 0) tma_add_3d(&maps.out, out_stage, w.n0 + c0, m, w.e);
            else tma_store_3d(&maps.out, out_stage, w.n0 + c0, m, w.e, policy);
            bulk_commit_group();
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
      if (++acc == n_acc) acc = 0, ++use;
      if (kGrad || !part) continue;
      part = false;
      const int first = 2 * w.n0 * parts + static_cast<int>(rank);   // the CTA with the item's first part
      epilogue_all(true);
      if (tid == 32 * kEpiWarp0) {
        // releases the parts stored by all threads before the barrier, and
        // acquires the others'
        int arrived;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                     : "=r"(arrived)
                     : "l"(a.split_cnt + first)
                     : "memory");
        last_flag = arrived == parts - 1;
      }
      epilogue_all(true);
      if (!last_flag) continue;
      if (tid == 32 * kEpiWarp0) a.split_cnt[first] = 0;   // for the next launch
      for (int c0 = 8 * t; c0 < w.rows; c0 += 16)
        add_parts<kF16>(a.partial + (32 * q + lane) * 4, first, parts, c0, w.rows, a.out + w.row0 * a.ldo + m + lane,
                        a.ldo, m + lane < a.m);
    }
    if (kGrad && lane == 0) bulk_wait_all();
  }
  // A wait that ran out: copies that the other CTA, which may have stopped
  // elsewhere, does not account for have landed by then.
  if (!ok)
    for (int i = 0; i < 1 << 14; ++i) __nanosleep(64);

  tc_fence_before();
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  return fn;
}

// A map of [experts][rows][cols] (rows and experts at the given strides, in
// elements; experts 0: two dimensions) in boxes of 128 bytes by `height` rows,
// 128-byte swizzle.
bool encode(CUtensorMap* map, const void* p, bool f16, bool f32, long long cols, long long rows, long long ld,
            int experts, long long expert_stride, int height) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int size = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(experts)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * size, static_cast<cuuint64_t>(expert_stride) * size};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(height), 1};
  const cuuint32_t one[3] = {1, 1, 1};
  const CUtensorMapDataType type = f32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(map, type, experts ? 3 : 2, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Mode kMode, bool kF16>
cudaError_t launch(const Maps& maps, const Args& a, cudaStream_t st) {
  cudaError_t err = ensure_smem_limit<expert_gemm_kernel<kMode, kF16>>(kSmemBytes<kMode>);
  if (err != cudaSuccess) return err;
  return launch_kernel(expert_gemm_kernel<kMode, kF16>, dim3(std::max(2, std::min(kMaxCtas, sm_count() & ~1))),
                       dim3(kThreads), kSmemBytes<kMode>, st, true, maps, a);
}

}  // namespace

size_t expert_gemm_workspace_bytes() {
  return CHORD_EXPERT_GEMM_COUNTER_BYTES + sizeof(float) * kMaxCtas * kSlotFloats;
}

cudaError_t expert_gemm_launch(const ExpertGemm& g, cudaStream_t st) {
  if (!g.transposed && !g.test_timeout && expert_gemv_serves(g)) return expert_gemv_launch(g, st);
  Args a{};
  a.counts = g.counts, a.offsets = g.offsets, a.status = g.status;
  a.E = g.E, a.capacity = g.capacity, a.test_timeout = g.test_timeout ? 1 : 0;
  a.out = static_cast<uint16_t*>(g.out), a.ldo = g.ldo;
  a.split_cnt = static_cast<int*>(g.ws);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(g.ws) + CHORD_EXPERT_GEMM_COUNTER_BYTES);
  a.m = g.transposed ? g.K : g.N, a.k = g.transposed ? g.N : g.K;
  a.m_tiles = (a.m + kTileM - 1) / kTileM;
  Maps maps{};
  if (!encode(&maps.a, g.w, g.f16, false, g.K, g.N, g.ldw, g.E, g.expert_stride, g.transposed ? kStageK : 128))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 8; ++i)
    if (!encode(&maps.b[i], g.x, g.f16, false, a.k, g.capacity, g.ldx, 0, 0, 16 * (i + 1)))
      return cudaErrorInvalidValue;
  if (g.transposed) return g.f16 ? launch<kTransposed, true>(maps, a, st) : launch<kTransposed, false>(maps, a, st);
  return g.f16 ? launch<kProduct, true>(maps, a, st) : launch<kProduct, false>(maps, a, st);
}

cudaError_t expert_wgrad_launch(const ExpertWgrad& g, cudaStream_t st) {
  Args a{};
  a.counts = g.counts, a.offsets = g.offsets, a.status = g.status;
  a.E = g.E, a.capacity = g.capacity, a.test_timeout = g.test_timeout ? 1 : 0;
  a.m = g.N, a.k = g.K;
  a.m_tiles = (g.N + kTileM - 1) / kTileM;
  a.n_tiles = (g.K + kMaxTok - 1) / kMaxTok;
  a.paced = static_cast<size_t>(g.E) * g.N * g.K * (g.f32 ? 4 : 2) >= kPacedBytes;
  Maps maps{};
  if (!encode(&maps.a, g.dout, g.f16, false, g.N, g.capacity, g.ldd, 0, 0, kStageK) ||
      !encode(&maps.b[0], g.x, g.f16, false, g.K, g.capacity, g.ldx, 0, 0, kStageK) ||
      !encode(&maps.out, g.dw, g.f16, g.f32, g.K, g.N, g.K, g.E, static_cast<long long>(g.N) * g.K, 32))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 5; ++i)
    if (!encode(&maps.b[3 + i], g.x, g.f16, false, g.K, g.capacity, g.ldx, 0, 0, 1 << i)) return cudaErrorInvalidValue;
  if (g.f32) return g.f16 ? launch<kGradient32, true>(maps, a, st) : launch<kGradient32, false>(maps, a, st);
  return g.f16 ? launch<kGradient, true>(maps, a, st) : launch<kGradient, false>(maps, a, st);
}

}  // namespace chord
