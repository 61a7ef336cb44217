// The experts' product in MXFP4 on the 5th-generation tensor cores:
//   C[r, n] = sum_k A[r, k] W[e(r), n, k]
// over rows in the aligned expert order, both operands E2M1 with E8M0 scales
// per 32 of K, FP32 accumulation, with an optional SiLU(gate) * up.
//
// Design on sm_103a (one persistent CTA per SM):
//   * an item is two tiles of 128 weight rows (two MMAs of M = 128 on the same
//     rows) times up to kMaxTok of an expert's rows (N, a multiple of 16), so
//     one decoded token costs 16 columns, not 128 rows; one kernel serves
//     decoding and prefill.  The second weight tile halves the traffic of the
//     rows (16384 rows of 8 experts: 199 us against 218 with one tile);
//   * items are dealt whole and in turn, so that CTAs at work at one time
//     share weights and rows in L2 (a contiguous run of items per CTA spread
//     the live weights over more than L2: many rows per expert 346 us).  Where
//     what does not divide evenly among the CTAs leaves half of them idle or
//     more, those items come first and are divided.  With up to kSplitTok rows
//     per tile, along K into equal parts (one token's few items spread over
//     all SMs), which the CTA that finishes last sums from FP32 partials in
//     workspace, in K order, so results do not depend on timing.  With more
//     rows adding partials costs more than the work (8 prefill items in 19
//     parts each: 110 us), and they are divided into single weight tiles and
//     runs of rows instead;
//   * per unit one bulk copy brings the pair's weight rows with their scales
//     (34 KB, contiguous, already swizzled), one or two the rows;
//   * the rows' scales lie in row order in memory, and a row tile may start at
//     any multiple of 8, so warp 3 copies them four bytes at a time into the
//     block layout of a ring of their own, four units ahead (cp.async);
//   * issuing a tcgen05 instruction takes about 45 cycles, and a unit has 14 to
//     18 of them, so each weight tile has a warp of its own that issues its
//     scale copies (tcgen05.cp, to TMEM columns of its own, in order with the
//     MMAs) and MMAs;
//   * the epilogue reads accumulators in the 16-lane layout, where one thread
//     has a weight row's values of two adjacent tokens (and gate and up of
//     the same index), packs them and turns them with stmatrix.trans, so that
//     C is written 16 bytes per lane;
//   * one warp decodes the items and hands them to the others through a ring of
//     eight words each (decoded by every role itself, finding an item took
//     1600 cycles, as long as a short item's work);
//   * stages and accumulators are laid out for the launch's largest row tile,
//     which every CTA finds from the counts: decoding has five stages and four
//     accumulators, a full tile three stages and one accumulator.  One expert
//     with many rows so sets the layout for the small items too, and keeps them
//     from being divided along K.
// Measured (kernel alone): 64 tokens on 48 of 384 experts, N 4096, K 7168: 85
// us, 6.1 TB/s of DRAM, its bound; 8192 tokens: 137 us, DRAM at 5.8 TB/s and
// exposed epilogues; 16384 rows of 8 experts: 177 us, 5.4 PFLOP/s: 54 bytes a
// cycle into each SM, of about 64 that its port takes (tensor pipe 56 %
// busy); one token, N 512: 8.7 us, latency.
// TMEM: accumulators from column 0, scales from column kSfCol.
// Every mbarrier wait is bounded.  A warp whose wait runs out records
// CHORD_ERR_TIMEOUT and stops, so the others' waits run out in turn; the CTA
// drains its own copies and MMAs, frees TMEM and exits.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mxfp4.cuh"
#include "tc5.cuh"

namespace chord {
namespace {

constexpr int kMaxTok = 224;
constexpr int kPair = 2;               // weight tiles per item
constexpr int kMaxStages = 5, kMaxAcc = 4;
constexpr int kEpiWarp0 = 4, kEpiWarps = 4 * kPair, kEpiThreads = 32 * kEpiWarps;
constexpr int kItemWarp = kEpiWarp0 + kEpiWarps;
constexpr int kThreads = 32 * (kItemWarp + 1);
constexpr int kItemSlots = 8;
constexpr int kItemReaders = 1 + kPair + 1 + kEpiWarps;   // copies, MMAs, scales, epilogue
constexpr int kMaxExperts = 1024;
constexpr int kNoOrder = 1 << 16;      // for the largest row tile: the experts' rows overlap
// stage: weight tiles with their scales | rows
constexpr int kBOff = kPair * kMxUnitBytes;
__host__ __device__ constexpr int stage_bytes(int tok) { return kBOff + tok * kMxRowBytes; }
constexpr int kStageBudget = 3 * stage_bytes(kMaxTok);
// ring of the rows' scales in block layout: two K halves of up to 256 rows
constexpr int kSfSlots = 6, kSfAhead = 4;   // slots, and units in flight (fewer)
constexpr int kSfbHalf = 1024, kSfSlotBytes = 2 * kSfbHalf;
// an epilogue warp's 32 tokens x 32 weight rows on their way to C; the pitch
// of 80 bytes spreads stmatrix's and the reads' 16-byte parts over the banks
constexpr int kOutPitch = 80, kOutBytes = 32 * kOutPitch;
constexpr int kSfOff = kStageBudget, kOutOff = kSfOff + kSfSlots * kSfSlotBytes;
constexpr int kSmemBytes = kOutOff + kEpiWarps * kOutBytes + 1024;
constexpr int kMmaWarp0 = 1, kSfWarp = kMmaWarp0 + kPair;
constexpr int kSfCol = kPair * kMaxTok, kSfCols = 32;   // per tile: SFA at +0 and +8 (alternate units), SFB at +16
constexpr int kTmemCols = 512;
constexpr int kSplitUnits = 6, kSplitUnitsHidden = 2;
constexpr int kSplitTok = 48;          // largest row tile whose items are cut along K
constexpr int kSlotFloats = kPair * kSplitTok * 128;   // one CTA's part of a cut item
static_assert(kSplitTok % 16 == 0, "whole runs of rows");
static_assert(kSfCol + kPair * kSfCols <= kTmemCols, "TMEM budget");
static_assert(stage_bytes(16) % 1024 == 0 && kMaxTok % 16 == 0 && kMaxTok <= 256, "stage layout");
static_assert(kMaxStages * stage_bytes(16) <= kStageBudget, "stage budget");
static_assert(kSfAhead < kSfSlots, "a slot is reused after its unit was signalled");
static_assert(kSfWarp + 1 <= kEpiWarp0 && kEpiWarp0 % 4 == 0, "warp roles; warp index selects the TMEM lane quarter");
static_assert(kSmemBytes + (kMaxExperts + 1) * 4 + 1024 <= 232448, "shared memory budget");

struct MxArgs {
  const uint8_t* w;
  const uint8_t* rows;
  const int32_t* counts;
  const int32_t* offsets;
  int* split_cnt;        // [kMxMaxCtas] parts arrived, zero between launches
  float* partial;        // [kMxMaxCtas][tile of the pair][tokens / 4][128 weight rows][4]
  uint16_t* C;
  int* status;
  int E, N, K, ldc, capacity, n_tiles, max_tok;
  int test_timeout;      // test of the timeout path: no item is handed out, waits for one are short
  size_t rows_padded;
};

// Largest row tile.  A full tile's accumulators fill TMEM, so its epilogue
// (3.2 us) is not hidden; tiles of 96 have two accumulators and four stages,
// but draw the weights from L2 twice as often (0.8 us against 0.6 us per unit
// and 224 rows).  They even out at about 15 units.
constexpr int kShortTok = 96, kShortUnits = 14;
inline int largest_tile(int units) { return units <= kShortUnits ? kShortTok : kMaxTok; }
__device__ __forceinline__ int row_tiles(int cnt, int max_tok) {
  return max_tok == kMaxTok ? (cnt + kMaxTok - 1) / kMaxTok : (cnt + kShortTok - 1) / kShortTok;
}
// a / b for 0 <= a < 2^24, 0 < b and a quotient below 2^20 (the correction
// makes up for a division that is one off): a launch's first instructions are
// fetched as they run, and an integer division is three times as many.
__device__ __forceinline__ int small_div(int a, int b) {
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  q -= q * b > a;
  q += (q + 1) * b <= a;
  return q;
}
__device__ __forceinline__ float approx_sqrt(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Rows of an expert's row tiles: equal to within the rounding to 16.
__device__ __forceinline__ int tile_rows(int cnt, int n_rt) {
  return ((n_rt > 1 ? (cnt + n_rt - 1) / n_rt : cnt) + 15) & ~15;
}

// A CTA's segments: its part of the divided items [0, cut), if it has one,
// then its whole items.  Items: experts in order; per expert, weight tile
// pairs; per pair, row tiles.
struct Plan {
  const int* prefix;                 // shared: first item of each expert
  const int32_t *cnts, *offs;        // rows and first row of each expert (checked where it has items)
  int E, n_tiles, units, max_tok, items, cut;
  int parts;                         // of a divided item: CTA i has part i % parts of item i / parts
  int chunks;                        // runs of rows per single tile, 0: divided along K
};

// A segment as the roles read it (two 16-byte words).
struct alignas(16) Seg {
  int item, e, row0, rows;           // rows 0: the end of the work
  int tile, tiles, u0, u1;           // first weight tile and tiles; K units
};

// Run by the item warp (the search for the expert is one ballot of 32).
struct Walk {
  const Plan& p;
  int item, e;
  int row0, rows, tile, tiles, u0, u1;
  bool more;

  __device__ explicit Walk(const Plan& plan) : p(plan), item(-1), e(0), u0(0), u1(plan.units) {
    const int cta = blockIdx.x;
    if (cta < p.cut * p.parts) {
      item = small_div(cta, p.parts);
      const int part = cta - item * p.parts;
      more = true;
      locate();
      if (!p.chunks) {
        u0 = small_div(part * p.units, p.parts);
        u1 = small_div((part + 1) * p.units, p.parts);
        return;
      }
      const int t = part >= p.chunks, c = part - t * p.chunks;   // one tile, one run of rows
      const int run = (small_div(rows + p.chunks - 1, p.chunks) + 15) & ~15;
      tile += t;
      tiles -= t;
      if (tiles > 1) tiles = 1;
      row0 += c * run;
      rows = min(run, rows - c * run);
      if (rows > 0 && tiles > 0) return;
    }
    advance();
  }
  __device__ void advance() {
    u0 = 0;
    u1 = p.units;
    item = item < p.cut ? p.cut + static_cast<int>(blockIdx.x) : item + static_cast<int>(gridDim.x);
    more = item < p.items;
    if (more) locate();
  }
  // The item's expert: the largest e with prefix[e] <= item (items only grow).
  __device__ void locate() {
    const int lane = threadIdx.x & 31;
    auto past = [&](int at) { return __ballot_sync(0xffffffffu, at > p.E || p.prefix[at] > item); };
    uint32_t found = past(e + 1 + lane);
    if (!found) {                    // further on: the 32nd of the experts, then the expert
      const int block = (p.E + 31) / 32;
      static_assert(kMaxExperts <= 32 * 32, "two steps of 32");
      e = block * (__ffs(past(min(block * (lane + 1), p.E))) - 1);
      found = past(e + 1 + lane);
    }
    e += __ffs(found) - 1;
    const int cnt = ld_ca(p.cnts + e), local = item - p.prefix[e];
    row0 = ld_ca(p.offs + e);
    rows = cnt;
    tile = kPair * local;
    if (cnt > p.max_tok) {           // several row tiles (divisions: about 100 cycles each)
      const int n_rt = row_tiles(cnt, p.max_tok), pair = local / n_rt;
      const int rt = local - pair * n_rt, per = tile_rows(cnt, n_rt);
      row0 += rt * per;
      rows = min(per, cnt - rt * per);
      tile = kPair * pair;
    }
    tiles = min(kPair, p.n_tiles - tile);
  }
};

// A role's end of the item ring.
struct ItemRing {
  uint64_t *full, *empty;
  const Seg* slots;
  uint32_t polls;
  int slot, ph;
  // The next segment: false at the end of the work or on a timeout.  All
  // lanes of the calling warp take it; lane 0 releases the slot.
  __device__ __forceinline__ bool next(Seg& s, int* status) {
    if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], ph, status, polls))) return false;
    const int4* src = reinterpret_cast<const int4*>(&slots[slot]);
    const int4 lo = src[0], hi = src[1];
    s.item = lo.x, s.e = lo.y, s.row0 = lo.z, s.rows = lo.w;
    s.tile = hi.x, s.tiles = hi.y, s.u0 = hi.z, s.u1 = hi.w;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[slot]);
    if (++slot == kItemSlots) slot = 0, ph ^= 1;
    return s.rows > 0;
  }
};

// Whether `ok` holds in all threads of the epilogue warps.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "n"(kEpiThreads)
      : "memory");
  return r != 0;
}

// With the exponential of -|g|, whose value and divisor stay within range: the
// divisor 1 + exp(-g) is past 2^126, where __fdividef gives 0, for g below -87.3.
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float t = __expf(-fabsf(g));
  return __fdividef(g < 0.f ? g * t : g, 1.0f + t) * u;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four 8 x 8 matrices of 16-bit values from the fragment layout (register i:
// row lane / 4 of matrix i, columns 2 (lane % 4) and + 1), transposed: lane
// 8 i + c gives the 16-byte place of matrix i's column c.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}

// Up to 32 tokens of a finished item to C: this warp's accumulators of its 32
// weight rows (lo: rows 0-15 of the lane quarter, hi: rows 16-31, gate and up),
// `n` tokens at `out`, through the warp's own staging rows.
template <bool kGateUp>
__device__ __forceinline__ void store_tokens(const MxArgs& a, const uint32_t (&lo)[16], const uint32_t (&hi)[16],
                                             uint16_t* out, uint32_t stage_s, int tile, int q, int lane, int n) {
  // lane 8 i + c: token c of its 8-token group, weight rows 8 (i & 1) on
  const uint32_t dst = stage_s + ((lane & 7) + 8 * (lane >> 4)) * kOutPitch + ((lane >> 3) & 1) * 16;
  // 16 bytes (8 columns of C) per lane: 2 or 4 lanes per token
  constexpr int sh = kGateUp ? 1 : 2;
  const int part = lane & ((1 << sh) - 1);
  const int col = (kGateUp ? 64 * tile + 16 * q : kMxTileRows * tile + 32 * q) + 8 * part;
#pragma unroll
  for (int p = 0; p < 2; ++p) {   // tokens 16 p .. 16 p + 15
    uint32_t l[4], h[4];          // [token group of 8][weight rows 0-7, 8-15]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * p + 2 * i;
      const float l0 = __uint_as_float(lo[r]), l1 = __uint_as_float(lo[r + 1]);
      const float h0 = __uint_as_float(hi[r]), h1 = __uint_as_float(hi[r + 1]);
      l[i] = kGateUp ? bf16_pair(silu_mul(l0, h0), silu_mul(l1, h1)) : bf16_pair(l0, l1);
      h[i] = bf16_pair(h0, h1);
    }
    stmatrix_x4_trans(dst + 16 * p * kOutPitch, l[0], l[1], l[2], l[3]);
    if (!kGateUp) stmatrix_x4_trans(dst + 16 * p * kOutPitch + 32, h[0], h[1], h[2], h[3]);
  }
  __syncwarp();
  uint4 v[1 << sh];
#pragma unroll
  for (int j = 0; j < (1 << sh); ++j)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w)
                 : "r"(stage_s + ((lane >> sh) + j * (32 >> sh)) * kOutPitch + 16 * part)
                 : "memory");
  if (col < a.ldc) {
#pragma unroll
    for (int j = 0; j < (1 << sh); ++j) {
      const int token = (lane >> sh) + j * (32 >> sh);
      if (token < n) *reinterpret_cast<uint4*>(out + static_cast<size_t>(token) * a.ldc + col) = v[j];
    }
  }
  __syncwarp();
}

// Eight tokens of a summed item (this lane's weight row `lrow` of tile
// `tile`), `n` of them valid, at `out`.
template <bool kGateUp>
__device__ __forceinline__ void store_columns(const float (&v)[8], uint16_t* out, int ldc, int tile, int lrow,
                                              int n) {
  if (kGateUp) {
    // lanes 0-15 hold gate rows, 16-31 the up rows of the same indices: of
    // two columns, the low lanes finish the first and the high lanes the second
    const bool up = lrow & 16;
    const int col = (kMxTileRows / 2) * tile + 16 * (lrow / 32) + (lrow & 15);
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[c] : v[c + 1], 16);
      const float h = silu_mul(up ? other : v[c], up ? v[c + 1] : other);
      const int cc = c + (up ? 1 : 0);
      if (cc < n && col < ldc) out[static_cast<size_t>(cc) * ldc + col] = f32_to_bf16_rn(h);
    }
  } else {
    const int col = kMxTileRows * tile + lrow;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < n && col < ldc) out[static_cast<size_t>(c) * ldc + col] = f32_to_bf16_rn(v[c]);
  }
}

// The sum of an item's parts first .. last in K order, to C (this lane's weight
// row).  Twelve 16-byte loads in flight: six parts of eight tokens, or twelve
// parts of four where an item has more (one token's items have nine).  Parts
// past the last and tokens past the rows are loaded again, not added.
template <bool kGateUp>
__device__ __forceinline__ void add_parts(const float* partial, int first, int last, int rows, uint16_t* out, int ldc,
                                       int tile, int lrow) {
  auto add = [&](auto parts_c, auto quads_c) {
    constexpr int kParts = decltype(parts_c)::value, kQuads = decltype(quads_c)::value;
    for (int c0 = 0; c0 < rows; c0 += 4 * kQuads) {
      float f[8] = {};
      for (int p0 = first; p0 <= last; p0 += kParts) {
        float4 x[kParts][kQuads];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const int p = min(p0 + i, last);
          const float* src = partial + static_cast<size_t>(p) * kSlotFloats + c0 * 128;
#pragma unroll
          for (int c = 0; c < kQuads; ++c) x[i][c] = ld_cg_f4(src + (c0 + 4 * c < rows ? 512 * c : 0));
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          if (p0 + i <= last)
#pragma unroll
            for (int c = 0; c < kQuads; ++c) {
              f[4 * c] += x[i][c].x, f[4 * c + 1] += x[i][c].y;
              f[4 * c + 2] += x[i][c].z, f[4 * c + 3] += x[i][c].w;
            }
      }
      store_columns<kGateUp>(f, out + static_cast<size_t>(c0) * ldc, ldc, tile, lrow, min(rows - c0, 4 * kQuads));
    }
  };
  if (last - first < 6) add(std::integral_constant<int, 6>{}, std::integral_constant<int, 2>{});
  else add(std::integral_constant<int, 12>{}, std::integral_constant<int, 1>{});
}

template <bool kGateUp>
__global__ void __launch_bounds__(kThreads, 1) mxfp4_gemm_kernel(MxArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], sf_full[kSfSlots], sf_empty[kSfSlots];
  __shared__ __align__(8) uint64_t tfull[kMaxAcc], tempty[kMaxAcc], done_bar[kPair];
  __shared__ __align__(8) uint64_t item_full[kItemSlots], item_empty[kItemSlots];
  __shared__ Seg item_slots[kItemSlots];
  __shared__ uint32_t tmem_base_s;
  __shared__ int prefix[kMaxExperts + 1];
  __shared__ int warp_sum[kThreads / 32], warp_max[kThreads / 32];
  __shared__ int hdr_ok, last_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem0 - smem_u32(smem_raw));

  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kPair);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_empty[s], kPair);
    }
    for (int b = 0; b < kMaxAcc; ++b) {
      mbar_init(&tfull[b], kPair);
      mbar_init(&tempty[b], kEpiWarps);
    }
    for (int t = 0; t < kPair; ++t) mbar_init(&done_bar[t], 1);
    for (int q = 0; q < kItemSlots; ++q) {
      mbar_init(&item_full[q], 1);
      mbar_init(&item_empty[q], kItemReaders);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base_s, kTmemCols);
  // programmatic launch: nothing above touches global memory
  grid_dep_wait();
  grid_dep_launch();
  uint4 h0{}, h1{};   // the weights' header, on its way while the counts are read
  if (tid == kThreads - 1) {
    h0 = ld_cg_v4(a.w);
    h1 = ld_cg_v4(a.w + 16);
  }

  // first item of each expert, and the largest row tile: thread i covers
  // experts [i * per, (i + 1) * per)
  const int per = 1 + (a.E > kThreads) + (a.E > 2 * kThreads);
  static_assert(3 * kThreads >= kMaxExperts, "three experts per thread at most");
  const int n_pairs = (a.n_tiles + kPair - 1) / kPair;
  int mine = 0, most = 16;
#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e >= a.E) break;
    int cnt = ld_ca(a.counts + e);
    const int off = ld_ca(a.offsets + e), next = ld_ca(a.offsets + e + 1);
    const bool alone = cnt >= 0 && off >= 0 && off % 8 == 0 && cnt <= a.capacity && off <= a.capacity - cnt;
    // Experts that end before the next one begins have disjoint rows, so that
    // the items number at most what the host has checked.
    if (!alone || off + cnt > next) {
      set_status(a.status, CHORD_ERR_INVALID_ARG);   // not an aligned order of `capacity` rows
      if (alone || off > next) most = kNoOrder;
      cnt = 0;
    }
    prefix[e] = mine;
    if (cnt > 0) {
      const int n_rt = cnt <= a.max_tok ? 1 : row_tiles(cnt, a.max_tok);
      mine += n_pairs * n_rt;
      most = max(most, tile_rows(cnt, n_rt));
    }
  }
  if (tid == kThreads - 1) {
    hdr_ok = h0.x == kMxMagic && h0.y == kMxVersion && static_cast<int>(h0.z) >= a.E &&
             static_cast<int>(h0.w) == a.N && static_cast<int>(h1.x) == a.K && static_cast<int>(h1.y) == (kGateUp ? 1 : 0);
    if (!hdr_ok) set_status(a.status, CHORD_ERR_PREPACK_MISMATCH);
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    warp_sum[warp] = inc;
    warp_max[warp] = most;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // every warp adds up the warps' sums itself
  int sum = lane < kThreads / 32 ? warp_sum[lane] : 0;
  int tok = lane < kThreads / 32 ? warp_max[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += t;
  }
  tok = __reduce_max_sync(0xffffffffu, tok);
  const int run = inc - mine + (warp ? __shfl_sync(0xffffffffu, sum, warp - 1) : 0);

#pragma unroll 1
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e >= a.E) break;
    prefix[e] += run;
  }
  if (tid == kThreads - 1) prefix[a.E] = run + mine;   // the last thread ends at the total
  __syncthreads();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, tmem_base_s, 0);
  tok = __shfl_sync(0xffffffffu, tok, 0);
  const int units = mx_units(a.K), ctas = gridDim.x;
  Plan plan;
  plan.prefix = prefix, plan.cnts = a.counts, plan.offs = a.offsets;
  plan.E = a.E, plan.n_tiles = a.n_tiles, plan.units = units, plan.max_tok = a.max_tok;
  plan.items = hdr_ok && tok <= kMaxTok ? prefix[a.E] : 0;
  plan.cut = plan.items % ctas;
  // The items that are left over when each CTA has had the same number are
  // divided where that leaves every CTA one part at most; otherwise they are
  // dealt like the others (128 items of 28 units on 152 CTAs took 20.3 us, cut
  // into 152 ranges of K 23.8: fewer CTAs at work draw more each).  A unit
  // takes about 0.4 us.  Adding up an item's parts takes tok / 80 of a unit
  // for each (8 ns a token), so a part has at least the square root of units *
  // tok / 80 units, and about kSplitUnits units' time besides (less where
  // whole items follow and hide it), which the division has to save: one
  // token's 32 items of 3 units take 6.6 us undivided and 7.7 divided, of 16
  // units 11.7 and 9.7.
  plan.chunks = 0;
  plan.parts = plan.cut > 0 ? small_div(ctas, plan.cut) : 0;
  if (tok > kSplitTok) {
    plan.chunks = min(plan.parts / kPair, tok / 16);
    plan.parts = kPair * plan.chunks;
  } else {
    const int least = max(1, static_cast<int>(approx_sqrt(units * tok * (1 / 80.f))));
    plan.parts = min(plan.parts, small_div(units, least));
    const int saved = units - small_div(units + plan.parts - 1, max(plan.parts, 1));
    if (saved < (plan.items > plan.cut ? kSplitUnitsHidden : kSplitUnits)) plan.parts = 0;
  }
  if (plan.parts < 2) plan.cut = plan.parts = 0;
  const int stage = stage_bytes(tok), n_stages = min(kMaxStages, kStageBudget / stage);
  const int n_acc = min(kMaxAcc, kSfCol / (kPair * tok));
  ItemRing items{item_full, item_empty, item_slots, a.test_timeout ? kTestWaitPolls : kWaitPolls, 0, 0};
  Seg w;

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    // The whole warp runs the loop, one elected lane issues.
    const size_t tile_bytes = static_cast<size_t>(units) * kMxUnitBytes;
    int it = 0, st = 0, ph = 0;
    bool ok = true;
    while (ok && items.next(w, a.status)) {
      const int n16 = (w.rows + 15) & ~15;
      int u = w.u0;
      const int t0 = w.tile % kPair;
      const int step = min(kPair, a.n_tiles - (w.tile - t0)) * kMxUnitBytes;   // the pair's unit
      const uint8_t* wsrc = a.w + kPackHeaderBytes +
                            (static_cast<size_t>(w.e) * a.n_tiles + w.tile - t0) * tile_bytes +
                            static_cast<size_t>(u) * step + t0 * kMxUnitBytes;
      // the tile's rows: up to the end of their slab, then the next one's
      const int head = min(n16, kMxSlabRows - w.row0 % kMxSlabRows);
      const uint8_t* rsrc = a.rows + mx_row_place(u, units, w.row0) * kMxRowBytes;
      const uint8_t* rsrc2 = a.rows + mx_row_place(u, units, w.row0 + head) * kMxRowBytes;
      for (; u < w.u1; ++u, ++it) {
        if (it >= n_stages && !(ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1, a.status)))) break;
        const uint32_t dst = smem0 + st * stage;
        mbar_arrive_expect_tx_elect(&full[st], w.tiles * kMxUnitBytes + n16 * kMxRowBytes);
        bulk_g2s_elect(dst, wsrc, w.tiles * kMxUnitBytes, &full[st]);
        bulk_g2s_elect(dst + kBOff, rsrc, head * kMxRowBytes, &full[st]);
        if (head < n16)
          bulk_g2s_elect(dst + kBOff + head * kMxRowBytes, rsrc2, (n16 - head) * kMxRowBytes, &full[st]);
        wsrc += step;
        rsrc += kMxSlabRows * kMxRowBytes;
        rsrc2 += kMxSlabRows * kMxRowBytes;
        if (++st == n_stages) st = 0, ph ^= 1;
      }
    }
    // every issued copy lands before the CTA can exit
    for (int j = max(0, it - n_stages); j < it; ++j) mbar_wait(&full[j % n_stages], (j / n_stages) & 1, a.status);
  } else if (warp == kSfWarp) {
    // --------------------------------------------------- row scales to blocks
    // Slot reuse waits for the MMAs of a unit that was signalled already, so
    // the wait always ends.
    const uint8_t* row_scales = a.rows + units * a.rows_padded * kMxRowBytes;
    int issued = 0, signalled = 0, in = 0, in_ph = 0, out = 0;
    bool ok = true;
    auto signal = [&] {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sf_full[out]);
      ++signalled;
      if (++out == kSfSlots) out = 0;
    };
    while (ok && items.next(w, a.status)) {
      const int n16 = (w.rows + 15) & ~15;
      // this lane's rows of the tile, 32 apart: those below `head` are in the
      // first slab, the others in the next
      const int head = kMxSlabRows - w.row0 % kMxSlabRows;
      const uint8_t* src = row_scales + mx_row_place(w.u0, units, w.row0 + lane) * kMxRowScales;
      const size_t slab = static_cast<size_t>(units - 1) * kMxSlabRows * kMxRowScales;
      for (int u = w.u0; u < w.u1; ++u, ++issued) {
        if (issued >= kSfSlots && !(ok = __all_sync(0xffffffffu, mbar_wait(&sf_empty[in], in_ph ^ 1, a.status))))
          break;
        const uint32_t dst = smem0 + kSfOff + in * kSfSlotBytes + lane * 16;
#pragma unroll
        for (int i = 0; i < (kMaxTok + 31) / 32; ++i) {
          const int r = 32 * i + lane;
          if (r < n16) {
            const uint8_t* at = src + 32 * i * kMxRowScales + (lane < head && r >= head ? slab : 0);
            cp_async4(dst + (i / 4) * 512 + (i % 4) * 4, at);
            cp_async4(dst + (i / 4) * 512 + (i % 4) * 4 + kSfbHalf, at + 4);
          }
        }
        cp_async_commit();
        src += kMxSlabRows * kMxRowScales;
        if (++in == kSfSlots) in = 0, in_ph ^= 1;
        if (issued + 1 - signalled == kSfAhead) {
          cp_async_wait<kSfAhead - 1>();
          signal();
        }
      }
    }
    cp_async_wait<0>();
    while (ok && signalled < issued) signal();
  } else if (warp >= kMmaWarp0 && warp < kMmaWarp0 + kPair) {
    // ------------------------------------------------------------------ MMAs
    // One warp per weight tile; the whole warp runs the loop, one elected
    // lane issues.  Both commit every unit and item, also a tile that the
    // item lacks.
    const int t = warp - kMmaWarp0;
    int st = 0, ph = 0, slot = 0, sf_ph = 0, acc = 0, use = 0;
    const uint32_t sfb = tmem_base + kSfCol + t * kSfCols + 16;
    uint32_t sfa = sfb - 16;
    bool issued = false, ok = true;
    while (ok && items.next(w, a.status)) {
      const int n16 = (w.rows + 15) & ~15;
      const bool active = t < w.tiles;
      const uint32_t d = tmem_base + (acc * kPair + t) * tok;
      const uint32_t idesc0 = idesc_mxf4(n16, 0), idesc2 = idesc_mxf4(n16, 2);
      uint32_t accumulate = 0;
      if (use >= 1) ok = mbar_wait(&tempty[acc], (use - 1) & 1, a.status);
      for (int left = w.u1 - w.u0; left > 0; --left) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait2(&full[st], ph, &sf_full[slot], sf_ph, a.status));
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const uint32_t base = smem0 + st * stage, wt = base + t * kMxUnitBytes;
          tc_mxf4_scales_elect<kSfbHalf>(scales_desc(smem0 + kSfOff + slot * kSfSlotBytes), sfb, n16 > 128);
          tc_mxf4_unit_elect(d, sw128_kmajor_desc(wt), sw128_kmajor_desc(base + kBOff), scales_desc(wt + kMxTileBytes),
                             sfa, sfb, idesc0, idesc2, accumulate);
        }
        tc_commit2_elect(&empty[st], &sf_empty[slot]);
        sfa = 2 * sfb - 24 - sfa;   // the other of the two sets: sfb - 16, sfb - 8
        accumulate = 1;
        issued = true;
        if (++st == n_stages) st = 0, ph ^= 1;
        if (++slot == kSfSlots) slot = 0, sf_ph ^= 1;
      }
      if (!ok) break;
      tc_commit_elect(&tfull[acc]);
      if (++acc == n_acc) acc = 0, ++use;
    }
    // all issued MMAs complete before TMEM can be freed
    if (issued) {
      tc_commit_elect(&done_bar[t]);
      mbar_wait(&done_bar[t], 0, a.status);
    }
  } else if (warp == kItemWarp) {
    // ----------------------------------------------------------------- items
    Walk walk(plan);
    int slot = 0, ph = 0;
    for (bool first = true, more = !a.test_timeout; more;) {
      if (!first && !__all_sync(0xffffffffu, mbar_wait_backoff(&item_empty[slot], ph ^ 1, a.status))) break;
      more = walk.more;
      if (lane == 0) {
        Seg& s = item_slots[slot];
        s.item = walk.item, s.e = walk.e, s.row0 = walk.row0, s.rows = more ? walk.rows : 0;
        s.tile = walk.tile, s.tiles = walk.tiles, s.u0 = walk.u0, s.u1 = walk.u1;
        mbar_arrive(&item_full[slot]);   // release: the segment is visible to the waiters
      }
      if (more) walk.advance();
      if (++slot == kItemSlots) slot = 0, ph ^= 1, first = false;
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3, lrow = 32 * q + lane;        // TMEM lane quarter; weight row of the tile
    const int t = (warp - kEpiWarp0) / 4;                // weight tile of the pair
    const uint32_t out_stage = smem0 + kOutOff + (warp - kEpiWarp0) * kOutBytes;
    int acc = 0, use = 0;
    // A wait that ran out ends a warp; at a segment cut along K, whose
    // handling has barriers, the epilogue warps end together.
    bool cut_next = !plan.chunks && static_cast<int>(blockIdx.x) < plan.cut * plan.parts;
    while (true) {
      const bool on = items.next(w, a.status);
      bool ok = on && __all_sync(0xffffffffu, mbar_wait(&tfull[acc], use & 1, a.status));
      if (cut_next) {
        cut_next = false;
        ok = epilogue_all(ok);
      }
      if (!ok) break;
      tc_fence_after();
      const int rows = t < w.tiles ? w.rows : 0;
      const uint32_t taddr = tmem_base + (acc * kPair + t) * tok + (static_cast<uint32_t>(32 * q) << 16);
      uint16_t* out = a.C + static_cast<size_t>(w.row0) * a.ldc;
      const bool whole = w.u0 == 0 && w.u1 == units;
      const size_t part = static_cast<size_t>(t) * kSplitTok * 128 + 4 * lrow;
      float* mine_p = a.partial + static_cast<size_t>(blockIdx.x) * kSlotFloats + part;
      if (whole) {
        // the next 32 tokens' accumulators are on their way while these go out
        uint32_t next[2][16];
        auto load = [&](int c0) {
          tmem_ld_16x256b_x4(taddr + c0, next[0]);
          tmem_ld_16x256b_x4(taddr + c0 + (16u << 16), next[1]);
        };
        if (rows > 0) load(0);
#pragma unroll 1
        for (int c0 = 0; c0 < rows; c0 += 32) {
          tmem_ld_wait();
          uint32_t v[2][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[0][i] = next[0][i], v[1][i] = next[1][i];
          if (c0 + 32 < rows) load(c0 + 32);
          store_tokens<kGateUp>(a, v[0], v[1], out + static_cast<size_t>(c0) * a.ldc, out_stage, w.tile + t, q, lane,
                                rows - c0);
        }
      } else {
        for (int c0 = 0; c0 < rows; c0 += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c0, v);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            if (c0 + c < rows)
              *reinterpret_cast<uint4*>(mine_p + (c0 + c) * 128) = make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == n_acc) acc = 0, ++use;
      if (whole) continue;
      // a cut item: the CTA that arrives last adds the parts in K order
      const int first = w.item * plan.parts, last = first + plan.parts - 1;
      epilogue_all(true);
      if (tid == 32 * kEpiWarp0) {
        // releases the parts stored by all threads before the barrier, and
        // acquires the others'
        int arrived;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                     : "=r"(arrived)
                     : "l"(a.split_cnt + first)
                     : "memory");
        last_flag = arrived == last - first;
      }
      epilogue_all(true);
      if (!last_flag) continue;
      if (tid == 32 * kEpiWarp0) a.split_cnt[first] = 0;   // for the next launch
      add_parts<kGateUp>(a.partial + part, first, last, rows, out, a.ldc, w.tile + t, lrow);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

}  // namespace

size_t mxfp4_gemm_workspace_bytes() {
  return kMxMaxCtas * sizeof(int) + static_cast<size_t>(kMxMaxCtas) * kSlotFloats * sizeof(float);
}

cudaError_t mxfp4_gemm_launch(const uint8_t* rows, const uint8_t* w, int E, int N, int K, const int32_t* counts,
                              const int32_t* offsets, int capacity, bool gate_up, uint16_t* C, void* ws,
                              bool test_timeout, int* status, cudaStream_t st) {
  MxArgs a{};
  a.test_timeout = test_timeout ? 1 : 0;
  a.w = w, a.rows = rows, a.counts = counts, a.offsets = offsets;
  a.split_cnt = static_cast<int*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kMxMaxCtas * sizeof(int));
  a.C = C, a.status = status;
  a.E = E, a.N = N, a.K = K, a.ldc = gate_up ? N / 2 : N, a.capacity = capacity;
  a.n_tiles = mx_tiles(N), a.max_tok = largest_tile(mx_units(K));
  a.rows_padded = mx_rows_padded(capacity);
  cudaError_t err = gate_up ? ensure_smem_limit<mxfp4_gemm_kernel<true>>(kSmemBytes)
                            : ensure_smem_limit<mxfp4_gemm_kernel<false>>(kSmemBytes);
  if (err != cudaSuccess) return err;
  return launch_kernel(gate_up ? mxfp4_gemm_kernel<true> : mxfp4_gemm_kernel<false>, dim3(sm_count() < kMxMaxCtas ? sm_count() : kMxMaxCtas), dim3(kThreads),
                       kSmemBytes, st, true, a);
}

}  // namespace chord
