// The experts' product in MXFP4 on the 5th-generation tensor cores:
//   C[r, n] = sum_k A[r, k] W[e(r), n, k]
// over rows in the aligned expert order, both operands E2M1 with E8M0 scales
// per 32 of K, FP32 accumulation, with an optional SiLU(gate) * up.
//
// Design on sm_103a (one persistent CTA per SM):
//   * an item is two tiles of 128 weight rows (two MMAs of M = 128 on the same
//     rows) times up to kMaxTok of an expert's rows (N, a multiple of 16), so
//     one decoded token costs 16 columns, not 128 rows; one kernel serves
//     decoding and prefill.  Every SM draws its operands from L2 at about
//     60 GB/s, which bounds all sizes above a few dozen rows per expert: a
//     second weight tile on the same rows brings 66 KB for what took 100;
//   * the work is the list of items times their K units of 256, cut into one
//     contiguous range per CTA of equal length to within a unit.  Every SM
//     streams the same number of bytes whatever the number of items, and one
//     token's few items spread over all SMs.  An item that a range boundary
//     cuts is summed by the CTA that finishes last, from FP32 partials in
//     workspace, in K order, so results do not depend on timing;
//   * per unit and weight tile one bulk copy brings 128 weight rows with their
//     scales (17 KB, contiguous, already swizzled), one more the rows and one
//     the rows' scales;
//   * the rows' scales arrive in row order; warp 2 rearranges them into the
//     block layout in shared memory; tcgen05.cp moves both operands' scales
//     to TMEM ahead of the MMAs of the unit, in order with them;
//   * stages and accumulators are laid out for the launch's largest row tile,
//     which every CTA finds from the counts: decoding has five stages and four
//     accumulators, a full tile three stages and one accumulator.
// TMEM: accumulators from column 0, scales from column 480.
// Every mbarrier wait is bounded; on a timeout the CTA records
// CHORD_ERR_TIMEOUT, drains its own copies and MMAs, frees TMEM and exits.
#include "common.cuh"
#include "kernels.h"
#include "mxfp4.cuh"
#include "tc5.cuh"

namespace chord {
namespace {

constexpr int kMaxTok = 240;
constexpr int kPair = 2;               // weight tiles per item
constexpr int kMaxStages = 5, kMaxAcc = 4;
constexpr int kEpiWarp0 = 4, kEpiWarps = 4 * kPair, kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 32 * kEpiWarp0 + kEpiThreads;
constexpr int kMaxExperts = 1024;
// stage: weight tiles with their scales | rows | row scales as they arrive |
// row scales in block layout (two K halves of up to 256 rows)
constexpr int kBOff = kPair * kMxUnitBytes;
constexpr int kSfbHalf = 1024;
__host__ __device__ constexpr int stage_bytes(int tok) {
  return (kBOff + tok * (kMxRowBytes + kMxRowScales) + 2 * kSfbHalf + 1023) / 1024 * 1024;
}
constexpr int kStageBudget = 3 * stage_bytes(kMaxTok);
constexpr int kSmemBytes = kStageBudget + 1024;
constexpr int kSfCol = 480;            // SFA of tile t, half h at +8 t + 4 h; SFB half h at +16 + 8 h
constexpr int kTmemCols = 512;
constexpr int kSlotFloats = kPair * kMaxTok * 128;   // one CTA's part of a cut item
static_assert(kPair * kMaxTok <= kSfCol && kSfCol + 32 <= kTmemCols, "TMEM budget");
static_assert(kBOff % 1024 == 0 && kMaxTok % 16 == 0 && kMaxTok <= 256, "stage layout");
static_assert(kMaxStages * stage_bytes(16) <= kStageBudget, "stage budget");
static_assert(kSmemBytes + (3 * kMaxExperts + 1) * 4 + 1024 <= 232448, "shared memory budget");

struct MxArgs {
  const uint8_t* w;
  const uint8_t* rows;
  const int32_t* counts;
  const int32_t* offsets;
  int* split_cnt;        // [kMxMaxCtas], zero between launches
  float* partial;        // [2 * kMxMaxCtas][kSlotFloats]
  uint16_t* C;
  int* status;
  int E, N, K, ldc, capacity, n_tiles, gate_up;
  size_t rows_padded;
};

__device__ __forceinline__ int row_tiles(int cnt) { return (cnt + kMaxTok - 1) / kMaxTok; }
// Rows of an expert's row tiles: equal to within the rounding to 16.
__device__ __forceinline__ int tile_rows(int cnt, int n_rt) { return ((cnt + n_rt - 1) / n_rt + 15) & ~15; }

// A role's walk over the CTA's range of (item, K unit).  Items: experts in
// order; per expert, weight tile pairs; per pair, row tiles (the pair's
// weights are in L2 for the second).
struct Walk {
  const int *cnts, *offs;
  int E, n_tiles, units;
  long long left;              // units of the range not yet taken
  int e, cnt, n_rt, per, pair, rt, u0, u1;

  __device__ void expert(int at) {
    e = at;
    cnt = cnts[at];
    n_rt = row_tiles(cnt);
    per = n_rt ? tile_rows(cnt, n_rt) : 0;
  }
  __device__ void cut() { u1 = left < units - u0 ? u0 + static_cast<int>(left) : units; }
  __device__ Walk(const int* prefix, const int* c, const int* o, int E_, int tiles, int units_, long long begin,
                  long long end)
      : cnts(c), offs(o), E(E_), n_tiles(tiles), units(units_), left(end - begin) {
    if (left <= 0) return;
    const int item = static_cast<int>(begin / units);
    u0 = static_cast<int>(begin - static_cast<long long>(item) * units);
    int lo = 0, hi = E - 1;    // largest e with prefix[e] <= item
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= item) lo = mid; else hi = mid - 1;
    }
    expert(lo);
    pair = (item - prefix[lo]) / n_rt;
    rt = item - prefix[lo] - pair * n_rt;
    cut();
  }
  __device__ void next() {
    left -= u1 - u0;
    if (left <= 0) return;
    u0 = 0;
    if (++rt == n_rt) {
      rt = 0;
      if (++pair * kPair >= n_tiles) {
        pair = 0;
        do expert(e + 1);      // units are left, so an expert with rows follows
        while (cnt == 0);
      }
    }
    cut();
  }
  __device__ int row0() const { return offs[e] + rt * per; }
  __device__ int rows() const { return min(per, cnt - rt * per); }
  __device__ int tiles() const { return min(kPair, n_tiles - kPair * pair); }
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

// 32 columns of accumulators (this lane's weight row `lrow` of tile `tile`)
// into rows c0 .. of C; `out` is C's row of column 0, `n` the valid columns.
__device__ __forceinline__ void store_columns(const MxArgs& a, const uint32_t (&v)[32], uint16_t* out, int tile,
                                              int lrow, int n) {
  if (a.gate_up) {
    // lanes 0-15 hold gate rows, 16-31 the up rows of the same indices: of
    // two columns, the low lanes finish the first and the high lanes the second
    const bool up = lrow & 16;
    const int col = (kMxTileRows / 2) * tile + 16 * (lrow / 32) + (lrow & 15);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float other = __uint_as_float(__shfl_xor_sync(0xffffffffu, up ? v[c] : v[c + 1], 16));
      const float g = up ? other : __uint_as_float(v[c]);
      const float h = __fdividef(g, 1.0f + __expf(-g)) * (up ? __uint_as_float(v[c + 1]) : other);
      const int cc = c + (up ? 1 : 0);
      if (cc < n && col < a.ldc) out[static_cast<size_t>(cc) * a.ldc + col] = f32_to_bf16_rn(h);
    }
  } else {
    const int col = kMxTileRows * tile + lrow;
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c < n && col < a.ldc) out[static_cast<size_t>(c) * a.ldc + col] = f32_to_bf16_rn(__uint_as_float(v[c]));
  }
}

__global__ void __launch_bounds__(kThreads, 1) mxfp4_gemm_kernel(MxArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], sf_full[kMaxStages], empty[kMaxStages];
  __shared__ __align__(8) uint64_t tfull[kMaxAcc], tempty[kMaxAcc], done_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int prefix[kMaxExperts + 1];
  __shared__ int s_cnt[kMaxExperts], s_off[kMaxExperts];
  __shared__ int warp_sum[kThreads / 32], warp_max[kThreads / 32];
  __shared__ int hdr_ok, last_flag;
  __shared__ volatile int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem0 - smem_u32(smem_raw));

  if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&sf_full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kMaxAcc; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    mbar_init(&done_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base_s, kTmemCols);
  // programmatic launch: nothing above touches global memory
  grid_dep_wait();
  grid_dep_launch();
  if (tid == 0) {
    const int32_t* h = reinterpret_cast<const int32_t*>(a.w);
    hdr_ok = ld_ca(h) == static_cast<int>(kMxMagic) && ld_ca(h + 1) == static_cast<int>(kMxVersion) &&
             ld_ca(h + 2) >= a.E && ld_ca(h + 3) == a.N && ld_ca(h + 4) == a.K && ld_ca(h + 5) == a.gate_up;
    if (!hdr_ok) set_status(a.status, CHORD_ERR_PREPACK_MISMATCH);
  }

  // first item of each expert, and the largest row tile: thread i covers
  // experts [i * per, (i + 1) * per)
  const int per = (a.E + kThreads - 1) / kThreads;
  const int n_pairs = (a.n_tiles + kPair - 1) / kPair;
  int mine = 0, most = 16;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e >= a.E) break;
    int cnt = ld_ca(a.counts + e);
    const int off = ld_ca(a.offsets + e);
    if (cnt < 0 || off < 0 || off % 8 != 0 || cnt > a.capacity || off > a.capacity - cnt) {
      set_status(a.status, CHORD_ERR_INVALID_ARG);   // not an aligned order of `capacity` rows
      cnt = 0;
    }
    s_cnt[e] = cnt;
    s_off[e] = off;
    mine += n_pairs * row_tiles(cnt);
    if (cnt) most = max(most, tile_rows(cnt, row_tiles(cnt)));
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
  int run = inc - mine, tok = 16;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) run += warp_sum[i];
    tok = max(tok, warp_max[i]);
  }
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e >= a.E) break;
    prefix[e] = run;
    run += n_pairs * row_tiles(s_cnt[e]);
  }
  if (tid == kThreads - 1) prefix[a.E] = run;   // the last thread ends at the total
  __syncthreads();
  const uint32_t tmem_base = tmem_base_s;

  const int units = mx_units(a.K);
  const long long total = hdr_ok ? static_cast<long long>(prefix[a.E]) * units : 0;
  // CTAs that take work: all, or as many as there are units (a range is
  // never empty, so the parts of a cut item are in consecutive CTAs)
  const long long G = total < gridDim.x ? total : gridDim.x;
  const long long begin = blockIdx.x < G ? blockIdx.x * total / G : 0;
  const long long end = blockIdx.x < G ? (blockIdx.x + 1) * total / G : 0;
  const int stage = stage_bytes(tok), n_stages = min(kMaxStages, kStageBudget / stage);
  const int raw_off = kBOff + tok * kMxRowBytes, sfb_off = raw_off + tok * kMxRowScales;
  const int n_acc = min(kMaxAcc, kSfCol / (kPair * tok));
  Walk w(prefix, s_cnt, s_off, a.E, a.n_tiles, units, begin, end);

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      const uint8_t* row_scales = a.rows + static_cast<size_t>(units) * a.rows_padded * kMxRowBytes;
      const size_t tile_bytes = static_cast<size_t>(units) * kMxUnitBytes;
      int it = 0, st = 0, ph = 0;
      for (; w.left > 0 && !abort_flag; w.next()) {
        const int n16 = (w.rows() + 15) & ~15, tiles = w.tiles();
        const uint8_t* wsrc =
            a.w + kPackHeaderBytes + (static_cast<size_t>(w.e) * a.n_tiles + kPair * w.pair) * tile_bytes;
        const size_t row0 = w.row0();
        for (int u = w.u0; u < w.u1; ++u, ++it) {
          if (it >= n_stages && !mbar_wait(&empty[st], ph ^ 1, a.status)) {
            abort_flag = 1;
            break;
          }
          uint8_t* dst = smem + st * stage;
          const size_t row = static_cast<size_t>(u) * a.rows_padded + row0;
          mbar_arrive_expect_tx(&full[st], tiles * kMxUnitBytes + n16 * (kMxRowBytes + kMxRowScales));
          for (int t = 0; t < tiles; ++t)
            bulk_g2s(dst + t * kMxUnitBytes, wsrc + t * tile_bytes + static_cast<size_t>(u) * kMxUnitBytes,
                     kMxUnitBytes, &full[st]);
          bulk_g2s(dst + kBOff, a.rows + row * kMxRowBytes, n16 * kMxRowBytes, &full[st]);
          bulk_g2s(dst + raw_off, row_scales + row * kMxRowScales, n16 * kMxRowScales, &full[st]);
          if (++st == n_stages) st = 0, ph ^= 1;
        }
      }
      // every issued copy lands before the CTA can exit
      for (int j = max(0, it - n_stages); j < it; ++j) mbar_wait(&full[j % n_stages], (j / n_stages) & 1, a.status);
    }
  } else if (warp == 2) {
    // --------------------------------------------------- row scales to blocks
    int st = 0, ph = 0;
    for (; w.left > 0 && !abort_flag; w.next()) {
      const int n16 = (w.rows() + 15) & ~15;
      for (int u = w.u0; u < w.u1; ++u) {
        bool ok = mbar_wait(&full[st], ph, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          abort_flag = 1;
          break;
        }
        uint8_t* base = smem + st * stage;
        for (int r = lane; r < n16; r += 32) {
          const uint2 v = *reinterpret_cast<const uint2*>(base + raw_off + r * kMxRowScales);
          uint8_t* dst = base + sfb_off + (r / 128) * 512 + (r % 32) * 16 + (r / 32 % 4) * 4;
          *reinterpret_cast<uint32_t*>(dst) = v.x;
          *reinterpret_cast<uint32_t*>(dst + kSfbHalf) = v.y;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[st]);
        if (++st == n_stages) st = 0, ph ^= 1;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      int st = 0, ph = 0, acc = 0, use = 0;
      bool issued = false;
      for (; w.left > 0 && !abort_flag; w.next()) {
        const int n16 = (w.rows() + 15) & ~15, tiles = w.tiles();
        if (use >= 1 && !mbar_wait(&tempty[acc], (use - 1) & 1, a.status)) {
          abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * kPair * tok, sf = tmem_base + kSfCol;
        const uint32_t idesc[2] = {idesc_mxf4(n16, 0), idesc_mxf4(n16, 2)};
        for (int u = w.u0; u < w.u1; ++u) {
          if (!mbar_wait2(&full[st], ph, &sf_full[st], ph, a.status)) {
            abort_flag = 1;
            break;
          }
          tc_fence_after();
          const uint32_t base = smem0 + st * stage;
          for (int t = 0; t < tiles; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tc_cp_scales(sf + 8 * t + 4 * h, scales_desc(base + t * kMxUnitBytes + kMxTileBytes + 512 * h));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tc_cp_scales(sf + 16 + 8 * h, scales_desc(base + sfb_off + kSfbHalf * h));
            if (n16 > 128) tc_cp_scales(sf + 20 + 8 * h, scales_desc(base + sfb_off + kSfbHalf * h + 512));
          }
          const uint64_t ad = sw128_kmajor_desc(base), bd = sw128_kmajor_desc(base + kBOff);
          for (int t = 0; t < tiles; ++t)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_mxf4(d + t * tok, ad + t * (kMxUnitBytes >> 4) + 2 * kk, bd + 2 * kk, idesc[kk & 1],
                          sf + 8 * t + 4 * (kk >> 1), sf + 16 + 8 * (kk >> 1), u > w.u0 || kk ? 1u : 0u);
          tc_commit(&empty[st]);
          issued = true;
          if (++st == n_stages) st = 0, ph ^= 1;
        }
        if (abort_flag) break;
        tc_commit(&tfull[acc]);
        if (++acc == n_acc) acc = 0, ++use;
      }
      // all issued MMAs complete before TMEM can be freed
      if (issued) {
        tc_commit(&done_bar);
        mbar_wait(&done_bar, 0, a.status);
      }
    }
  } else if (warp >= kEpiWarp0) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3, lrow = 32 * q + lane;        // TMEM lane quarter; weight row of the tile
    const int t = (warp - kEpiWarp0) / 4;                // weight tile of the pair
    int acc = 0, use = 0;
    for (; w.left > 0; w.next()) {
      // all epilogue warps go on or stop together: barriers follow
      if (!epilogue_all(mbar_wait(&tfull[acc], use & 1, a.status))) {
        abort_flag = 1;
        break;
      }
      tc_fence_after();
      const bool active = t < w.tiles();
      const int rows = active ? w.rows() : 0;
      const uint32_t taddr = tmem_base + (acc * kPair + t) * tok + (static_cast<uint32_t>(32 * q) << 16);
      uint16_t* out = a.C + static_cast<size_t>(w.row0()) * a.ldc;
      const bool whole = w.u0 == 0 && w.u1 == units;
      const size_t part = static_cast<size_t>(t) * kMaxTok * 128 + lrow;
      float* mine_p = a.partial + static_cast<size_t>(2 * blockIdx.x + (w.u0 == 0)) * kSlotFloats + part;
      for (int c0 = 0; c0 < rows; c0 += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c0, v);
        tmem_ld_wait();
        if (whole) {
          store_columns(a, v, out + static_cast<size_t>(c0) * a.ldc, kPair * w.pair + t, lrow, rows - c0);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < rows) mine_p[(c0 + c) * 128] = __uint_as_float(v[c]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == n_acc) acc = 0, ++use;
      if (whole) continue;
      // a cut item: the CTA that arrives last adds the parts in K order
      const long long i0 = end - w.left - w.u0;          // the item's units are [i0, i0 + units)
      const int first = static_cast<int>(((i0 + 1) * G - 1) / total);
      const int last = static_cast<int>(((i0 + units) * G - 1) / total);
      __threadfence();
      epilogue_all(true);
      if (tid == 32 * kEpiWarp0) {
        const int done = atomicAdd(a.split_cnt + first, 1) == last - first;
        if (done) atomicExch(a.split_cnt + first, 0);    // zero for the next launch
        last_flag = done;
      }
      epilogue_all(true);
      if (!last_flag) continue;
      __threadfence();
      for (int c0 = 0; c0 < rows; c0 += 32) {
        float f[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) f[c] = 0.f;
        for (int p0 = first; p0 <= last; p0 += 4) {      // four parts' loads in flight
#pragma unroll
          for (int h = 0; h < 32; h += 8) {
            if (c0 + h >= rows) break;
            float x[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int p = min(p0 + i, last);
              const float* src = a.partial + static_cast<size_t>(2 * p + (p == first)) * kSlotFloats + part;
#pragma unroll
              for (int c = 0; c < 8; ++c) x[i][c] = c0 + h + c < rows ? ld_cg(src + (c0 + h + c) * 128) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (p0 + i <= last)
#pragma unroll
                for (int c = 0; c < 8; ++c) f[h + c] += x[i][c];
          }
        }
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(f[c]);
        store_columns(a, v, out + static_cast<size_t>(c0) * a.ldc, kPair * w.pair + t, lrow, rows - c0);
      }
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
  return kMxMaxCtas * sizeof(int) + 2 * static_cast<size_t>(kMxMaxCtas) * kSlotFloats * sizeof(float);
}

cudaError_t mxfp4_gemm_launch(const uint8_t* rows, const uint8_t* w, int E, int N, int K, const int32_t* counts,
                              const int32_t* offsets, int capacity, bool gate_up, uint16_t* C, void* ws, int* status,
                              cudaStream_t st) {
  MxArgs a{};
  a.w = w, a.rows = rows, a.counts = counts, a.offsets = offsets;
  a.split_cnt = static_cast<int*>(ws);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kMxMaxCtas * sizeof(int));
  a.C = C, a.status = status;
  a.E = E, a.N = N, a.K = K, a.ldc = gate_up ? N / 2 : N, a.capacity = capacity;
  a.n_tiles = mx_tiles(N), a.gate_up = gate_up ? 1 : 0;
  a.rows_padded = mx_rows_padded(capacity);
  cudaError_t err = ensure_smem_limit<mxfp4_gemm_kernel>(kSmemBytes);
  if (err != cudaSuccess) return err;
  static int sms[64] = {0};
  int dev = 0;
  err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!sms[dev]) {
    err = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
  }
  return launch_kernel(mxfp4_gemm_kernel, dim3(sms[dev] < kMxMaxCtas ? sms[dev] : kMxMaxCtas), dim3(kThreads),
                       kSmemBytes, st, true, a);
}

}  // namespace chord
