// The experts' product in MXFP4 on the 5th-generation tensor cores:
//   C[r, n] = sum_k A[r, k] W[e(r), n, k]
// over rows in the aligned expert order, both operands E2M1 with E8M0 scales
// per 32 of K, FP32 accumulation, with an optional SiLU(gate) * up.
//
// Design on sm_103a (one persistent CTA per SM):
//   * the 128 weight rows of a tile are the MMA's M and an expert's rows its
//     N (a multiple of 16 up to kMaxTok), so one decoded token costs 16
//     columns, not 128 rows; one kernel serves decoding and prefill;
//   * the work is the list of (expert, weight tile, row tile) items times
//     their K units of 256, cut into one contiguous range per CTA of equal
//     length to within a unit.  Every SM streams the same number of bytes
//     whatever the number of items, and one token's few items spread over
//     all SMs.  An item that a range boundary cuts is summed by the CTA that
//     finishes last, from FP32 partials in workspace, in K order, so results
//     do not depend on timing;
//   * per unit one bulk copy brings 128 weight rows with their scales (17 KB,
//     contiguous, already swizzled), one the rows and one the rows' scales;
//   * the rows' scales arrive in row order; warp 2 rearranges them into the
//     block layout in shared memory; tcgen05.cp moves both operands' scales
//     to TMEM ahead of the MMAs of the unit, in order with them;
//   * two accumulators: the epilogue warps drain one while the MMAs of the
//     next item fill the other.
// TMEM: accumulators at columns 0 and kMaxTok, scales from column 480.
// Every mbarrier wait is bounded; on a timeout the CTA records
// CHORD_ERR_TIMEOUT, drains its own copies and MMAs, frees TMEM and exits.
#include "common.cuh"
#include "kernels.h"
#include "mxfp4.cuh"
#include "tc5.cuh"

namespace chord {
namespace {

constexpr int kMaxTok = 240;
constexpr int kStages = 4;
constexpr int kThreads = 256;
constexpr int kMaxExperts = 1024;
constexpr int kEpiWarp0 = 4;
// stage: weights | weight scales | rows | row scales as they arrive | row
// scales in block layout (two K halves of up to 256 rows)
constexpr int kAOff = 0, kSfaOff = kMxTileBytes, kBOff = kMxUnitBytes;
constexpr int kRawOff = kBOff + kMaxTok * kMxRowBytes;
constexpr int kSfbOff = kRawOff + kMaxTok * kMxRowScales;
constexpr int kSfbHalf = 1024;
constexpr int kStageBytes = (kSfbOff + 2 * kSfbHalf + 1023) / 1024 * 1024;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
constexpr int kSfCol = 480;      // SFA halves at +0, +4; SFB halves at +8, +16
constexpr int kTmemCols = 512;
static_assert(2 * kMaxTok <= kSfCol && kSfCol + 24 <= kTmemCols, "TMEM budget");
static_assert(kBOff % 1024 == 0 && kSfbOff % 128 == 0 && kMaxTok % 16 == 0 && kMaxTok <= 256, "stage layout");
static_assert(kSmemBytes + (3 * kMaxExperts + 1) * 4 + 1024 <= 232448, "shared memory budget");

struct MxArgs {
  const uint8_t* w;
  const uint8_t* rows;
  const int32_t* counts;
  const int32_t* offsets;
  int* split_cnt;        // [kMxMaxCtas], zero between launches
  float* partial;        // [2 * kMxMaxCtas][kMaxTok][128]
  uint16_t* C;
  int* status;
  int E, N, K, ldc, capacity, n_tiles, gate_up;
  size_t rows_padded;
};

struct Work {
  const int* prefix;     // shared: first item of each expert
  int E, n_tiles, units;
  long long begin, end, total;
};

struct Seg {
  int e, wt, row0, rows;   // item: expert, weight tile, first row, rows
  int u0, u1;              // its K units in this segment
};

// The segment that starts at work position `pos` (< w.end).
__device__ __forceinline__ Seg segment_at(const Work& w, const int* s_cnt, const int* s_off, long long pos) {
  const int item = static_cast<int>(pos / w.units);
  Seg s;
  s.u0 = static_cast<int>(pos - static_cast<long long>(item) * w.units);
  const long long rest = w.end - pos;
  s.u1 = rest < w.units - s.u0 ? s.u0 + static_cast<int>(rest) : w.units;
  int lo = 0, hi = w.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (w.prefix[mid] <= item) lo = mid; else hi = mid - 1;
  }
  s.e = lo;
  const int cnt = s_cnt[lo], local = item - w.prefix[lo];
  const int n_rt = (cnt + kMaxTok - 1) / kMaxTok;
  const int per = ((cnt + n_rt - 1) / n_rt + 15) & ~15;
  s.wt = local / n_rt;
  const int rt = local - s.wt * n_rt;
  s.row0 = s_off[lo] + rt * per;
  s.rows = min(per, cnt - rt * per);
  return s;
}

// Whether `ok` holds in all 128 threads of the epilogue warps.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

__global__ void __launch_bounds__(kThreads, 1) mxfp4_gemm_kernel(MxArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], sf_full[kStages], empty[kStages];
  __shared__ __align__(8) uint64_t tfull[2], tempty[2], done_bar;
  __shared__ uint32_t tmem_base_s;
  __shared__ int prefix[kMaxExperts + 1];
  __shared__ int s_cnt[kMaxExperts], s_off[kMaxExperts];
  __shared__ int warp_sum[kThreads / 32];
  __shared__ int hdr_ok, last_flag;
  __shared__ volatile int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (smem0 - smem_u32(smem_raw));

  if (tid == 0) {
    const uint32_t* h = reinterpret_cast<const uint32_t*>(a.w);
    hdr_ok = h[0] == kMxMagic && h[1] == kMxVersion && static_cast<int>(h[2]) >= a.E && static_cast<int>(h[3]) == a.N &&
             static_cast<int>(h[4]) == a.K && static_cast<int>(h[5]) == a.gate_up;
    if (!hdr_ok) set_status(a.status, CHORD_ERR_PREPACK_MISMATCH);
    abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&sf_full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(&done_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base_s, kTmemCols);

  // first item of each expert: thread i sums experts [i * per, (i + 1) * per)
  const int per = (a.E + kThreads - 1) / kThreads;
  int mine = 0;
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
    mine += a.n_tiles * ((cnt + kMaxTok - 1) / kMaxTok);
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) warp_sum[warp] = inc;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int run = inc - mine;
  for (int i = 0; i < warp; ++i) run += warp_sum[i];
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e >= a.E) break;
    prefix[e] = run;
    run += a.n_tiles * ((s_cnt[e] + kMaxTok - 1) / kMaxTok);
  }
  if (tid == kThreads - 1) prefix[a.E] = run;   // the last thread ends at the total
  __syncthreads();
  const uint32_t tmem_base = tmem_base_s;

  Work w;
  w.prefix = prefix;
  w.E = a.E;
  w.n_tiles = a.n_tiles;
  w.units = mx_units(a.K);
  w.total = hdr_ok ? static_cast<long long>(prefix[a.E]) * w.units : 0;
  // CTAs that take work: all, or as many as there are units (a range is
  // never empty, so the parts of a cut item are in consecutive CTAs)
  const long long G = w.total < gridDim.x ? w.total : gridDim.x;
  w.begin = blockIdx.x < G ? blockIdx.x * w.total / G : 0;
  w.end = blockIdx.x < G ? (blockIdx.x + 1) * w.total / G : 0;

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      const uint8_t* row_scales = a.rows + static_cast<size_t>(w.units) * a.rows_padded * kMxRowBytes;
      int it = 0;
      for (long long pos = w.begin; pos < w.end && !abort_flag;) {
        const Seg s = segment_at(w, s_cnt, s_off, pos);
        const int n16 = (s.rows + 15) & ~15;
        const uint8_t* wsrc = a.w + kPackHeaderBytes +
                              (static_cast<size_t>(s.e) * a.n_tiles + s.wt) * w.units * static_cast<size_t>(kMxUnitBytes);
        for (int u = s.u0; u < s.u1; ++u, ++it) {
          const int st = it % kStages;
          if (it >= kStages && !mbar_wait(&empty[st], ((it / kStages) - 1) & 1, a.status)) {
            abort_flag = 1;
            break;
          }
          uint8_t* dst = smem + st * kStageBytes;
          const size_t row = static_cast<size_t>(u) * a.rows_padded + s.row0;
          mbar_arrive_expect_tx(&full[st], kMxUnitBytes + n16 * (kMxRowBytes + kMxRowScales));
          bulk_g2s(dst + kAOff, wsrc + static_cast<size_t>(u) * kMxUnitBytes, kMxUnitBytes, &full[st]);
          bulk_g2s(dst + kBOff, a.rows + row * kMxRowBytes, n16 * kMxRowBytes, &full[st]);
          bulk_g2s(dst + kRawOff, row_scales + row * kMxRowScales, n16 * kMxRowScales, &full[st]);
        }
        pos += s.u1 - s.u0;
      }
      // every issued copy lands before the CTA can exit
      for (int j = max(0, it - kStages); j < it; ++j) mbar_wait(&full[j % kStages], (j / kStages) & 1, a.status);
    }
  } else if (warp == 2) {
    // --------------------------------------------------- row scales to blocks
    int it = 0;
    for (long long pos = w.begin; pos < w.end && !abort_flag;) {
      const Seg s = segment_at(w, s_cnt, s_off, pos);
      const int n16 = (s.rows + 15) & ~15;
      for (int u = s.u0; u < s.u1; ++u, ++it) {
        const int st = it % kStages;
        bool ok = mbar_wait(&full[st], (it / kStages) & 1, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          abort_flag = 1;
          break;
        }
        uint8_t* base = smem + st * kStageBytes;
        for (int r = lane; r < n16; r += 32) {
          const uint2 v = *reinterpret_cast<const uint2*>(base + kRawOff + r * kMxRowScales);
          uint8_t* dst = base + kSfbOff + (r / 128) * 512 + (r % 32) * 16 + (r / 32 % 4) * 4;
          *reinterpret_cast<uint32_t*>(dst) = v.x;
          *reinterpret_cast<uint32_t*>(dst + kSfbHalf) = v.y;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[st]);
      }
      pos += s.u1 - s.u0;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      int it = 0, j = 0;
      for (long long pos = w.begin; pos < w.end && !abort_flag; ++j) {
        const Seg s = segment_at(w, s_cnt, s_off, pos);
        const int n16 = (s.rows + 15) & ~15;
        const int acc = j & 1, use = j >> 1;
        if (use >= 1 && !mbar_wait(&tempty[acc], (use - 1) & 1, a.status)) {
          abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem_base + acc * kMaxTok;
        const uint32_t idesc[2] = {idesc_mxf4(n16, 0), idesc_mxf4(n16, 2)};
        for (int u = s.u0; u < s.u1; ++u, ++it) {
          const int st = it % kStages;
          if (!mbar_wait2(&full[st], (it / kStages) & 1, &sf_full[st], (it / kStages) & 1, a.status)) {
            abort_flag = 1;
            break;
          }
          tc_fence_after();
          const uint32_t base = smem0 + st * kStageBytes;
          const uint32_t sf = tmem_base + kSfCol;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tc_cp_scales(sf + 4 * h, scales_desc(base + kSfaOff + 512 * h));
            tc_cp_scales(sf + 8 + 8 * h, scales_desc(base + kSfbOff + kSfbHalf * h));
            if (n16 > 128) tc_cp_scales(sf + 12 + 8 * h, scales_desc(base + kSfbOff + kSfbHalf * h + 512));
          }
          const uint64_t ad = sw128_kmajor_desc(base + kAOff), bd = sw128_kmajor_desc(base + kBOff);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_mxf4(d, ad + 2 * kk, bd + 2 * kk, idesc[kk & 1], sf + 4 * (kk >> 1), sf + 8 + 8 * (kk >> 1),
                        u > s.u0 || kk ? 1u : 0u);
          tc_commit(&empty[st]);
        }
        if (abort_flag) break;
        tc_commit(&tfull[acc]);
        pos += s.u1 - s.u0;
      }
      // all issued MMAs complete before TMEM can be freed
      if (it > 0) {
        tc_commit(&done_bar);
        mbar_wait(&done_bar, 0, a.status);
      }
    }
  } else if (warp >= kEpiWarp0) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3, lrow = 32 * q + lane;   // TMEM lane quarter; weight row of the tile
    int j = 0;
    for (long long pos = w.begin; pos < w.end; ++j) {
      const Seg s = segment_at(w, s_cnt, s_off, pos);
      const int acc = j & 1, use = j >> 1;
      // the four warps go on or stop together: barriers follow
      if (!epilogue_all(mbar_wait(&tfull[acc], use & 1, a.status))) {
        abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem_base + acc * kMaxTok + (static_cast<uint32_t>(32 * q) << 16);
      const bool whole = s.u0 == 0 && s.u1 == w.units;
      int c_first = 0, c_last = 0;   // the CTAs that hold parts of a cut item
      bool finish = whole;
      if (!whole) {
        const long long i0 = pos - s.u0, i1 = i0 + w.units - 1;
        c_first = static_cast<int>(((i0 + 1) * G - 1) / w.total);
        c_last = static_cast<int>(((i1 + 1) * G - 1) / w.total);
        float* dst = a.partial + static_cast<size_t>(2 * blockIdx.x + (s.u0 == 0)) * kMaxTok * 128 + lrow;
        for (int c0 = 0; c0 < s.rows; c0 += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c0, v);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < s.rows) dst[(c0 + c) * 128] = __uint_as_float(v[c]);
        }
        __threadfence();
        epilogue_all(true);
        if (tid == 32 * kEpiWarp0) {
          const int last = atomicAdd(a.split_cnt + c_first, 1) == c_last - c_first;
          if (last) atomicExch(a.split_cnt + c_first, 0);   // zero for the next launch
          last_flag = last;
        }
        epilogue_all(true);
        finish = last_flag != 0;
        __threadfence();
      }
      if (finish) {
        for (int c0 = 0; c0 < s.rows; c0 += 32) {
          uint32_t v[32];
          if (whole) {
            tmem_ld_32x32b_x32(taddr + c0, v);
            tmem_ld_wait();
          } else {
            float f[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) f[c] = 0.f;
            for (int p = c_first; p <= c_last; ++p) {
              const float* src =
                  a.partial + static_cast<size_t>(2 * p + (p == c_first)) * kMaxTok * 128 + lrow;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c0 + c < s.rows) f[c] += ld_cg(src + (c0 + c) * 128);
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(f[c]);
          }
          uint16_t* out = a.C + static_cast<size_t>(s.row0 + c0) * a.ldc;
          if (a.gate_up) {
            // lanes 0-15 hold gate rows, 16-31 the up rows of the same
            // indices: of two columns, the low lanes finish the first and
            // the high lanes the second
            const int col = (kMxTileRows / 2) * s.wt + 16 * q + (lane & 15);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const bool up = lane & 16;
              const float other = __uint_as_float(__shfl_xor_sync(0xffffffffu, up ? v[c] : v[c + 1], 16));
              const float g = up ? other : __uint_as_float(v[c]);
              const float h = __fdividef(g, 1.0f + __expf(-g)) * (up ? __uint_as_float(v[c + 1]) : other);
              const int cc = c + (up ? 1 : 0);
              if (c0 + cc < s.rows && col < a.ldc) out[static_cast<size_t>(cc) * a.ldc + col] = f32_to_bf16_rn(h);
            }
          } else {
            const int col = kMxTileRows * s.wt + lrow;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c0 + c < s.rows && col < a.ldc)
                out[static_cast<size_t>(c) * a.ldc + col] = f32_to_bf16_rn(__uint_as_float(v[c]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      pos += s.u1 - s.u0;
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
  return kMxMaxCtas * sizeof(int) + 2 * static_cast<size_t>(kMxMaxCtas) * kMaxTok * 128 * sizeof(float);
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
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  mxfp4_gemm_kernel<<<sms < kMxMaxCtas ? sms : kMxMaxCtas, kThreads, kSmemBytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace chord
