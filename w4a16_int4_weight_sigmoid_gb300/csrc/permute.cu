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
// weight gradient: FP32 in a tree fixed by the call's sizes), each result
// rounded once; no atomics, so a call repeats bit for bit.
// Measured: permute of 8192 tokens x 7168 BF16 to 48 of 384 experts 39.3 us
// (239 MB with the zeroed padding: 6.1 TB/s), its weighted sum's gradient
// 56 us (312 MB: 5.6 TB/s), of 6.7 TB/s that a copy reaches; 20 tokens at
// block 128, 99 % padding, 34 us (7.1 TB/s); weighted sum of 128 FP32 tokens
// 5.2 us; 64 tokens permuted 2.4 us, bound by the launch and two dependent
// loads.
//
// Rows are moved in accesses of B bytes: 32 where every base, row stride and
// row length allows it, otherwise the largest power of two they share, down
// to one element (permute: 32 or 16, or shifted).  All kernels are programmatic launches that touch no memory
// before the work ahead of them in the stream has completed.
#include <algorithm>
#include <type_traits>

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

constexpr int kThreads = 128, kWarps = kThreads / 32;
// CTAs per SM that permute is compiled for, and its grid in such waves: 8192
// rows of 7168 took 48.3 us with one wave, 45.7 with two, 43.6 with four (the
// CTAs' shares even out) and 49.2 with a CTA for every token.
constexpr int kCtas = 12, kWaves = 4;

// ------------------------------------------------------------ padding rows
// Zeros in the padding rows (sorted >= M * topk) of the aligned order: CTA b
// of nb takes every nb-th run of rows below the padded total, all threads on
// one row (a warp on a row of its own took 25 us at 64 tokens).  A run is
// kPadBytes long, one to eight rows (eight rows of 7168 BF16 values each: one
// token permuted at block 16 3.2 us against 1.9, 8192 at block 128 43.0
// against 39.3).
constexpr int kPadBytes = 8192;
__host__ __device__ constexpr int pad_run(int row_bytes) {
  return row_bytes > kPadBytes ? 1 : row_bytes < kPadBytes / 8 ? 8 : kPadBytes / row_bytes;
}

// Zeros at any element alignment, by all threads: 16-byte stores between a
// first and a last part of up to 14 bytes (2-byte stores throughout took 20 us
// for 5000 rows of 3323 BF16 values).
__device__ __forceinline__ void zero_bytes(uint8_t* dst, int bytes) {
  const int head = min(static_cast<int>(-reinterpret_cast<uintptr_t>(dst) & 15u), bytes);
  const int body = (bytes - head) / 16, tail = bytes - head - 16 * body;
  const int i = threadIdx.x;
  if (i < head / 2) reinterpret_cast<uint16_t*>(dst)[i] = 0;
  for (int c = i; c < body; c += kThreads) reinterpret_cast<uint4*>(dst + head)[c] = make_uint4(0, 0, 0, 0);
  if (i < tail / 2) reinterpret_cast<uint16_t*>(dst + head + 16 * body)[i] = 0;
}

__device__ __forceinline__ void zero_padding(const RowArgs& a, int row_bytes, long long out_stride, int b, int nb) {
  const int lane = threadIdx.x & 31, sentinel = a.M * a.topk;
  // neighbouring rows without a gap are one stretch (of kPadBytes at
  // most, or one row)
  const bool dense = out_stride == row_bytes;
  const int run = pad_run(row_bytes);
  // A run's entries are read ahead, before the total is known and while the run
  // before is written: entries past the total exist, and are dropped.  (32 rows
  // of many runs in one load took 0-20 % longer with much padding.)
  auto entry = [&](int r) { return lane < run && r < a.rows ? ld_ca(a.sorted + r) : 0; };
  int f = entry(b * run + lane);
  const int total = min(ld_ca(a.ntpp), a.rows);
  for (int r0 = b * run; r0 < total; r0 += nb * run) {
    uint32_t pad = __ballot_sync(0xffffffffu, lane < run && r0 + lane < total && f >= sentinel);
    f = entry(r0 + nb * run + lane);
    while (pad) {
      const int first = __ffs(pad) - 1, n = dense ? __ffs(~(pad >> first)) - 1 : 1;
      zero_bytes(static_cast<uint8_t*>(a.out) + (r0 + first) * out_stride, n * row_bytes);
      pad &= ~(((1u << n) - 1u) << first);
    }
  }
}

// ----------------------------------------------------------------- permute
// Copies, so element types do not matter.  A thread moves one access of a
// token's row to each of its rows; 2^wpt_log2 warps (1, 2 or 4) of a CTA
// share a token, so that short rows do not leave warps idle.  CTAs walk over the
// tokens, the next one's row and the positions of the one after it in flight.
// The CTAs of the last `pad_y` grid rows zero the padding.
template <int B>
__global__ void __launch_bounds__(kThreads, kCtas) permute_kernel(RowArgs a, int row_bytes, long long x_stride,
                                                                  long long out_stride, int pad_y, int wpt_log2) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, token_ctas = gridDim.y - pad_y;
  if (static_cast<int>(blockIdx.y) >= token_ctas) {
    zero_padding(a, row_bytes, out_stride, (blockIdx.y - token_ctas) * gridDim.x + blockIdx.x,
                    pad_y * gridDim.x);
    return;
  }
  const int tokens = kWarps >> wpt_log2, step = token_ctas * tokens;   // tokens per CTA, and at once
  const int t_first = blockIdx.y * tokens + (warp >> wpt_log2);
  const int c = (((blockIdx.x << wpt_log2) + (warp & ((1 << wpt_log2) - 1))) * 32 + lane) * B;
  const bool in = c < row_bytes;
  auto position = [&](int t) {
    const int p = t < a.M && lane < a.topk ? ld_ca(a.pos + static_cast<long long>(t) * a.topk + lane) : -1;
    return p < a.rows ? p : -1;
  };
  auto load = [&](int p, Chunk<B>& v, int t) {
    const uint32_t left = __ballot_sync(0xffffffffu, p >= 0);
    if (left && in) load_chunk<B>(static_cast<const uint8_t*>(a.x) + t * x_stride + c, v);
    return left;
  };
  auto store = [&](int p, uint32_t left, const Chunk<B>& v) {
    for (; left; left &= left - 1) {
      const long long row = __shfl_sync(0xffffffffu, p, __ffs(left) - 1);
      if (in) store_chunk<B>(static_cast<uint8_t*>(a.out) + row * out_stride + c, v);
    }
  };
  Chunk<B> v0, v1;
  int p0 = position(t_first), p1 = position(t_first + step);
  uint32_t left0 = load(p0, v0, t_first);
  for (int t = t_first; t < a.M; t += 2 * step) {
    const int p2 = position(t + 2 * step), p3 = position(t + 3 * step);
    const uint32_t left1 = load(p1, v1, t + step);
    store(p0, left0, v0);
    left0 = load(p2, v0, t + 2 * step);
    store(p1, left1, v1);
    p0 = p2;
    p1 = p3;
  }
}

// The same for rows that are not all aligned to 16 bytes.  A warp has up to
// kShiftBytes of a token's row: it stages them in shared memory at the offset
// that the source has from a 16-byte boundary, and writes each destination
// with 16-byte stores at that row's own offset, each put together from two
// staged chunks.  What lies before the first and after the last boundary goes
// element by element, so that no access leaves the row.  4000 rows of 3323
// BF16 values to two experts each took 35.6 us in accesses of 2 bytes, of 3324
// in accesses of 8 bytes 18.6 us; here 17.7 and 17.5, and rows of 3328, which
// are aligned, 14.2 above.
constexpr int kShiftBytes = 2048, kShiftCtas = 12;
__global__ void __launch_bounds__(kThreads, kShiftCtas) permute_shift_kernel(RowArgs a, int row_bytes,
                                                                             long long x_stride, long long out_stride,
                                                                             int pad_y, int wpt_log2) {
  // one chunk of room for the offset and one that is read past the end
  __shared__ __align__(16) uint8_t s_rows[kWarps][kShiftBytes + 32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, token_ctas = gridDim.y - pad_y;
  if (static_cast<int>(blockIdx.y) >= token_ctas) {
    zero_padding(a, row_bytes, out_stride, (blockIdx.y - token_ctas) * gridDim.x + blockIdx.x, pad_y * gridDim.x);
    return;
  }
  uint8_t* stage = s_rows[warp];
  const int tokens = kWarps >> wpt_log2, step = token_ctas * tokens;
  const int c = ((blockIdx.x << wpt_log2) + (warp & ((1 << wpt_log2) - 1))) * kShiftBytes;
  const int bytes = min(kShiftBytes, row_bytes - c);
  if (bytes <= 0) return;
  for (int t = blockIdx.y * tokens + (warp >> wpt_log2); t < a.M; t += step) {
    int p = lane < a.topk ? ld_ca(a.pos + static_cast<long long>(t) * a.topk + lane) : -1;
    if (p >= a.rows) p = -1;
    const uint8_t* src = static_cast<const uint8_t*>(a.x) + t * x_stride + c;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15u);
    {
      const int head = min((16 - off) & 15, bytes), body = (bytes - head) / 16, tail = bytes - head - 16 * body;
      Chunk<16> v[kShiftBytes / 512];
      Chunk<2> h, e;
#pragma unroll
      for (int i = 0; i < kShiftBytes / 512; ++i)
        if (lane + 32 * i < body) load_chunk<16>(src + head + 16 * (lane + 32 * i), v[i]);
      if (lane < head / 2) load_chunk<2>(src + 2 * lane, h);
      if (lane < tail / 2) load_chunk<2>(src + head + 16 * body + 2 * lane, e);
      __syncwarp();   // the last token's chunks are read
#pragma unroll
      for (int i = 0; i < kShiftBytes / 512; ++i)
        if (lane + 32 * i < body) store_chunk<16>(stage + off + head + 16 * (lane + 32 * i), v[i]);
      if (lane < head / 2) store_chunk<2>(stage + off + 2 * lane, h);
      if (lane < tail / 2) store_chunk<2>(stage + off + head + 16 * body + 2 * lane, e);
      __syncwarp();
    }
    for (uint32_t left = __ballot_sync(0xffffffffu, p >= 0); left; left &= left - 1) {
      const long long row = __shfl_sync(0xffffffffu, p, __ffs(left) - 1);
      uint8_t* dst = static_cast<uint8_t*>(a.out) + row * out_stride + c;
      const int head = min(static_cast<int>(-reinterpret_cast<uintptr_t>(dst) & 15u), bytes);
      const int body = (bytes - head) / 16, tail = bytes - head - 16 * body;
      // destination chunk i starts `words` words and `bits` bits into staged
      // chunk i + first
      const int first = (off + head) / 16, words = (off + head) / 4 & 3, bits = (off + head & 3) * 8;
#pragma unroll
      for (int i = 0; i < kShiftBytes / 512; ++i) {
        const int k = lane + 32 * i;
        if (k >= body) break;
        const uint4 lo = *reinterpret_cast<const uint4*>(stage + 16 * (first + k));
        const uint4 hi = *reinterpret_cast<const uint4*>(stage + 16 * (first + k + 1));
        uint32_t u[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z}, last = hi.w;
        if (words & 2) {
          u[0] = u[2], u[1] = u[3], u[2] = u[4], u[3] = u[5], u[4] = u[6], u[5] = last;
        }
        if (words & 1) {
          u[0] = u[1], u[1] = u[2], u[2] = u[3], u[3] = u[4], u[4] = u[5];
        }
        Chunk<16> o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o.w[q] = __funnelshift_r(u[q], u[q + 1], bits);
        store_chunk<16>(dst + head + 16 * k, o);
      }
      const uint8_t* s = stage + off;
      if (lane < head / 2) reinterpret_cast<uint16_t*>(dst)[lane] = reinterpret_cast<const uint16_t*>(s)[lane];
      if (lane < tail / 2) {
        const int q = head + 16 * body + 2 * lane;
        *reinterpret_cast<uint16_t*>(dst + q) = *reinterpret_cast<const uint16_t*>(s + q);
      }
    }
  }
}

// ---------------------------------------------------- weighted sum of rows
// Warp (t, chunk): VPT accesses per lane of the token's local rows, kRows of
// them in flight, added in increasing j.  A CTA's warps have four tokens (a
// CTA per token took 12.0 us for 6521 rows of 272 values).  Chunks lie along the
// grid's y, which ends at 65535, and its z.
template <typename T, int B, int VPT, int kRows, bool kWeighted>
__global__ void __launch_bounds__(kThreads) combine_kernel(RowArgs a) {
  constexpr int V = B / sizeof(T);
  const int lane = threadIdx.x & 31, t = blockIdx.x * kWarps + threadIdx.x / 32;
  grid_dep_wait();
  grid_dep_launch();
  if (t >= a.M) return;
  int p = -1;
  float w = 1.f;
  if (lane < a.topk) {
    const long long o = static_cast<long long>(t) * a.topk + lane;
    p = ld_ca(a.pos + o);
    if (kWeighted) w = ld_ca(a.w + o);
  }
  uint32_t left = __ballot_sync(0xffffffffu, p >= 0 && p < a.rows);
  const int nv = a.H / V, c0 = (blockIdx.z * gridDim.y + blockIdx.y) * 32 * VPT + lane;
  float acc[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) acc[i][e] = 0.f;
  while (left) {
    Chunk<B> v[kRows][VPT];
    float wj[kRows];
    const uint32_t batch = left;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (!left) break;
      const int j = __ffs(left) - 1;
      left &= left - 1;
      const T* src = static_cast<const T*>(a.y) + __shfl_sync(0xffffffffu, p, j) * a.ldy;
      wj[r] = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (c0 + 32 * i < nv) load_chunk<B>(src + V * (c0 + 32 * i), v[r][i]);
    }
    const int n = __popc(batch ^ left);
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r < n)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (c0 + 32 * i < nv)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float y = chunk_f32<T, B>(v[r][i], e);
              acc[i][e] = kWeighted ? fmaf(wj[r], y, acc[i][e]) : acc[i][e] + y;
            }
  }
  T* dst = static_cast<T*>(a.out) + t * a.ldo;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (c0 + 32 * i < nv) {
      Chunk<B> o;
      f32_chunk<T, B>(o, acc[i]);
      store_chunk<B>(dst + V * (c0 + 32 * i), o);
    }
}

// ------------------------------------------------- gradient of the weighted sum
// A group of kGroup threads (a CTA, or for short rows a warp) per (t, s) after
// the padding CTAs: assignments j = s, s + S, ... of token t (S = gridDim.y).
// One pass over dout[t] and y[p] gives both dy[p] and the dot product; dout[t]
// comes from L1 for every j after the first.
template <typename T, int B, int kGroup>
__global__ void __launch_bounds__(kThreads) unpermute_backward_kernel(RowArgs a, int pad_x) {
  // accesses in flight: with short ones more (4000 odd rows of 3323 BF16 values
  // 39.7 us with four, 33.4 with eight; 16 cost short rows up to a third)
  constexpr int V = B / sizeof(T), kUnroll = B >= 32 ? 2 : B >= 8 ? 4 : 8;
  __shared__ float s_part[kGroup == 32 ? 1 : kMaxTopk][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x % kGroup;
  grid_dep_wait();
  grid_dep_launch();
  if (static_cast<int>(blockIdx.x) < pad_x) {
    zero_padding(a, a.H * static_cast<int>(sizeof(T)), a.ldo * static_cast<long long>(sizeof(T)),
                 blockIdx.x * gridDim.y + blockIdx.y, pad_x * gridDim.y);
    return;
  }
  const int t = (blockIdx.x - pad_x) * (kThreads / kGroup) + (kGroup == 32 ? warp : 0), nv = a.H / V;
  if (kGroup == 32 && t >= a.M) return;
  const T* g = static_cast<const T*>(a.x) + t * a.ldx;
  // lane j holds assignment j: the rows of all are known after one load
  const long long f = static_cast<long long>(t) * a.topk + lane;
  const bool mine = lane < a.topk && lane % gridDim.y == blockIdx.y;
  const int p = mine ? ld_ca(a.pos + f) : -1;
  const float w = mine ? ld_ca(a.w + f) : 0.f;
  float dw = 0.f;   // lane j's weight gradient (a warp per token), 0 where not local
  const uint32_t local = __ballot_sync(0xffffffffu, p >= 0 && p < a.rows);
  for (uint32_t left = local; left; left &= left - 1) {
    const int j = __ffs(left) - 1;
    const long long row = __shfl_sync(0xffffffffu, p, j);
    const float wj = __shfl_sync(0xffffffffu, w, j);
    const T* y = static_cast<const T*>(a.y) + row * a.ldy;
    T* dy = static_cast<T*>(a.out) + row * a.ldo;
    float dot = 0.f;
    for (int c0 = tid; c0 < nv; c0 += kUnroll * kGroup) {
      Chunk<B> vg[kUnroll], vy[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
        if (c0 + i * kGroup < nv) {
          load_chunk<B>(g + V * (c0 + i * kGroup), vg[i]);
          load_chunk<B>(y + V * (c0 + i * kGroup), vy[i]);
        }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i)
        if (c0 + i * kGroup < nv) {
          float d[V];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float gv = chunk_f32<T, B>(vg[i], e);
            dot = fmaf(gv, chunk_f32<T, B>(vy[i], e), dot);
            d[e] = wj * gv;
          }
          Chunk<B> o;
          f32_chunk<T, B>(o, d);
          store_chunk<B>(dy + V * (c0 + i * kGroup), o);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (kGroup == 32) {
      if (lane == j) dw = dot;
    } else if (lane == 0) {
      s_part[j][warp] = dot;
    }
  }
  if (kGroup != 32) {
    __syncthreads();
    if (warp) return;
    if (local >> lane & 1) {
#pragma unroll
      for (int i = 0; i < kWarps; ++i) dw += s_part[lane][i];
    }
  }
  if (mine) a.dw[f] = dw;
}

// CTAs that cover `rows` rows of the order for their padding: one for each
// run, and for each 4 KB at most (most of an order's capacity is past its
// padded total).
int padding_ctas(int rows, int row_bytes) {
  const int run = pad_run(row_bytes);
  return static_cast<int>(std::min<long long>((rows + run - 1) / run, static_cast<long long>(rows) * row_bytes / 4096 + 1));
}

// warp_bytes: what one warp has of a row at a time.
template <typename Kernel>
cudaError_t launch_permute(Kernel kernel, int warp_bytes, int ctas, const RowArgs& a, int elem, cudaStream_t st) {
  const int row_bytes = a.H * elem;
  const int warps = (row_bytes + warp_bytes - 1) / warp_bytes, wpt = warps >= 3 ? 4 : warps;
  const int columns = (warps + wpt - 1) / wpt;
  // CTAs for tokens: kWaves of what is resident; for padding a fifth more, or
  // what few tokens leave over
  const int slots = std::max(1, std::min(kWaves * ctas * sm_count() / columns, 60000));
  const int tokens = std::min((a.M + kWarps / wpt - 1) / (kWarps / wpt), slots);
  const int pads = padding_ctas(a.rows, row_bytes);
  const int pad_y = std::max(1, std::min(std::max(slots / 5, slots - tokens), (pads + columns - 1) / columns));
  return launch_kernel(kernel, dim3(columns, tokens + pad_y), dim3(kThreads), 0, st, true, a, row_bytes, a.ldx * elem,
                       a.ldo * elem, pad_y, wpt / 2);
}

template <typename T, int B>
cudaError_t launch_combine(const RowArgs& a, cudaStream_t st) {
  const int nv = a.H / (B / static_cast<int>(sizeof(T))), ctas = (a.M + kWarps - 1) / kWarps;
  // accesses per lane: many, where there are at least four CTAs per SM then;
  // eight rows in flight with few, four with many
  constexpr int kFew = B >= 16 ? 1 : 4, kMany = 2 * kFew;
  const int many = (nv + 32 * kMany - 1) / (32 * kMany), few = (nv + 32 * kFew - 1) / (32 * kFew);
  auto grid = [&](int chunks) {
    const int z = (chunks + 65534) / 65535;
    return dim3(ctas, (chunks + z - 1) / z, z);
  };
  if (static_cast<long long>(ctas) * many >= 4LL * sm_count())
    return launch_kernel(a.w ? combine_kernel<T, B, kMany, 4, true> : combine_kernel<T, B, kMany, 4, false>,
                         grid(many), dim3(kThreads), 0, st, true, a);
  return launch_kernel(a.w ? combine_kernel<T, B, kFew, 8, true> : combine_kernel<T, B, kFew, 8, false>,
                       grid(few), dim3(kThreads), 0, st, true, a);
}

template <typename T, int B>
cudaError_t launch_unpermute_backward(const RowArgs& a, cudaStream_t st) {
  int split = 1;
  while (split < a.topk && static_cast<long long>(a.M) * split < 4LL * sm_count()) split *= 2;
  split = std::min(split, a.topk);
  const int pads = std::min(padding_ctas(a.rows, a.H * static_cast<int>(sizeof(T))), 8 * sm_count());
  const int pad_x = (pads + split - 1) / split;
  // a warp per token where its lanes pass over the row at most four times and
  // the tokens fill the SMs (3296 rows of 117 values: 8.0 us with a CTA each)
  const int nv = a.H / (B / static_cast<int>(sizeof(T)));
  if (nv <= 128 && a.M >= 16 * sm_count())
    return launch_kernel(unpermute_backward_kernel<T, B, 32>, dim3((a.M + kWarps - 1) / kWarps + pad_x, split),
                         dim3(kThreads), 0, st, true, a, pad_x);
  return launch_kernel(unpermute_backward_kernel<T, B, kThreads>, dim3(a.M + pad_x, split), dim3(kThreads), 0, st, true,
                       a, pad_x);
}

// Access size shared by all row matrices of the call.
int access_bytes(const RowArgs& a, size_t es) {
  int bytes = row_access_bytes(a.out, a.ldo, a.H, es, 32);
  if (a.x) bytes = std::min(bytes, row_access_bytes(a.x, a.ldx, a.H, es, 32));
  if (a.y) bytes = std::min(bytes, row_access_bytes(a.y, a.ldy, a.H, es, 32));
  return bytes;
}

// Calls f(element type, access size); access sizes below the element's do
// not occur (bases and strides are element-aligned).
template <typename F>
cudaError_t with_access(int dtype, int bytes, F f) {
  auto typed = [&](auto t) {
    using T = decltype(t);
    switch (bytes) {
      case 32: return f(t, std::integral_constant<int, 32>{});
      case 16: return f(t, std::integral_constant<int, 16>{});
      case 8: return f(t, std::integral_constant<int, 8>{});
      case 4: return f(t, std::integral_constant<int, 4>{});
      default: return f(t, std::integral_constant<int, static_cast<int>(sizeof(T))>{});
    }
  };
  if (dtype == CHORD_DTYPE_BF16) return typed(Bf16{});
  if (dtype == CHORD_DTYPE_FP16) return typed(Fp16{});
  return typed(0.f);
}

}  // namespace

cudaError_t moe_permute_launch(const void* x, int dtype, long long ldx, const int32_t* pos, const int32_t* sorted,
                               const int32_t* ntpp, int M, int topk, int H, int rows, void* out, long long ldo,
                               cudaStream_t st) {
  RowArgs a{};
  a.x = x, a.ldx = ldx, a.pos = pos, a.sorted = sorted, a.ntpp = ntpp, a.out = out, a.ldo = ldo;
  a.M = M, a.topk = topk, a.H = H, a.rows = rows;
  const int es = static_cast<int>(dtype_bytes(dtype));
  const int bytes = access_bytes(a, es);
  if (bytes == 32) return launch_permute(permute_kernel<32>, 32 * 32, kCtas, a, es, st);
  if (bytes == 16) return launch_permute(permute_kernel<16>, 32 * 16, kCtas, a, es, st);
  return launch_permute(permute_shift_kernel, kShiftBytes, kShiftCtas, a, es, st);
}

cudaError_t moe_combine_launch(const void* y, int dtype, long long ldy, const float* w, const int32_t* pos, int M,
                               int topk, int H, int rows, void* out, long long ldo, cudaStream_t st) {
  RowArgs a{};
  a.y = y, a.ldy = ldy, a.w = w, a.pos = pos, a.out = out, a.ldo = ldo;
  a.M = M, a.topk = topk, a.H = H, a.rows = rows;
  return with_access(dtype, access_bytes(a, dtype_bytes(dtype)), [&](auto t, auto b) {
    return launch_combine<decltype(t), decltype(b)::value>(a, st);
  });
}

cudaError_t moe_unpermute_backward_launch(const void* dout, const void* y, int dtype, long long ldd, long long ldy,
                                          const float* w, const int32_t* pos, const int32_t* sorted,
                                          const int32_t* ntpp, int M, int topk, int H, int rows, void* dy,
                                          long long ldo, float* dw, cudaStream_t st) {
  RowArgs a{};
  a.x = dout, a.ldx = ldd, a.y = y, a.ldy = ldy, a.w = w, a.pos = pos, a.sorted = sorted, a.ntpp = ntpp;
  a.out = dy, a.ldo = ldo, a.dw = dw, a.M = M, a.topk = topk, a.H = H, a.rows = rows;
  return with_access(dtype, access_bytes(a, dtype_bytes(dtype)), [&](auto t, auto b) {
    return launch_unpermute_backward<decltype(t), decltype(b)::value>(a, st);
  });
}

}  // namespace chord
