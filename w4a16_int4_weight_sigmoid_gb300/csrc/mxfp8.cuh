// MXFP8 (E4M3 values, 32 of a row share an E8M0 scale) in registers: a block of
// 32 is held by 32 / kN lanes of a warp, kN consecutive values each.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "elem.cuh"

namespace chord {

constexpr int kMx8Block = 32;

// The largest magnitude of a block as FP32 bits (ordered like the magnitudes,
// infinity and NaN above all of them), from each lane's values; all lanes of
// the warp take part.
template <typename T, int B>
__device__ __forceinline__ uint32_t block_top(const Chunk<B>& c) {
  constexpr int kN = B / sizeof(T);
  uint32_t top = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < kN; ++i) top = max(top, c.w[i] & 0x7fffffffu);
  } else if constexpr (kN == 1) {
    top = c.w[0] & 0x7fffu;
  } else {
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) top = __vmaxu2(top, c.w[i] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
  }
#pragma unroll
  for (int o = 1; o < kMx8Block / kN; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if constexpr (sizeof(T) == 4) {
    return top;
  } else {
    T t;
    t.v = static_cast<uint16_t>(top);
    return __float_as_uint(to_f32(t)) & 0x7fffffffu;
  }
}
// Its scale: the smallest power of two from 2^-127 on with which no magnitude
// passes 448 = 1.75 * 2^8, as the byte s of 2^(s - 127); 255 where the block
// holds an infinity or a NaN.
__device__ __forceinline__ uint32_t block_scale(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  const int s = static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
  return s > 0 ? s : 0;
}
__device__ __forceinline__ float scale_value(uint32_t s) {
  return s == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(s ? s << 23 : 0x400000u);
}
// 2^(127 - s) for scales of finite blocks (255: some value).
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// kN codes as bytes of words, from values over the scale.
template <int kN>
__device__ __forceinline__ void to_codes(const float (&v)[kN], uint32_t s, uint32_t (&code)[kN < 4 ? 1 : kN / 4]) {
  const float inv = inverse_scale(s);
  float q[kN];
#pragma unroll
  for (int i = 0; i < kN; i += 2) {                 // at most 448
    const float2 two = mul2(make_float2(v[i], i + 1 < kN ? v[i + 1] : 0.f), make_float2(inv, inv));
    q[i] = two.x;
    if (i + 1 < kN) q[i + 1] = two.y;
  }
  if (s >= 247) {   // 256 times 2^120, the scale of values from 2^127 on, is past FP32; infinities and NaN
#pragma unroll
    for (int i = 0; i < kN; ++i) q[i] = s == 255 ? 0.f : fminf(fmaxf(q[i], -240.f), 240.f);
  }
  auto pair = [](float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return static_cast<uint32_t>(r);
  };
  if constexpr (kN == 1) {
    code[0] = pair(q[0], 0.f) & 0xffu;
  } else if constexpr (kN == 2) {
    code[0] = pair(q[0], q[1]);
  } else {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) code[i] = pair(q[4 * i], q[4 * i + 1]) | pair(q[4 * i + 2], q[4 * i + 3]) << 16;
  }
}
// The values that kN codes stand for.
template <int kN>
__device__ __forceinline__ void from_codes(const uint32_t (&code)[kN < 4 ? 1 : kN / 4], float scale, float (&v)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; i += 2) {
    const uint16_t two = static_cast<uint16_t>(code[i / 4] >> (8 * (i & 3)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const __half2 x = *reinterpret_cast<const __half2*>(&h);
    const float2 f = mul2(__half22float2(x), make_float2(scale, scale));
    v[i] = f.x;
    if (i + 1 < kN) v[i + 1] = f.y;
  }
}
template <int kN>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&code)[kN < 4 ? 1 : kN / 4]) {
  if constexpr (kN == 1) {
    uint16_t v;
    asm volatile("{\n\t.reg .u32 t;\n\tld.global.u8 t, [%1];\n\tcvt.u16.u32 %0, t;\n\t}" : "=h"(v) : "l"(p) : "memory");
    code[0] = v;
  } else {
    Chunk<kN> c;
    load_chunk<kN>(p, c);
#pragma unroll
    for (int i = 0; i < (kN < 4 ? 1 : kN / 4); ++i) code[i] = c.w[i];
  }
}
template <int kN>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&code)[kN < 4 ? 1 : kN / 4]) {
  if constexpr (kN == 1) {
    *p = static_cast<uint8_t>(code[0]);
  } else {
    Chunk<kN> c;
#pragma unroll
    for (int i = 0; i < (kN < 4 ? 1 : kN / 4); ++i) c.w[i] = code[i];
    store_chunk<kN>(p, c);
  }
}
__device__ __forceinline__ uint32_t load_scale(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// How a CTA of kRowThreads threads shares rows: `lanes` threads (a power of
// two, whole warps) to a row, each with up to `unroll` of its chunks in flight.
// Enough threads that a row takes one turn where there are few rows (the
// capacity of an order is several times the rows of one rank), four otherwise.
constexpr int kRowThreads = 256;
inline int row_lanes(long long rows, int chunks, int unroll) {
  const int turns = rows < 16384 ? 1 : 4;
  int lanes = 32;
  while (lanes < kRowThreads && lanes * unroll * turns < chunks) lanes *= 2;
  return lanes;
}

}  // namespace chord
