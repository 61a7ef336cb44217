// Element types of the row operators: BF16, FP16 and FP32 values as FP32
// registers, and vectors of them as one aligned access.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "chord_moe.h"

namespace chord {

struct Bf16 {
  uint16_t v;
};
struct Fp16 {
  uint16_t v;
};

__device__ __forceinline__ float to_f32(Bf16 a) { return __uint_as_float(static_cast<uint32_t>(a.v) << 16); }
__device__ __forceinline__ float to_f32(Fp16 a) { return __half2float(__ushort_as_half(a.v)); }
__device__ __forceinline__ float to_f32(float a) { return a; }
// One rounding to nearest even (FP32: none).
__device__ __forceinline__ void from_f32(Bf16& d, float f) { d.v = __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
__device__ __forceinline__ void from_f32(Fp16& d, float f) { d.v = __half_as_ushort(__float2half_rn(f)); }
__device__ __forceinline__ void from_f32(float& d, float f) { d = f; }

// B bytes as one access (32: one 256-bit access), kept in program order: a
// programmatic launch reads nothing before its wait.
template <int B>
struct Chunk {
  static_assert(B == 2 || B == 4 || B == 8 || B == 16 || B == 32, "access size");
  uint32_t w[B < 4 ? 1 : B / 4];
};
template <int B>
__device__ __forceinline__ void load_chunk(const void* p, Chunk<B>& c) {
  if constexpr (B == 32) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3]), "=r"(c.w[4]), "=r"(c.w[5]), "=r"(c.w[6]),
                   "=r"(c.w[7])
                 : "l"(p)
                 : "memory");
  } else if constexpr (B == 16) {
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3])
                 : "l"(p)
                 : "memory");
  } else if constexpr (B == 8) {
    asm volatile("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(c.w[0]), "=r"(c.w[1]) : "l"(p) : "memory");
  } else if constexpr (B == 4) {
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(c.w[0]) : "l"(p) : "memory");
  } else {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
    c.w[0] = v;
  }
}
template <int B>
__device__ __forceinline__ void store_chunk(void* p, const Chunk<B>& c) {
  if constexpr (B == 32) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(c.w[0]), "r"(c.w[1]), "r"(c.w[2]),
                 "r"(c.w[3]), "r"(c.w[4]), "r"(c.w[5]), "r"(c.w[6]), "r"(c.w[7])
                 : "memory");
  } else if constexpr (B == 16) {
    *static_cast<uint4*>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
  } else if constexpr (B == 8) {
    *static_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
  } else if constexpr (B == 4) {
    *static_cast<uint32_t*>(p) = c.w[0];
  } else {
    *static_cast<uint16_t*>(p) = static_cast<uint16_t>(c.w[0]);
  }
}
// Element i of a chunk of T as FP32, and back.
template <typename T, int B>
__device__ __forceinline__ float chunk_f32(const Chunk<B>& c, int i) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(c.w[i]);
  } else {
    T t;
    t.v = static_cast<uint16_t>(c.w[i / 2] >> (16 * (i & 1)));
    return to_f32(t);
  }
}
template <typename T, int B>
__device__ __forceinline__ void f32_chunk(Chunk<B>& c, const float (&f)[B / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) c.w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      T t;
      from_f32(t, f[i]);
      c.w[i / 2] = i & 1 ? c.w[i / 2] | (static_cast<uint32_t>(t.v) << 16) : t.v;
    }
  }
}

inline size_t dtype_bytes(int dtype) {
  return dtype == CHORD_DTYPE_FP32 ? 4 : dtype == CHORD_DTYPE_BF16 || dtype == CHORD_DTYPE_FP16 ? 2 : 0;
}

// Largest power-of-two access (in bytes, at most `most`) to which every row of a
// [rows, H] matrix with the given row stride (in elements) is aligned and by
// which its row length divides.
inline int row_access_bytes(const void* p, long long stride, long long H, size_t elem, unsigned most = 16) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride * static_cast<long long>(elem)) |
                        static_cast<uintptr_t>(H * static_cast<long long>(elem)) | most;
  return static_cast<int>(all & (~all + 1));
}

}  // namespace chord
