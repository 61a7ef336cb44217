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

// V consecutive elements, one access of V * sizeof(T) bytes (at most 16).
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

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
