// MXFP4 (OCP Microscaling Formats v1.0): 32 consecutive values along K share
// one E8M0 scale 2^(code - 127); each value is an E2M1 number
// (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte, low nibble first.
//
// Operand layouts of the experts' product.  K is padded to units of 256 (128
// bytes of values, one row of the tensor core's 128-byte swizzle) with zeros.
//   weights  [256-byte header][expert][pair of tiles][unit][tile of the pair]
//            of kMxUnitBytes: 128 weight rows x 128 B, then the unit's scales
//            as two 512-byte blocks (128 of K each).  One bulk copy moves a
//            pair's unit.  The last pair of an odd number of tiles has one.
//            Gate/up weights: 32 rows of a tile hold 16 gate rows and the 16
//            up rows of the same indices, so one warp of the epilogue has both.
//   rows     [slab of 256 rows][unit][row] of 128 B, then the same of 8 scale
//            bytes, for mx_rows_padded(capacity) rows: a tile's rows of a unit
//            are one or two contiguous runs, and its units lie 32 KB apart
//            whatever the capacity (units a whole capacity apart missed the
//            TLB: 0.3 us more per unit at 71,632 rows).
// In both, the 16-byte chunk c of row r sits at chunk c ^ (r % 8) of its 128
// bytes (the 128-byte swizzle; tiles start at multiples of 8 rows), and a
// chunk is exactly one block of 32 values.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace chord {

constexpr int kMxBlock = 32;
constexpr int kMxUnitK = 256;
constexpr int kMxRowBytes = kMxUnitK / 2;                     // 128
constexpr int kMxRowScales = kMxUnitK / kMxBlock;             // 8
constexpr int kMxTileRows = 128;
constexpr int kMxTileBytes = kMxTileRows * kMxRowBytes;       // 16384
constexpr int kMxTileScaleBytes = kMxTileRows * kMxRowScales; // 1024
constexpr int kMxUnitBytes = kMxTileBytes + kMxTileScaleBytes;
// Largest grid of the product (one CTA per SM): sizes its split workspace.
constexpr int kMxMaxCtas = 160;
constexpr uint32_t kMxMagic = 0x4D344843u;                    // "CH4M"
constexpr uint32_t kMxVersion = 1u;

__host__ __device__ inline int mx_units(int K) { return (K + kMxUnitK - 1) / kMxUnitK; }
__host__ __device__ inline int mx_tiles(int N) { return (N + kMxTileRows - 1) / kMxTileRows; }
constexpr int kMxSlabRows = 256;
// A tile of rows starts at a multiple of 8 and is read in whole runs of 16.
__host__ __device__ inline size_t mx_rows_padded(size_t rows) {
  return (rows + 15 + kMxSlabRows - 1) / kMxSlabRows * kMxSlabRows;
}
// Place of row r's part of a unit, in rows of 128 B (values) or 8 B (scales).
__host__ __device__ inline size_t mx_row_place(int unit, int units, size_t r) {
  return (r / kMxSlabRows * units + unit) * kMxSlabRows + r % kMxSlabRows;
}

// Scale code of a block: floor(log2(amax)) - 2 (so that amax / scale lies in
// [4, 8)), at least 2^-127; 0xFF (NaN) when the block holds an infinity or a
// NaN, whose 32 values then all read as NaN.
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23);
  return e == 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
}
// 2^(127 - code): exact, and multiplying by it is exact wherever the result
// is not far below the smallest E2M1 midpoint.
__device__ __forceinline__ float mx_inverse_scale(uint32_t code) {
  return __uint_as_float(min(254u, 254u - code) << 23);
}
// Eight values as eight E2M1 codes (nearest, ties to even, at most 6).
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
__device__ __forceinline__ uint32_t e2m1x8_from_f16(const uint32_t (&h)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b0, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b1, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b2, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b3, %4;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return r;
}
// The inverse: eight codes as FP16 pairs (exact).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t q, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
}

}  // namespace chord
