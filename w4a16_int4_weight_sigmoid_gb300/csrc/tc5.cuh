// Blackwell tensor-core (tcgen05 / TMEM) and TMA tensor-copy wrappers, inline PTX.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "common.cuh"

namespace chord {

// --------------------------------------------------------------- TMEM
// Allocate `ncols` (power of two >= 32) TMEM columns; the base address is
// written to *dst (shared memory).  Executed by one whole warp.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Generic-proxy shared-memory writes -> visible to the async proxy (tensor core, TMA).
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, BF16 inputs, FP32 accumulate, one CTA.
__device__ __forceinline__ void tc_mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc]^T, BF16, FP32 accumulate, one CTA.  A (M=128)
// sits in TMEM lanes 0-127 (lane = row), column c holding the BF16 pair
// (k = 2c low half, 2c + 1 high half), 8 columns per K=16 step.
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One K = 256 unit of a block-scaled MXFP4 product (E2M1 operands, an E8M0
// scale per 32 of K), issued by one elected lane of a converged warp in one
// block: an instruction of its own election took about 60 cycles to issue,
// longer than its MMA ran.  M = 128 rows of A times N columns of B.
//   a, b      SW128 K-major descriptors (a K = 64 step is 32 bytes on)
//   fa, fb    scales_desc of A's two 512-byte scale blocks (128 of K each)
//             and of B's (kHalf bytes apart; 512 more for N > 128)
//   sfa, sfb  TMEM columns for them: 4 per block of A, 8 per block of B
// tcgen05.cp copies 512 bytes (32 rows of 16 B) to four columns, the 32 lanes
// repeated in all four lane quarters: byte k of column c, lane i is scale k
// of row 32 c + i.  It executes in order with the MMAs of the same thread.
#define CHORD_MXF4_MMA(dst, a, b, id, sa, sb, acc) \
  "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [" dst "], " a ", " b ", " id ", [" sa "], [" sb "], " acc ";\n\t"
#define CHORD_CP_SCALES(dst, src) "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [" dst "], " src ";\n\t"
__device__ __forceinline__ void tc_mxf4_unit_elect(uint32_t d, uint64_t a, uint64_t b, uint64_t fa, uint32_t sfa,
                                                   uint32_t sfb, uint32_t idesc0, uint32_t idesc2,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, q;\n\t.reg .b32 r, sa, sb;\n\t.reg .b64 f, a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %8, 0;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t"
      "add.s32 sa, %4, 4;\n\tadd.s32 sb, %5, 8;\n\tadd.s64 f, %3, 32;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      CHORD_CP_SCALES("%4", "%3")
      CHORD_CP_SCALES("sa", "f")
      CHORD_MXF4_MMA("%0", "%1", "%2", "%6", "%4", "%5", "p")
      CHORD_MXF4_MMA("%0", "a1", "b1", "%7", "%4", "%5", "q")
      CHORD_MXF4_MMA("%0", "a2", "b2", "%6", "sa", "sb", "q")
      CHORD_MXF4_MMA("%0", "a3", "b3", "%7", "sa", "sb", "q")
      "}" ::"r"(d), "l"(a), "l"(b), "l"(fa), "r"(sfa), "r"(sfb), "r"(idesc0), "r"(idesc2), "r"(accumulate)
      : "memory");
}
// B's scales of a unit: two blocks, four when N > 128.
template <int kHalf>
__device__ __forceinline__ void tc_mxf4_scales_elect(uint64_t fb, uint32_t sfb, bool wide) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t.reg .b32 r, s1, s2, s3;\n\t.reg .b64 f1, f2, f3;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "add.s32 s1, %1, 8;\n\tadd.s32 s2, %1, 4;\n\tadd.s32 s3, %1, 12;\n\t"
      "add.s64 f1, %0, %3;\n\tadd.s64 f2, %0, 32;\n\tadd.s64 f3, f1, 32;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      CHORD_CP_SCALES("%1", "%0")
      CHORD_CP_SCALES("s1", "f1")
      "and.pred e, e, p;\n\t"
      CHORD_CP_SCALES("s2", "f2")
      CHORD_CP_SCALES("s3", "f3")
      "}" ::"l"(fb), "r"(sfb), "r"(wide ? 1u : 0u), "n"(kHalf >> 4)
      : "memory");
}
#undef CHORD_MXF4_MMA
#undef CHORD_CP_SCALES
__device__ __forceinline__ void tc_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// Arrive on `bar` once every tcgen05.mma issued so far by this thread completes.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void tc_commit2_elect(uint64_t* bar0, uint64_t* bar1) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(smem_u32(bar0)),
      "r"(smem_u32(bar1))
      : "memory");
}
// 16 lanes x 32 columns -> 16 registers per thread: with g = lane / 4 and
// t = lane % 4, registers {4i, 4i+1} are (lane g, columns 8i + 2t, 8i + 2t + 1)
// and {4i+2, 4i+3} the same columns of lane g + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// 32 lanes x 32 consecutive columns of 32-bit TMEM cells -> 32 registers per thread.
__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// 16 lanes x 32 columns from 16 registers per thread, in the m16n8k16 A
// fragment order: registers {4i, 4i+1, 4i+2, 4i+3} of the thread with
// g = lane / 4, t = lane % 4 land at (lane g, column 8i + t), (lane g + 8,
// column 8i + t), (lane g, column 8i + 4 + t) and (lane g + 8, column
// 8i + 4 + t) -- one K=16 step of a 16-row slab per i (mapping measured on
// sm_103a by storing tagged values and reading them back with 32x32b).
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------- UMMA descriptors
// Shared-memory matrix descriptor, K-major, 128-byte swizzle: rows of 128 B
// (64 BF16 along K), 8-row groups 1024 B apart, tile base 1024-B aligned.
// Fields: start address >> 4 [0,14), leading byte offset >> 4 [16,30) (unused
// for swizzled K-major; 1), stride byte offset >> 4 [32,46), descriptor
// version 1 [46,48), layout SWIZZLE_128B = 2 [61,64).
__device__ __forceinline__ uint64_t sw128_kmajor_desc(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// Instruction descriptor, kind::f16: D FP32 [4,6)=1, A BF16 [7,10)=1, B BF16
// [10,13)=1, both K-major (bits 15, 16 = 0), N>>3 at [17,23), M>>4 at [24,29).
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor of a scale block for tcgen05.cp: no swizzle, rows of 16 B,
// 8-row groups 128 B apart.
__device__ __forceinline__ uint64_t scales_desc(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128u >> 4) << 32) |
         (static_cast<uint64_t>(1u) << 46);
}
// Instruction descriptor, kind::mxf4: A and B E2M1 (1 at [7,10) and [10,12)),
// both K-major, N>>3 at [17,23), scales E8M0 (bit 23), M>>7 at [27,29); the
// byte pair of a TMEM cell that holds this K = 64 step's scales (0 or 2) at
// [4,6) for B and [29,31) for A; dense K = 64 (bit 31 zero).
__host__ __device__ constexpr uint32_t idesc_mxf4(int N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (1u << 27) |
         (sf_id << 29);
}

// ------------------------------------------------------------ TMA tensor
// 2-D tiled TMA load (coordinates: inner element, row) into shared memory,
// completing on `bar`.  The inner coordinate is a multiple of 64 here
// (128-byte aligned), rows need no alignment; out-of-range rows read zeros.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int c0, int c1,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

}  // namespace chord
