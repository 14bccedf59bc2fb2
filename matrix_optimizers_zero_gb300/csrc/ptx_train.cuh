// PTX wrappers of the training-step operators (sm_103a), beside those of
// ptx.cuh: 4-bit block-scaled tensor-core products and a few others. Written from the PTX ISA descriptions.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace mo {
namespace ptx {

// Instruction descriptor of kind::mxf4 / kind::mxf4nvf4 (e2m1 operands, both
// K-major, fp32 accumulator).
//   bits 4-5 B scale id, 7-9 A format (1 = e2m1), 10-12 B format, 17-22 N >> 3,
//   bit 23 scale type (0 = e4m3, 1 = e8m0), bits 27-28 M >> 7, 29-30 A scale id
// The scale id is the first byte, of the four in each 32-bit scale column,
// that the instruction uses (0 or 2; always 0 with four scales a row).
__host__ __device__ constexpr uint32_t idesc_fp4(uint32_t M, uint32_t N, bool e8m0, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((e8m0 ? 1u : 0u) << 23) | ((M >> 7) << 27) |
         (sf_id << 29);
}

// Shared-memory descriptor of a 512-byte scale tile (32 rows of 16 bytes, no
// swizzle): 8-row groups of 128 bytes, one after the other.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
  return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(128u >> 4) << 32) | (uint64_t(1) << 46);
}

// Copies a 512-byte scale tile from shared memory to four TMEM columns,
// repeated in the four lane quarters.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D (+)= (A sA)(B sB)^T over K = 64. kMx: a scale for 32 elements (e8m0),
// otherwise for 16 (e4m3). The accumulator, and the A scales, are those of
// each CTA's own rows; each CTA holds the B scales of all N columns. The
// descriptors share their upper halves (desc_hi): one thread issues these, and
// every instruction it spends on an operand delays the tensor core.
template <bool kPair, bool kMx>
__device__ __forceinline__ void umma_fp4(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t desc_hi, uint32_t idesc,
                                         uint32_t sfa_tmem, uint32_t sfb_tmem, bool accumulate) {
#define MO_UMMA_FP4(GROUP, KIND, VEC)                                                                    \
  asm volatile(                                                                                          \
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"                              \
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"                                                 \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VEC                      \
      " [%0], a, b, %4, [%6], [%7], p;\n\t}" ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(desc_hi), "r"(idesc), \
      "r"(accumulate ? 1u : 0u), "r"(sfa_tmem), "r"(sfb_tmem)                                            \
      : "memory")
  if (kPair && kMx) MO_UMMA_FP4("2", "mxf4", "2X");
  if (kPair && !kMx) MO_UMMA_FP4("2", "mxf4nvf4", "4X");
  if (!kPair && kMx) MO_UMMA_FP4("1", "mxf4", "2X");
  if (!kPair && !kMx) MO_UMMA_FP4("1", "mxf4nvf4", "4X");
#undef MO_UMMA_FP4
}

// Upper half of the descriptor of a K-major operand of 128-byte rows
// (smem_desc_sw128 with 1024 bytes between 8-row groups); the lower half is
// the address / 16 with the unused leading dimension (1) above it.
constexpr uint32_t kDescHiSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo_sw128(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Adds to a counter in global memory, releasing the block's earlier writes
// (after a block barrier) and acquiring those of the blocks that added before.
__device__ __forceinline__ uint32_t atomic_add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t r;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(r) : "l"(p), "r"(v) : "memory");
  return r;
}

// Arrives on an mbarrier of any CTA of the cluster without releasing memory:
// hands over accesses to TMEM, which tcgen05.wait and
// tcgen05.fence::before_thread_sync have ordered.
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Whether the phase with the given parity has completed, without waiting; its
// arrives may be another CTA's.
__device__ __forceinline__ bool mbar_peek_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}

// ---------------------------------------------------------------- one CTA by itself
__device__ __forceinline__ void tmem_alloc_one(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_one() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_one(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void umma_commit_one(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// TMA load into this CTA's shared memory, completion on its own mbarrier.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Each lane of the warp writes n consecutive 32-bit columns of its TMEM lane.
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float4 ld_shared_cluster_v4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// 16 bytes from global to shared memory, asynchronously; wait for all of the
// thread's copies.
__device__ __forceinline__ void cp_async16(uint32_t saddr, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(saddr), "l"(g) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---------------------------------------------------------------- conversions
// Eight fp32 values to e2m1 (to nearest, ties to even, saturating at 6), the
// first in the lowest four bits.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

}  // namespace ptx
}  // namespace mo
