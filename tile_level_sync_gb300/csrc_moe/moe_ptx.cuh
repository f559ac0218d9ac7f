// Inline PTX that the expert layer needs beside ptx.cuh (kept apart: the chain kernel's
// sources stay as its profiles know them).
#pragma once
#include "../csrc/ptx.cuh"

namespace cusync {
namespace ptx {

// True in one lane of a converged warp.  Code that a whole warp runs, with only the
// instruction itself under this predicate, keeps operands such as descriptors in uniform
// registers; in a branch of one lane each has to be moved there first.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// Four rows of a 2-D tensor map with a one-row box, given by index: row i lands box-width
// bytes after row i - 1.  Rows outside the tensor read as zero.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* m, uint64_t* bar, int32_t c0, int4 rows,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(rows.x), "r"(rows.y), "r"(rows.z),
      "r"(rows.w), "l"(policy)
      : "memory");
}

// A 5-D load whose completion is counted on the pair leader's mbarrier.
__device__ __forceinline__ void tma_load_5d_to_leader(void* dst, const CUtensorMap* m, uint32_t leader_bar, int32_t c0,
                                                      int32_t c1, int32_t c2, int32_t c3, int32_t c4,
                                                      uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(leader_bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "l"(policy)
      : "memory");
}

// 3-D TMA store of a shared-memory box; elements outside the tensor are not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns of TMEM.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Shared-memory matrix descriptor for an operand whose M (or N) index is contiguous, in the
// 128-byte-swizzle layout of TMA boxes of 64 such elements x some k rows: 64-element chunks
// `chunk` bytes apart (leading-dimension offset), groups of 8 k rows 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t saddr, uint32_t chunk) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(chunk >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// Bits of the instruction descriptor that make A or B contiguous along M or N instead of K.
constexpr uint32_t kIdescAMn = 1u << 15;
constexpr uint32_t kIdescBMn = 1u << 16;

}  // namespace ptx
}  // namespace cusync
