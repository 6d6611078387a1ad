// tcgen05.cuh - the fifth generation's tensor instructions (inline PTX): tensor
// memory, CTA-wide products that one thread issues, and their descriptors.
#pragma once

#include <cstdint>

namespace cmdx {

// ---- tensor memory -----------------------------------------------------------
// 128 lanes of 512 32-bit columns; an address is lane << 16 | column. Warp w of
// a CTA reaches lanes 32 * (w % 4) and on.
__device__ __forceinline__ void tmem_alloc(uint32_t where, int columns) {  // (a whole warp)
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int columns) {  // (the same warp)
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
// 32 columns of this warp's lanes, one lane to a thread.
__device__ __forceinline__ void tmem_load(uint32_t (&r)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// (the registers that a load fills pass through the wait: nothing reads them before)
__device__ __forceinline__ void tmem_wait_load(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---- order between threads ------------------------------------------------------
__device__ __forceinline__ void tcgen05_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- products ---------------------------------------------------------------------
// Operands of 16-bit numbers in shared memory, in slabs of 64 of them (128
// bytes) to a row, 16-byte pieces swizzled over 8 rows (1024 bytes).
constexpr uint64_t kSwizzled128 = (uint64_t(1) << 46) | (uint64_t(2) << 61) | (uint64_t(1024 >> 4) << 32);
// rows along the product's rows or columns, 64 deep in K (a slab); steps of 16
// in K are 32 bytes apart
__device__ __forceinline__ uint64_t smem_along_k(uint32_t at) { return kSwizzled128 | (uint64_t(1) << 16) | ((at & 0x3ffff) >> 4); }
// rows along K, 64 columns to a slab, slabs `slab` bytes apart; steps of 16 in K
// are 2048 bytes apart
__device__ __forceinline__ uint64_t smem_across_k(uint32_t at, uint32_t slab) {
  return kSwizzled128 | (uint64_t(slab >> 4) << 16) | ((at & 0x3ffff) >> 4);
}
// Byte offset of 16-byte piece c of row r in a slab.
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// The instruction: 32-bit sums, 16-bit operands (both f16 or both bf16), M = 128
// rows, n columns (a multiple of 16), B along K or across it.
__device__ __forceinline__ uint32_t tcgen05_shape(bool bf16, int n, bool b_across) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_across ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// One lane of the warp (the same one each time).
__device__ __forceinline__ uint32_t elected() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
// d (+)= a * b, one step of 16 in K, issued by the elected lane. (A predicate,
// not a branch: all lanes work out the addresses, which stay in the warp's
// uniform registers, where the instruction takes them from. Issued from a branch
// of one lane, a product took 95 cycles, of any size.)
__device__ __forceinline__ void tcgen05_mma(uint32_t lane, uint32_t d, uint64_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add), "r"(lane)
      : "memory");
}
// ... with a in tensor memory (two 16-bit numbers to a column)
__device__ __forceinline__ void tcgen05_mma(uint32_t lane, uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(shape), "r"((uint32_t)add), "r"(lane)
      : "memory");
}
// An arrival on the mbarrier once everything that the elected lane has issued is done.
__device__ __forceinline__ void tcgen05_commit(uint32_t lane, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(lane)
      : "memory");
}

}  // namespace cmdx
