// tcgen05.cuh -- fifth-generation tensor core forms for sm_103a: tensor memory, matrix products of binary16
// tiles with binary32 sums, and their completion on an mbarrier.
//
// Tiles in shared memory are stored in atoms of 64 elements (128 bytes) a row, eight rows (1024 bytes) to a
// swizzle group, the 16-byte chunks of row r exchanged by XOR with r % 8. The same bytes serve as a K-major
// operand (rows are M or N, the 64 elements are K) and as an MN-major one (rows are K).
#pragma once

#include <cstdint>

#include "pipeline.cuh"

namespace nvfp4 {

constexpr uint32_t kTmemColumns = 512;

// Whether a phase is complete; if not, the thread may sleep for some microseconds before it says so. A wait is given up
// after kNapLimit naps: half a second (a nap takes 4 us, measured), and 1.3 s at most (what a warp waits for takes the
// others some ten microseconds).
constexpr uint32_t kNap = 10000;  // ns
constexpr uint32_t kNapLimit = 1u << 17;
__device__ __forceinline__ bool mbar_wait_nap(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "n"(kNap)
      : "memory");
  return ok != 0;
}

// The registers of a warpgroup's threads from here on (all of its warps call it): fewer, or more, which waits until
// others have given theirs up.
template <int N, bool MORE>
__device__ __forceinline__ void set_registers() {
  if (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// All 32 lanes of one warp; the address goes to shared memory. Waits while another CTA of the SM holds columns.
__device__ __forceinline__ void tmem_alloc(uint32_t* address) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(address)),
               "n"(kTmemColumns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t address) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(address), "n"(kTmemColumns));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Ordinary stores to shared memory become visible to the tensor cores.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The low word of a shared-memory operand in 128-byte swizzle atoms. `mn_stride`: bytes between atoms of 64 along M
// or N (of an MN-major operand; a K-major one does not use it). An address further on by n bytes adds n / 16.
__device__ __forceinline__ uint32_t smem_operand(uint32_t address, uint32_t mn_stride) {
  return (address & 0x3FFFFu) >> 4 | (mn_stride >> 4) << 16;
}
// The high word: eight rows are 1024 bytes apart.
constexpr uint32_t kOperandHigh = 1024 >> 4 | 1u << 14 | 2u << 29;

// Instruction descriptor: binary16 operands, binary32 sums, 128 x N; b_mn: B is MN-major.
__device__ __forceinline__ uint32_t mma_shape(uint32_t n, bool b_mn) {
  return 1u << 4 | (b_mn ? 1u << 16 : 0u) | (n >> 3) << 17 | (128u >> 4) << 24;
}

// True in one lane of the warp. Products are issued in code that the whole warp runs, and by that lane alone: so their
// operands are computed in uniform registers, where the instruction takes them.
__device__ __forceinline__ uint32_t elected() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one;
}
// The same value in all lanes, and known to be.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xFFFFFFFFu, v); }

// D (tensor memory) = A B + (sum ? D : 0) over 16 elements of K, by the lane where `leader` is set.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t shape, uint32_t sum) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\tmov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b),
      "r"(shape), "r"(sum), "n"(kOperandHigh), "r"(leader) : "memory");
}
// The same with A in tensor memory (two binary16 elements to a column).
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t shape, uint32_t sum) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(shape), "r"(sum),
      "n"(kOperandHigh), "r"(leader) : "memory");
}
// An arrival on `bar` when every product that the leader has issued is done.
__device__ __forceinline__ void mma_commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)), "r"(leader) : "memory");
}

// 32 or 16 columns of this warp's 32 lanes, a column to a register. Loads are asynchronous: the registers hold the
// values after tmem_wait, and tmem_loaded after it keeps uses of them from going ahead of it.
#define NVFP4_R8(v, i) "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3]), "=f"(v[i + 4]), "=f"(v[i + 5]), "=f"(v[i + 6]), "=f"(v[i + 7])
#define NVFP4_RW8(v, i) "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]), "+f"(v[i + 6]), "+f"(v[i + 7])
#define NVFP4_IN8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
#define NVFP4_INF8(v, i) "f"(v[i]), "f"(v[i + 1]), "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]), "f"(v[i + 6]), "f"(v[i + 7])
__device__ __forceinline__ void tmem_load(float (&v)[32], uint32_t address) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : NVFP4_R8(v, 0), NVFP4_R8(v, 8), NVFP4_R8(v, 16), NVFP4_R8(v, 24) : "r"(address));
}
__device__ __forceinline__ void tmem_load(float (&v)[16], uint32_t address) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : NVFP4_R8(v, 0), NVFP4_R8(v, 8) : "r"(address));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_loaded(float (&v)[32]) {
  asm volatile("" : NVFP4_RW8(v, 0), NVFP4_RW8(v, 8), NVFP4_RW8(v, 16), NVFP4_RW8(v, 24));
}
__device__ __forceinline__ void tmem_loaded(float (&v)[16]) { asm volatile("" : NVFP4_RW8(v, 0), NVFP4_RW8(v, 8)); }
__device__ __forceinline__ void tmem_store(uint32_t address, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::
          NVFP4_IN8(v, 0), NVFP4_IN8(v, 8), "r"(address) : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t address, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::
          NVFP4_INF8(v, 0), NVFP4_INF8(v, 8), "r"(address) : "memory");
}
__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#undef NVFP4_R8
#undef NVFP4_RW8
#undef NVFP4_IN8
#undef NVFP4_INF8

}  // namespace nvfp4
