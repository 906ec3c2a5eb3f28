// tcgen05.cuh -- operands and tensor memory of the kernels on the 5th-generation
// tensor cores, with the 128-byte swizzle.
#pragma once

#include <stdint.h>

#include "device_util.cuh"

namespace qtts {

// Operands in shared memory: rows of 64 16-bit values (128 bytes), rows one after the
// other, 64-wide blocks of columns one after the other, and in a row the 16-byte
// words exchanged by the row's low bits (the tensor cores' 128-byte swizzle), so
// that neither a row's words nor a word of neighbouring rows share banks.
__device__ __forceinline__ int word_at(int row, int word) { return row * 128 + ((word ^ (row & 7)) << 4); }
__device__ __forceinline__ uint64_t swizzled_desc(const void* p) {
  return (uint64_t)((smem_addr(p) >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// Waits, with a limit, until every product that this warp's elected lane has issued has
// run: before the tensor memory is given back, whichever other wait ran out its own limit.
// `bar`: initialised for one arrival, of no other use; whole warp.
__device__ __forceinline__ void drain_products(uint64_t* bar, int tries) {
  if (elect_one()) tc_commit(bar);
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < tries; ++i)
    if (mbar_test_sleep(bar, 0, 10000)) break;
  __syncwarp();
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// the same, for the registers of a load that was asked for earlier: their use stays behind it
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

}  // namespace qtts
