// Barriers in shared memory that asynchronous copies complete (mbarrier), and waits with a limit.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bsolve {

constexpr long long kPatience = 4000000000ll;  // clocks, about two seconds

__device__ __forceinline__ unsigned smem_address(const void* p) {
  return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void barrier_init(uint64_t* b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_address(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_address(b)) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint64_t* b, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_address(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool barrier_passed(uint64_t* b, unsigned parity) {
  unsigned done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done) : "r"(smem_address(b)), "r"(parity) : "memory");
  return done;
}
// False where the wait ran out, here or (`failed`) elsewhere in the block.
__device__ __forceinline__ bool wait_for(uint64_t* b, unsigned parity, volatile int* failed) {
  if (barrier_passed(b, parity)) return true;
  const long long start = clock64();
  while (!barrier_passed(b, parity)) {
    if (*failed) return false;
    if (clock64() - start > kPatience) {
      *failed = 1;
      return false;
    }
  }
  return true;
}

// A copy of whole 16-byte pieces, both addresses on 16 bytes, whose bytes the barrier counts.
__device__ __forceinline__ void copy_bytes(void* to, const void* from, int bytes, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_address(to)), "l"(from), "r"(bytes), "r"(smem_address(b)) : "memory");
}
// This thread arrives when its cp.async copies so far are there.
__device__ __forceinline__ void arrive_behind_copies(uint64_t* b) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_address(b)) : "memory");
}
// Barriers that were set up are seen by copies.
__device__ __forceinline__ void barriers_ready() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// Ordinary writes to shared memory come in front of copies that are asked for behind this (and a barrier).
__device__ __forceinline__ void writes_before_copies() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

}  // namespace bsolve
