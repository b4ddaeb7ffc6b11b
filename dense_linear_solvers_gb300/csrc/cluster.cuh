// Thread-block clusters of the recurrence kernels (bs_grec calls): rank, barrier, stores into a peer's
// shared memory, and the launch.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "row_types.cuh"

namespace bsolve {

constexpr int kMaxCluster = 8;   // the portable limit

__device__ __forceinline__ int cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_size() {
  unsigned n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return static_cast<int>(n);
}
// Every thread of every block of the cluster arrives. The barrier itself orders no memory on
// arrival: a warp that has stored to its peers publishes that with cluster_publish() first, so
// that the others need not wait for their own stores to global memory.
__device__ __forceinline__ void cluster_publish() {
  asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// Stores 16 bytes at `at` (an address in this block's shared memory) in block `rank`'s.
template <typename V>
__device__ __forceinline__ void store_remote(V* at, int rank, const V& v) {
  static_assert(sizeof(V) == 16, "16 bytes");
  const float4 f = *reinterpret_cast<const float4*>(&v);
  const unsigned local = static_cast<unsigned>(__cvta_generic_to_shared(at));
  unsigned remote;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(remote), "f"(f.x),
               "f"(f.y), "f"(f.z), "f"(f.w)
               : "memory");
}

__device__ __forceinline__ unsigned low_bits(const void* p) {
  return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p));
}

// Stores two neighbouring elements, as one value where `pairs` says that they are aligned.
// WHOLE: both are there and aligned.
template <typename T, bool WHOLE>
__device__ __forceinline__ void store_pair(T* at, float2 v, bool pairs, bool first, bool second) {
  const typename Pair<T>::type q = pair_from_f32<T>(v);
  if (WHOLE || (pairs && second)) {
    *reinterpret_cast<typename Pair<T>::type*>(at) = q;
  } else {
    if (first) at[0] = q.x;
    if (second) at[1] = q.y;
  }
}
template <typename T>
__device__ __forceinline__ T* row_at(T* base, int row, unsigned pitch) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(base) + row * static_cast<uint64_t>(pitch));
}

// Whether every row of an operand starts on a 16-byte boundary, or on one of two elements.
template <typename T>
bool rows_aligned(const T* p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * sizeof(T))) & 15) == 0;
}
template <typename T>
bool pair_stores(const T* p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * sizeof(T))) &
          (2 * sizeof(T) - 1)) == 0;
}

// Blocks of a cluster that share one sequence and channel tile: `units` such pairs are at hand, of
// `length` rows each (packed sequences: on average), `rows` rows a block at a time. As many as
// the GPU's 152 SMs hold at once, two blocks each, and no more than the sequence has pieces
// for: a second wave of few blocks costs more than idle slots.
inline int grec_cluster(int64_t units, int64_t length, int rows) {
  int n = 1;
  while (n < kMaxCluster && units * 2 * n <= 2 * 152 && length > static_cast<int64_t>(n) * rows)
    n *= 2;
  return n;
}

template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, int threads, int shared, int cluster,
                            cudaStream_t stream, A... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = shared;
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, static_cast<P>(args)...);
}

}  // namespace bsolve
