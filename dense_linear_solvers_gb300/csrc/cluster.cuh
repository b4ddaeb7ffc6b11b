// Thread-block clusters of the recurrence kernels (bs_grec calls): rank, barrier, stores into a peer's
// shared memory, and the launch.
#pragma once

#include <cmath>
#include <cstdint>
#include <mutex>
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
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
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

inline cudaLaunchConfig_t cluster_config(cudaLaunchAttribute* attr, dim3 grid, int threads, int shared,
                                  int cluster, cudaStream_t stream) {
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = shared;
  config.stream = stream;
  config.attrs = attr;
  config.numAttrs = 1;
  return config;
}

// How many clusters of 1, 2, 4, 8 blocks of a kernel the current device holds at once.
struct Held {
  int clusters[kMaxCluster + 1];
};

// The answers for one kernel, asked of the driver at its first launch on a device (a few us each); an
// error is handed on and asked again by the next launch.
class HeldClusters {
 public:
  template <typename... P>
  cudaError_t of(void (*kernel)(P...), int threads, int shared, Held* held) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    // a device's own limit: raised before every launch, as by the other launchers
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
    if (e != cudaSuccess) return e;
    const std::lock_guard<std::mutex> lock(mutex_);
    const bool kept = device < kDevices;
    if (kept && known_[device]) {
      *held = held_[device];
      return cudaSuccess;
    }
    Held h{};
    for (int n = 1; n <= kMaxCluster; n *= 2) {
      cudaLaunchAttribute attr{};
      const cudaLaunchConfig_t config = cluster_config(&attr, dim3(n), threads, shared, n, nullptr);
      e = cudaOccupancyMaxActiveClusters(&h.clusters[n], kernel, &config);
      if (e != cudaSuccess) return e;
    }
    if (kept) {
      held_[device] = h;
      known_[device] = true;
    }
    *held = h;
    return cudaSuccess;
  }

 private:
  static constexpr int kDevices = 64;  // beyond: asked every time
  std::mutex mutex_;
  bool known_[kDevices] = {};
  Held held_[kDevices] = {};
};

// Above so many pairs of a sequence and a channel tile, a block takes each alone.
constexpr int64_t kManyUnits = 8192;

// Blocks of a cluster (a power of two: others are placed badly, 3 and 5 to 7 blocks took 10 to 40%
// longer) that share one sequence and channel tile, of which `tiles` * `batch` are at hand with
// `length` rows each, on average where they are packed; a block takes `rows` of them in a step.
// Equal sequences run in waves of what the GPU holds, and a wave costs its steps and about two more
// to fill and drain. Uneven ones fill each other's gaps, but the longest, about 1 + ln(batch)
// times the average where they were cut at random, cannot take less than its own steps (8 x 1,500
// rows on average, 2,048 channels BF16: 56 us with the 4 blocks that this gives, 77 with one).
// The least such cost, the smaller cluster where two are alike.
inline int grec_cluster(const Held& held, int64_t tiles, int64_t batch, int64_t length,
                        bool packed, int rows) {
  const double units = static_cast<double>(tiles) * static_cast<double>(batch);
  if (units > kManyUnits) return 1;
  const double longest =
      static_cast<double>(length) * (packed ? 1.0 + std::log(static_cast<double>(batch)) : 1.0);
  int best = 1;
  double least = 0;
  for (int n = 1; n <= kMaxCluster; n *= 2) {
    if (held.clusters[n] < 1 || (n > 1 && longest <= static_cast<double>(n / 2 * rows))) break;
    double waves = units / held.clusters[n], cost;
    if (packed) {
      cost = std::fmax(waves * (length / (static_cast<double>(n) * rows) + 2),
                       longest / (static_cast<double>(n) * rows) + 2);
    } else {
      cost = std::ceil(waves) * (std::ceil(length / (static_cast<double>(n) * rows)) + 2);
    }
    if (n == 1 || cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, int threads, int shared, int cluster,
                            cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr{};
  const cudaLaunchConfig_t config = cluster_config(&attr, grid, threads, shared, cluster, stream);
  return cudaLaunchKernelEx(&config, kernel, static_cast<P>(args)...);
}

}  // namespace bsolve
