// The order in which packed sequences are taken (bs_grec calls).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bsolve {

// A few packed sequences are taken longest first, since what starts last ends last (60 prompts of 670
// rows on average, 1,024 channels BF16: 99 to 74 us): the number of the n-th longest, the same for
// a whole block. All threads take part; `scratch` holds kSortedBatch + 1 numbers.
constexpr int kSortedBatch = 128;

static __device__ __noinline__ int nth_longest(const int64_t* offsets, int batch, int n,
                                        int64_t* scratch) {
  const int t = threadIdx.x;
  if (t < batch) scratch[t] = offsets[t + 1] - offsets[t];
  __syncthreads();
  if (t < batch) {
    const int64_t mine = scratch[t];
    int rank = 0;
    for (int j = 0; j < batch; ++j) rank += scratch[j] > mine || (scratch[j] == mine && j < t);
    if (rank == n) scratch[kSortedBatch] = t;
  }
  __syncthreads();
  const int chosen = static_cast<int>(scratch[kSortedBatch]);
  __syncthreads();  // the scratch is free again
  return chosen;
}

}  // namespace bsolve
