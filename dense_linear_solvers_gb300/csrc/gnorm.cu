// The sums over rows of the norms' backward pass (bs_gnorm_backward_batched of bsolve.h).
#include "gnorm_shapes.cuh"
#include "kernels.h"

namespace bsolve {
namespace {

// The three sums over rows: 32 columns a block, each of its 16 warps every sixteenth part in
// order, then the warps' sums in order.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(32 * kSumWarps)
gnorm_sums_kernel(int width, int parts, const float* __restrict__ partial, float* dw_post,
                  float* dscale, float* dw_pre) {
  __shared__ float sums[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dscale : dw_pre;
  if (out == nullptr) return;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int k = warp; k < parts; k += kSumWarps)
      sum += partial[(static_cast<int64_t>(k) * 3 + blockIdx.y) * width + c];
  }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= width) return;
  sum = 0.f;
  for (int w = 0; w < kSumWarps; ++w) sum += sums[w][lane];
  out[c] = sum;
}

}  // namespace

cudaError_t launch_gnorm_sums(int width, int parts, const float* partial, float* dw_post,
                              float* dscale, float* dw_pre, cudaStream_t stream) {
  gnorm_sums_kernel<<<dim3((width + 31) / 32, 3), 32 * kSumWarps, 0, stream>>>(
      width, parts, partial, dw_post, dscale, dw_pre);
  return cudaGetLastError();
}

size_t gnorm_backward_workspace(int width, int64_t rows) {
  // the larger of the two element sizes' needs
  const int a = backward_blocks(width, 2, rows), b = backward_blocks(width, 4, rows);
  return static_cast<size_t>(a > b ? a : b) * 3 * width * sizeof(float);
}

}  // namespace bsolve
