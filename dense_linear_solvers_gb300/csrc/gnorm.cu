// The norms around a block with its gate and residual scale (bs_gnorm calls of bsolve.h).
//
// One block per row: three passes over the row, one for each mean and one for the outputs.
#include "gnorm_math.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {
namespace {

constexpr int kThreads = 256;
constexpr int kGradBlocks = 304;

// The sum of v over the block, the same bits in every thread. `red` holds 32 floats.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  v = 0.f;
  for (int k = 0; k < warps; ++k) v += red[k];
  return v;
}

template <typename T>
__device__ __forceinline__ float new_residual(const GnormRows<T>& p, int64_t row, int c, float r1) {
  float t = to_f32(p.f[row * p.ldf + c]);
  if (p.w_post) t = t * r1 * p.w_post[c];
  if (p.z) t *= gate_of(to_f32(p.z[row * p.ldz + c]), p.gate).act;
  if (p.scale) t *= p.scale[c];
  return p.x ? to_f32(p.x[row * p.ldx + c]) + t : t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
gnorm_kernel(GnormRows<T> p, T* __restrict__ y, int64_t ldy, T* __restrict__ u, int64_t ldu) {
  __shared__ float red[32];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float r1 = 1.f, r2 = 1.f;
    if (p.w_post) {
      float sum = 0.f;
      for (int c = threadIdx.x; c < p.width; c += blockDim.x) {
        const float v = to_f32(p.f[row * p.ldf + c]);
        sum = fmaf(v, v, sum);
      }
      r1 = 1.f / sqrtf(block_sum(sum, red) / p.width + p.eps);
    }
    if (u) {
      float sum = 0.f;
      for (int c = threadIdx.x; c < p.width; c += blockDim.x) {
        const float v = new_residual(p, row, c, r1);
        sum = fmaf(v, v, sum);
      }
      r2 = 1.f / sqrtf(block_sum(sum, red) / p.width + p.eps);
    }
    for (int c = threadIdx.x; c < p.width; c += blockDim.x) {
      const float v = new_residual(p, row, c, r1);
      if (y) y[row * ldy + c] = from_f32<T>(v);
      if (u) u[row * ldu + c] = from_f32<T>(v * r2 * p.w_pre[c]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
gnorm_backward_kernel(GnormRows<T> p, GnormGrads<T> g, float* __restrict__ partial) {
  __shared__ float red[32];
  const float inv = 1.f / p.width;
  float* part = partial + static_cast<int64_t>(blockIdx.x) * 3 * p.width;
  if (partial)
    for (int c = threadIdx.x; c < 3 * p.width; c += blockDim.x) part[c] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float r1 = 1.f, r2 = 1.f, dot2 = 0.f;
    if (p.w_post) {
      float sum = 0.f;
      for (int c = threadIdx.x; c < p.width; c += blockDim.x) {
        const float v = to_f32(p.f[row * p.ldf + c]);
        sum = fmaf(v, v, sum);
      }
      r1 = 1.f / sqrtf(block_sum(sum, red) * inv + p.eps);
    }
    if (g.du) {
      float sum = 0.f, dot = 0.f;
      for (int c = threadIdx.x; c < p.width; c += blockDim.x) {
        const float v = new_residual(p, row, c, r1);
        sum = fmaf(v, v, sum);
        dot = fmaf(to_f32(g.du[row * g.lddu + c]) * p.w_pre[c], v, dot);
      }
      r2 = 1.f / sqrtf(block_sum(sum, red) * inv + p.eps);
      dot2 = block_sum(dot, red) * inv * r2 * r2 * r2;
    }
    float dot1 = 0.f;
    for (int c = threadIdx.x; c < p.width; c += blockDim.x) {
      const float v = new_residual(p, row, c, r1);
      float d = g.dy ? to_f32(g.dy[row * g.lddy + c]) : 0.f;
      if (g.du) {
        const float du = to_f32(g.du[row * g.lddu + c]);
        d += du * p.w_pre[c] * r2 - v * dot2;
        if (g.dw_pre) part[2 * p.width + c] += du * v * r2;
      }
      if (g.dx) g.dx[row * g.lddx + c] = from_f32<T>(d);
      const float n = to_f32(p.f[row * p.ldf + c]) * r1;
      const float nw = p.w_post ? n * p.w_post[c] : n;
      const Gate t = p.z ? gate_of(to_f32(p.z[row * p.ldz + c]), p.gate) : Gate{1.f, 0.f};
      if (g.dscale) part[p.width + c] += d * nw * t.act;
      if (p.scale) d *= p.scale[c];
      if (g.dz) g.dz[row * g.lddz + c] = from_f32<T>(d * nw * t.slope);
      d *= t.act;
      if (g.dw_post) part[c] += d * n;
      if (p.w_post) dot1 = fmaf(d * p.w_post[c], n, dot1);
    }
    if (p.w_post) dot1 = block_sum(dot1, red) * inv;
    for (int c = threadIdx.x; c < p.width; c += blockDim.x) {
      const float v = new_residual(p, row, c, r1);
      float d = g.dy ? to_f32(g.dy[row * g.lddy + c]) : 0.f;
      if (g.du) d += to_f32(g.du[row * g.lddu + c]) * p.w_pre[c] * r2 - v * dot2;
      if (p.scale) d *= p.scale[c];
      if (p.z) d *= gate_of(to_f32(p.z[row * p.ldz + c]), p.gate).act;
      if (p.w_post) d = r1 * (d * p.w_post[c] - to_f32(p.f[row * p.ldf + c]) * r1 * dot1);
      g.df[row * g.lddf + c] = from_f32<T>(d);
    }
  }
}

// The three sums over rows: the blocks' parts in their order.
__global__ void __launch_bounds__(128)
gnorm_sums_kernel(int width, int parts, const float* __restrict__ partial, float* dw_post,
                  float* dscale, float* dw_pre) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  float* out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dscale : dw_pre;
  if (c >= width || out == nullptr) return;
  float sum = 0.f;
  for (int k = 0; k < parts; ++k)
    sum += partial[(static_cast<int64_t>(k) * 3 + blockIdx.y) * width + c];
  out[c] = sum;
}

int grad_blocks(int64_t rows) {
  return static_cast<int>(rows < kGradBlocks ? rows : kGradBlocks);
}

}  // namespace

size_t gnorm_backward_workspace(int width, int64_t rows) {
  return static_cast<size_t>(grad_blocks(rows)) * 3 * width * sizeof(float);
}

template <typename T>
cudaError_t launch_gnorm(const GnormRows<T>& p, T* y, int64_t ldy, T* u, int64_t ldu,
                         cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.rows < (1 << 20) ? p.rows : (1 << 20));
  gnorm_kernel<T><<<grid, kThreads, 0, stream>>>(p, y, ldy, u, ldu);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gnorm_backward(const GnormRows<T>& p, const GnormGrads<T>& g, void* work,
                                  cudaStream_t stream) {
  const bool sums = g.dw_post || g.dscale || g.dw_pre;
  float* partial = sums ? static_cast<float*>(work) : nullptr;
  const int parts = grad_blocks(p.rows);
  if (parts > 0) {
    gnorm_backward_kernel<T><<<parts, kThreads, 0, stream>>>(p, g, partial);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  gnorm_sums_kernel<<<dim3((p.width + 127) / 128, 3), 128, 0, stream>>>(
      p.width, parts, partial, g.dw_post, g.dscale, g.dw_pre);
  return cudaGetLastError();
}

#define BSOLVE_GNORM(T)                                                                         \
  template cudaError_t launch_gnorm<T>(const GnormRows<T>&, T*, int64_t, T*, int64_t,           \
                                       cudaStream_t);                                           \
  template cudaError_t launch_gnorm_backward<T>(const GnormRows<T>&, const GnormGrads<T>&,      \
                                                void*, cudaStream_t);
BSOLVE_GNORM(float)
BSOLVE_GNORM(__nv_bfloat16)
BSOLVE_GNORM(__half)
#undef BSOLVE_GNORM

}  // namespace bsolve
