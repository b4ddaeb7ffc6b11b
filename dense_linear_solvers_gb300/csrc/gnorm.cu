// The norms around a block with its gate and residual scale (bs_gnorm calls of bsolve.h).
//
// A row is read once into registers, by one warp where it is short and by one block of 4 to 32
// warps where it is long, reduced once for each mean, and its outputs are written once. Blocks
// walk the rows at the grid's distance, so that the parameters stay in the first cache level and
// the backward pass keeps its three sums over rows on the chip: each block adds them up in
// shared memory, every thread its own columns, and writes one part of them at its end; a
// second kernel adds the parts in order. Rows too long for a block's registers run the
// looped kernels at the end, which read a row once for each mean and once for the outputs.
#include <type_traits>

#include "gnorm_math.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {
namespace {

constexpr int kSms = 152;

// Sums of N values over a row's warps, the same bits in every thread. Consecutive calls take
// the two halves of `red` in turn, so that one barrier a call is enough.
template <int N, int WARPS>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N][32], int& turn) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], m);
  if constexpr (WARPS > 1) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) red[turn][k][warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = red[turn][k][lane & (WARPS - 1)];
#pragma unroll
      for (int m = WARPS / 2; m > 0; m >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], m);
    }
    turn ^= 1;
  }
}

// Row number and thread of the row, of the calling thread: WARPS == 1: four rows a block.
template <int WARPS>
struct Place {
  static constexpr int kThreads = 32 * WARPS;
  static constexpr int kBlock = WARPS == 1 ? 128 : kThreads;
  static constexpr int kRows = kBlock / kThreads;
  static __device__ __forceinline__ int thread() {
    return WARPS == 1 ? threadIdx.x & 31 : threadIdx.x;
  }
  static __device__ __forceinline__ int64_t first() {
    return WARPS == 1 ? blockIdx.x * int64_t(kRows) + (threadIdx.x >> 5) : blockIdx.x;
  }
  static __device__ __forceinline__ int64_t stride() { return gridDim.x * int64_t(kRows); }
};

// ------------------------------------------------------------------ forward
template <typename T, int K, int WARPS, bool ALIGNED>
__global__ void __launch_bounds__(Place<WARPS>::kBlock, WARPS == 1 ? 8 : 32 / WARPS)
gnorm_kernel(GnormRows<T> p, T* __restrict__ y, int64_t ldy, T* __restrict__ u, int64_t ldu) {
  using P = Place<WARPS>;
  constexpr int VE = kVecElements<T>, N = P::kThreads;
  __shared__ float red[2][1][32];
  int turn = 0;
  const int t = P::thread();
  const float inv = 1.f / p.width;
  for (int64_t row = P::first(); row < p.rows; row += P::stride()) {
    RowVec<T> f[K], z[K], x[K];
    const T* zr = p.z ? p.z + row * p.ldz : nullptr;
    const T* xr = p.x ? p.x + row * p.ldx : nullptr;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      f[k] = load_row<T, N, ALIGNED>(p.f + row * p.ldf, t, k, p.width);
      z[k] = load_row<T, N, ALIGNED>(zr, t, k, p.width);
      x[k] = load_row<T, N, ALIGNED>(xr, t, k, p.width);
    }
    float r1 = 1.f;
    if (p.w_post) {
      float sum[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VE; ++e) sum[0] = fmaf(to_f32(f[k].e[e]), to_f32(f[k].e[e]), sum[0]);
      row_sums<1, WARPS>(sum, red, turn);
      r1 = 1.f / sqrtf(fmaf(sum[0], inv, p.eps));
    }
    float v[K][VE], sum[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float w[VE];
      load_params<T, N, ALIGNED>(p.w_post, 1.f, t, k, p.width, w);
#pragma unroll
      for (int e = 0; e < VE; ++e) v[k][e] = to_f32(f[k].e[e]) * r1 * w[e];
      if (p.z)
#pragma unroll
        for (int e = 0; e < VE; ++e) v[k][e] *= gate_of(to_f32(z[k].e[e]), p.gate).act;
      load_params<T, N, ALIGNED>(p.scale, 1.f, t, k, p.width, w);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        v[k][e] = fmaf(v[k][e], w[e], to_f32(x[k].e[e]));
        sum[0] = fmaf(v[k][e], v[k][e], sum[0]);
      }
      if (y) store_row<T, N, ALIGNED>(y + row * ldy, t, k, p.width, v[k]);
    }
    if (u) {
      row_sums<1, WARPS>(sum, red, turn);
      const float r2 = 1.f / sqrtf(fmaf(sum[0], inv, p.eps));
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float w[VE];
        load_params<T, N, ALIGNED>(p.w_pre, 1.f, t, k, p.width, w);
#pragma unroll
        for (int e = 0; e < VE; ++e) v[k][e] *= r2 * w[e];
        store_row<T, N, ALIGNED>(u + row * ldu, t, k, p.width, v[k]);
      }
    }
  }
}

// ------------------------------------------------------------------ backward
//
// With n = f r1 (r1 = 1 / rms(f)), t = n w_post act(z), y = x + scale t, q = r2 = 1 / rms(y):
//   dx = dy + q du w_pre - y q^3 mean(du w_pre y),     dt = dx scale,
//   dz = dt n w_post act'(z),  dn = dt act(z) w_post,  df = r1 (dn - n mean(dn n)),
//   dw_pre = sum du y q,  dscale = sum dx t,  dw_post = sum dt act(z) n.
template <typename T, int K, int WARPS, bool ALIGNED>
__global__ void __launch_bounds__(Place<WARPS>::kBlock,
                                  WARPS == 1 ? 4 : (WARPS <= 16 && K == 1 ? 32 / WARPS : 1))
gnorm_backward_kernel(GnormRows<T> p, GnormGrads<T> g, float* __restrict__ partial) {
  using P = Place<WARPS>;
  constexpr int VE = kVecElements<T>, N = P::kThreads;
  __shared__ float red[2][2][32];
  __shared__ float red1[2][1][32];
  // [row of the block][3][K][VE][thread]: a warp's accesses fall into 32 banks
  extern __shared__ float sums[];
  int turn = 0, turn1 = 0;
  const int t = P::thread();
  const float inv = 1.f / p.width;
  float* mine = sums + (WARPS == 1 ? (threadIdx.x >> 5) * 3 * K * VE * N : 0) + t;
  if (partial)
#pragma unroll
    for (int j = 0; j < 3 * K * VE; ++j) mine[j * N] = 0.f;
  for (int64_t row = P::first(); row < p.rows; row += P::stride()) {
    RowVec<T> f[K], z[K], x[K], dy[K], du[K];
    const T* zr = p.z ? p.z + row * p.ldz : nullptr;
    const T* xr = p.x ? p.x + row * p.ldx : nullptr;
    const T* yr = g.dy ? g.dy + row * g.lddy : nullptr;
    const T* ur = g.du ? g.du + row * g.lddu : nullptr;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      f[k] = load_row<T, N, ALIGNED>(p.f + row * p.ldf, t, k, p.width);
      z[k] = load_row<T, N, ALIGNED>(zr, t, k, p.width);
      x[k] = load_row<T, N, ALIGNED>(xr, t, k, p.width);
      du[k] = load_row<T, N, ALIGNED>(ur, t, k, p.width);
      dy[k] = load_row<T, N, ALIGNED>(yr, t, k, p.width);
    }
    float r1 = 1.f;
    if (p.w_post) {
      float sum[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VE; ++e) sum[0] = fmaf(to_f32(f[k].e[e]), to_f32(f[k].e[e]), sum[0]);
      row_sums<1, WARPS>(sum, red1, turn1);
      r1 = 1.f / sqrtf(fmaf(sum[0], inv, p.eps));
    }
    float y[K][VE], both_sums[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float w[VE], c[VE];
      load_params<T, N, ALIGNED>(p.w_post, 1.f, t, k, p.width, w);
      load_params<T, N, ALIGNED>(p.scale, 1.f, t, k, p.width, c);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        float v = to_f32(f[k].e[e]) * r1 * w[e];
        if (p.z) v *= gate_of(to_f32(z[k].e[e]), p.gate).act;
        y[k][e] = fmaf(v, c[e], to_f32(x[k].e[e]));
      }
      if (g.du) {
        load_params<T, N, ALIGNED>(p.w_pre, 1.f, t, k, p.width, w);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          both_sums[0] = fmaf(y[k][e], y[k][e], both_sums[0]);
          both_sums[1] = fmaf(to_f32(du[k].e[e]) * w[e], y[k][e], both_sums[1]);
        }
      }
    }
    float r2 = 0.f, back = 0.f;
    if (g.du) {
      row_sums<2, WARPS>(both_sums, red, turn);
      r2 = 1.f / sqrtf(fmaf(both_sums[0], inv, p.eps));
      back = both_sums[1] * inv * r2 * r2 * r2;
    }
    float dn[K][VE], sum[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float w[VE], c[VE], d[VE], dz[VE];
      load_params<T, N, ALIGNED>(p.w_pre, 0.f, t, k, p.width, w);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float u = to_f32(du[k].e[e]);
        d[e] = fmaf(-y[k][e], back, fmaf(u * w[e], r2, to_f32(dy[k].e[e])));
        if (g.dw_pre) mine[((2 * K + k) * VE + e) * N] += u * y[k][e] * r2;
      }
      if (g.dx) store_row<T, N, ALIGNED>(g.dx + row * g.lddx, t, k, p.width, d);
      load_params<T, N, ALIGNED>(p.w_post, 1.f, t, k, p.width, w);
      load_params<T, N, ALIGNED>(p.scale, 1.f, t, k, p.width, c);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const Gate q = p.z ? gate_of(to_f32(z[k].e[e]), p.gate) : Gate{1.f, 0.f};
        const float n = to_f32(f[k].e[e]) * r1, nw = n * w[e];
        if (g.dscale) mine[((K + k) * VE + e) * N] += d[e] * nw * q.act;
        const float dt = d[e] * c[e];
        dz[e] = dt * nw * q.slope;
        const float da = dt * q.act;
        if (g.dw_post) mine[(k * VE + e) * N] += da * n;
        dn[k][e] = da * w[e];
        sum[0] = fmaf(dn[k][e], n, sum[0]);
      }
      if (g.dz) store_row<T, N, ALIGNED>(g.dz + row * g.lddz, t, k, p.width, dz);
    }
    float mean = 0.f;
    if (p.w_post) {
      row_sums<1, WARPS>(sum, red1, turn1);
      mean = sum[0] * inv;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (p.w_post)
#pragma unroll
        for (int e = 0; e < VE; ++e)
          dn[k][e] = r1 * fmaf(-(to_f32(f[k].e[e]) * r1), mean, dn[k][e]);
      store_row<T, N, ALIGNED>(g.df + row * g.lddf, t, k, p.width, dn[k]);
    }
  }
  if (!partial) return;
  // the block's part: [3][width]; the four warps of short rows in order
  if constexpr (WARPS == 1) __syncthreads();
  for (int j = WARPS == 1 ? threadIdx.x >> 5 : 0; j < 3 * K; j += P::kRows)
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const int c = row_element<T, N, ALIGNED>(t, j % K, e);
      if (c >= p.width) continue;
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < P::kRows; ++r) v += sums[(r * 3 * K * VE + j * VE + e) * N + t];
      partial[(blockIdx.x * int64_t(3) + j / K) * p.width + c] = v;
    }
}

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
  if (c < width)
    for (int k = warp; k < parts; k += kSumWarps)
      sum += partial[(static_cast<int64_t>(k) * 3 + blockIdx.y) * width + c];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= width) return;
  sum = 0.f;
  for (int w = 0; w < kSumWarps; ++w) sum += sums[w][lane];
  out[c] = sum;
}

// ------------------------------------------------------------------ long rows
constexpr int kLong = 1024;

__device__ __forceinline__ float block_sum(float v, float (*red)[1][32], int& turn) {
  float s[1] = {v};
  row_sums<1, kLong / 32>(s, red, turn);
  return s[0];
}

template <typename T>
__device__ __forceinline__ float new_residual(const GnormRows<T>& p, int64_t row, int c, float r1) {
  float t = to_f32(p.f[row * p.ldf + c]);
  if (p.w_post) t = t * r1 * p.w_post[c];
  if (p.z) t *= gate_of(to_f32(p.z[row * p.ldz + c]), p.gate).act;
  return fmaf(t, p.scale ? p.scale[c] : 1.f, p.x ? to_f32(p.x[row * p.ldx + c]) : 0.f);
}

template <typename T>
__device__ __forceinline__ float post_norm(const GnormRows<T>& p, int64_t row, float (*red)[1][32],
                                           int& turn) {
  if (!p.w_post) return 1.f;
  float sum = 0.f;
  for (int c = threadIdx.x; c < p.width; c += kLong) {
    const float v = to_f32(p.f[row * p.ldf + c]);
    sum = fmaf(v, v, sum);
  }
  return 1.f / sqrtf(fmaf(block_sum(sum, red, turn), 1.f / p.width, p.eps));
}

template <typename T>
__global__ void __launch_bounds__(kLong)
gnorm_long_kernel(GnormRows<T> p, T* __restrict__ y, int64_t ldy, T* __restrict__ u, int64_t ldu) {
  __shared__ float red[2][1][32];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float r1 = post_norm(p, row, red, turn);
    float r2 = 1.f;
    if (u) {
      float sum = 0.f;
      for (int c = threadIdx.x; c < p.width; c += kLong) {
        const float v = new_residual(p, row, c, r1);
        sum = fmaf(v, v, sum);
      }
      r2 = 1.f / sqrtf(fmaf(block_sum(sum, red, turn), 1.f / p.width, p.eps));
    }
    for (int c = threadIdx.x; c < p.width; c += kLong) {
      const float v = new_residual(p, row, c, r1);
      if (y) y[row * ldy + c] = from_f32<T>(v);
      if (u) u[row * ldu + c] = from_f32<T>(v * (r2 * p.w_pre[c]));
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kLong)
gnorm_long_backward_kernel(GnormRows<T> p, GnormGrads<T> g, float* __restrict__ partial) {
  __shared__ float red[2][1][32];
  int turn = 0;
  const float inv = 1.f / p.width;
  float* part = partial + static_cast<int64_t>(blockIdx.x) * 3 * p.width;
  if (partial)  // a thread touches its own columns only
    for (int j = 0; j < 3; ++j)
      for (int c = threadIdx.x; c < p.width; c += kLong) part[j * p.width + c] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float r1 = post_norm(p, row, red, turn);
    float r2 = 0.f, back = 0.f;
    if (g.du) {
      float sum = 0.f, dot = 0.f;
      for (int c = threadIdx.x; c < p.width; c += kLong) {
        const float v = new_residual(p, row, c, r1);
        sum = fmaf(v, v, sum);
        dot = fmaf(to_f32(g.du[row * g.lddu + c]) * p.w_pre[c], v, dot);
      }
      r2 = 1.f / sqrtf(fmaf(block_sum(sum, red, turn), inv, p.eps));
      back = block_sum(dot, red, turn) * inv * r2 * r2 * r2;
    }
    float dot = 0.f;
    for (int c = threadIdx.x; c < p.width; c += kLong) {
      const float v = new_residual(p, row, c, r1);
      float d = g.dy ? to_f32(g.dy[row * g.lddy + c]) : 0.f;
      if (g.du) {
        const float du = to_f32(g.du[row * g.lddu + c]);
        d = fmaf(-v, back, fmaf(du * p.w_pre[c], r2, d));
        if (g.dw_pre) part[2 * p.width + c] += du * v * r2;
      }
      if (g.dx) g.dx[row * g.lddx + c] = from_f32<T>(d);
      const float n = to_f32(p.f[row * p.ldf + c]) * r1;
      const float w = p.w_post ? p.w_post[c] : 1.f;
      const Gate q = p.z ? gate_of(to_f32(p.z[row * p.ldz + c]), p.gate) : Gate{1.f, 0.f};
      if (g.dscale) part[p.width + c] += d * (n * w) * q.act;
      const float dt = p.scale ? d * p.scale[c] : d;
      if (g.dz) g.dz[row * g.lddz + c] = from_f32<T>(dt * (n * w) * q.slope);
      const float da = dt * q.act;
      if (g.dw_post) part[c] += da * n;
      dot = fmaf(da * w, n, dot);
    }
    const float mean = p.w_post ? block_sum(dot, red, turn) * inv : 0.f;
    for (int c = threadIdx.x; c < p.width; c += kLong) {
      float d = g.dy ? to_f32(g.dy[row * g.lddy + c]) : 0.f;
      if (g.du)
        d = fmaf(-new_residual(p, row, c, r1), back,
                 fmaf(to_f32(g.du[row * g.lddu + c]) * p.w_pre[c], r2, d));
      if (p.scale) d *= p.scale[c];
      if (p.z) d *= gate_of(to_f32(p.z[row * p.ldz + c]), p.gate).act;
      if (p.w_post)
        d = r1 * fmaf(-(to_f32(p.f[row * p.ldf + c]) * r1), mean, d * p.w_post[c]);
      g.df[row * g.lddf + c] = from_f32<T>(d);
    }
  }
}

// ------------------------------------------------------------------ launches

// Warps a row and vectors a thread, from the vectors a row has: a warp while it holds them in two
// vectors a lane, then the fewest warps with one vector a thread (two for the longest).
struct Shape {
  int warps, vectors;
};

Shape shape_of(int width, int vec) {
  const int n = (width + vec - 1) / vec;
  if (n <= 32) return {1, 1};
  if (n <= 64) return {1, 2};
  if (n <= 128) return {4, 1};
  if (n <= 256) return {8, 1};
  if (n <= 512) return {16, 1};
  if (n <= 1024) return {32, 1};
  if (n <= 2048) return {32, 2};
  return {0, 0};  // long rows
}

// Blocks that walk the rows: what the GPU holds at once.
int blocks_for(const Shape& s, int64_t rows, int held) {
  const int64_t need = s.warps == 1 ? (rows + 3) / 4 : rows;
  return static_cast<int>(need < held ? need : held);
}

int backward_blocks(int width, int vec, int64_t rows) {
  const Shape s = shape_of(width, vec);
  const int held = s.warps == 0 ? kSms : kSms * (s.warps == 1 ? 4 : s.vectors == 1 ? 32 / s.warps : 1);
  return blocks_for(s, rows, held);
}

bool vec16(const void* p, int64_t bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(bytes)) & 15) == 0;
}

// Calls f with (vectors, warps) as compile-time values.
template <typename F>
cudaError_t with_shape(const Shape& s, F&& f) {
  using std::integral_constant;
  if (s.warps == 1 && s.vectors == 1) return f(integral_constant<int, 1>(), integral_constant<int, 1>());
  if (s.warps == 1) return f(integral_constant<int, 2>(), integral_constant<int, 1>());
  if (s.warps == 4) return f(integral_constant<int, 1>(), integral_constant<int, 4>());
  if (s.warps == 8) return f(integral_constant<int, 1>(), integral_constant<int, 8>());
  if (s.warps == 16) return f(integral_constant<int, 1>(), integral_constant<int, 16>());
  if (s.vectors == 1) return f(integral_constant<int, 1>(), integral_constant<int, 32>());
  return f(integral_constant<int, 2>(), integral_constant<int, 32>());
}

template <typename T, bool ALIGNED>
cudaError_t launch_forward(const Shape& s, const GnormRows<T>& p, T* y, int64_t ldy, T* u,
                           int64_t ldu, cudaStream_t stream) {
  return with_shape(s, [&](auto k, auto warps) {
    constexpr int K = decltype(k)::value, WARPS = decltype(warps)::value;
    const int grid = blocks_for(s, p.rows, kSms * (WARPS == 1 ? 8 : 64 / WARPS));
    gnorm_kernel<T, K, WARPS, ALIGNED><<<grid, Place<WARPS>::kBlock, 0, stream>>>(p, y, ldy, u, ldu);
    return cudaGetLastError();
  });
}

template <typename T, bool ALIGNED>
cudaError_t launch_backward(const Shape& s, const GnormRows<T>& p, const GnormGrads<T>& g,
                            float* partial, int parts, cudaStream_t stream) {
  return with_shape(s, [&](auto k, auto warps) {
    constexpr int K = decltype(k)::value, WARPS = decltype(warps)::value;
    constexpr int kShared = 3 * K * kVecElements<T> * Place<WARPS>::kBlock * 4;
    auto* kernel = gnorm_backward_kernel<T, K, WARPS, ALIGNED>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
    if (e != cudaSuccess) return e;
    kernel<<<parts, Place<WARPS>::kBlock, partial ? kShared : 0, stream>>>(p, g, partial);
    return cudaGetLastError();
  });
}

}  // namespace

size_t gnorm_backward_workspace(int width, int64_t rows) {
  // 16-bit rows have the fewest vectors; the larger of the two types' needs
  const int a = backward_blocks(width, 8, rows), b = backward_blocks(width, 4, rows);
  return static_cast<size_t>(a > b ? a : b) * 3 * width * sizeof(float);
}

template <typename T>
cudaError_t launch_gnorm(const GnormRows<T>& p, T* y, int64_t ldy, T* u, int64_t ldu,
                         cudaStream_t stream) {
  const Shape s = shape_of(p.width, kVecElements<T>);
  const int64_t es = sizeof(T);
  if (s.warps == 0) {
    gnorm_long_kernel<T><<<blocks_for(s, p.rows, 2 * kSms), kLong, 0, stream>>>(p, y, ldy, u, ldu);
    return cudaGetLastError();
  }
  const bool aligned = vec16(p.f, p.ldf * es) && vec16(p.z, p.ldz * es) && vec16(p.x, p.ldx * es) &&
                       vec16(y, ldy * es) && vec16(u, ldu * es) && vec16(p.w_post, 0) &&
                       vec16(p.scale, 0) && vec16(p.w_pre, 0);
  return aligned ? launch_forward<T, true>(s, p, y, ldy, u, ldu, stream)
                 : launch_forward<T, false>(s, p, y, ldy, u, ldu, stream);
}

template <typename T>
cudaError_t launch_gnorm_backward(const GnormRows<T>& p, const GnormGrads<T>& g, void* work,
                                  cudaStream_t stream) {
  const bool sums = g.dw_post || g.dscale || g.dw_pre;
  float* partial = sums ? static_cast<float*>(work) : nullptr;
  const Shape s = shape_of(p.width, kVecElements<T>);
  const int parts = backward_blocks(p.width, kVecElements<T>, p.rows);
  const int64_t es = sizeof(T);
  if (parts > 0) {
    cudaError_t e;
    if (s.warps == 0) {
      gnorm_long_backward_kernel<T><<<parts, kLong, 0, stream>>>(p, g, partial);
      e = cudaGetLastError();
    } else {
      const bool aligned =
          vec16(p.f, p.ldf * es) && vec16(p.z, p.ldz * es) && vec16(p.x, p.ldx * es) &&
          vec16(g.dy, g.lddy * es) && vec16(g.du, g.lddu * es) && vec16(g.df, g.lddf * es) &&
          vec16(g.dz, g.lddz * es) && vec16(g.dx, g.lddx * es) && vec16(p.w_post, 0) &&
          vec16(p.scale, 0) && vec16(p.w_pre, 0);
      e = aligned ? launch_backward<T, true>(s, p, g, partial, parts, stream)
                  : launch_backward<T, false>(s, p, g, partial, parts, stream);
    }
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  gnorm_sums_kernel<<<dim3((p.width + 31) / 32, 3), 32 * kSumWarps, 0, stream>>>(
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
