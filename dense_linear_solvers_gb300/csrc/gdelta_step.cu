// One row of the gated delta rule for each of a batch of sequences, from their kept states
// (bs_gdelta_step_batched).
//
//   m = k^T S, n = q^T S,  d = beta (v - a m),  S' = a S + k d^T,  o = scale (a n + (q k) d),  a = e^g.
// S is read once into registers, both products taken from it, and written once: bound by
// HBM for a batch, by latency for one sequence. A block has all dk rows of some columns of one head's state: 128
// columns by sixteen warps where that gives every SM several blocks, else 32 by eight. 200 rows of 32 heads 128 x 128:
// 140 us (6.0 TB/s of the states' one read and one write, 89% of a copy's rate; 128 columns by eight warps 176);
// one row 6 to 9 us, a call of torch and a launch.
#include "gdelta_tile.cuh"

namespace bsolve {
namespace {

constexpr int kMaxDk = 128;

// V columns a thread, LANES threads a row of the block's columns.
template <typename T, int V, int LANES, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 1024 / (kWarps * 32))
step_kernel(GdeltaRows<T> p, float* state, int64_t num_slots, const int32_t* slots, T* o, int64_t ldo,
            int slices) {
  constexpr int COLS = V * LANES, ROWS = 32 / LANES, N = kMaxDk / (kWarps * ROWS);
  using Vec = std::conditional_t<V == 4, float4, float>;
  __shared__ float qs[kMaxDk], ks[kMaxDk], qk[kWarps];
  __shared__ __align__(16) float part[kWarps][2][COLS];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int64_t part_blocks = static_cast<int64_t>(p.heads_v) * slices;
  const int64_t j = blockIdx.x / part_blocks;
  const int rest = static_cast<int>(blockIdx.x % part_blocks), h = rest / slices;
  const int c0 = (rest % slices) * COLS, c = c0 + (lane % LANES) * V;
  const int kh = h / (p.heads_v / p.heads_k);
  const int64_t slot = slots ? slots[j] : j;
  T* to = o + j * ldo + static_cast<int64_t>(h) * p.dv;
  if (slot < 0 || slot >= num_slots) {
    for (int x = c0 + threadIdx.x; x < min(c0 + COLS, p.dv); x += blockDim.x) to[x] = from_f32<T>(0.f);
    return;
  }
  float* S = state + (slot * p.heads_v + h) * p.dk * p.dv;
  const bool in = c < p.dv;  // V divides dv where it is 4
  float s[N][V];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int d = (n * kWarps + warp) * ROWS + lane / LANES;
    const bool have = in && d < p.dk;
    if constexpr (V == 4) {
      const float4 f = have ? *reinterpret_cast<const float4*>(S + d * p.dv + c)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
      s[n][0] = f.x, s[n][1] = f.y, s[n][2] = f.z, s[n][3] = f.w;
    } else {
      s[n][0] = have ? S[d * p.dv + c] : 0.f;
    }
  }
  if (threadIdx.x < kMaxDk) {
    const bool have = static_cast<int>(threadIdx.x) < p.dk;
    const float q = have ? to_f32(p.q[j * p.ldq + kh * p.dk + threadIdx.x]) : 0.f;
    const float k = have ? to_f32(p.k[j * p.ldk + kh * p.dk + threadIdx.x]) : 0.f;
    qs[threadIdx.x] = q;
    ks[threadIdx.x] = k;
    float sum = __fmul_rn(q, k);
#pragma unroll
    for (int m = 16; m; m /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
    if (lane == 0) qk[warp] = sum;
  }
  const float a = expf(p.g[j * p.ldg + h]), beta = p.beta[j * p.ldbeta + h];
  float v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = in ? to_f32(p.v[j * p.ldv + h * p.dv + c + e]) : 0.f;
  __syncthreads();
  float m[2][V];
#pragma unroll
  for (int e = 0; e < V; ++e) m[0][e] = m[1][e] = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int d = (n * kWarps + warp) * ROWS + lane / LANES;
    const float k = ks[d], q = qs[d];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      m[0][e] = __fmaf_rn(k, s[n][e], m[0][e]);
      m[1][e] = __fmaf_rn(q, s[n][e], m[1][e]);
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
      for (int d = 16; d >= LANES; d /= 2) m[x][e] += __shfl_xor_sync(0xFFFFFFFFu, m[x][e], d);
  if (lane < LANES) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      Vec w;
      if constexpr (V == 4) w = make_float4(m[x][0], m[x][1], m[x][2], m[x][3]);
      else w = m[x][0];
      *reinterpret_cast<Vec*>(&part[warp][x][lane * V]) = w;
    }
  }
  __syncthreads();
  const float dot = (qk[0] + qk[1]) + (qk[2] + qk[3]);
  float delta[V], y[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float km = 0.f, qm = 0.f;
    const int x = (lane % LANES) * V + e;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      km += part[w][0][x];
      qm += part[w][1][x];
    }
    delta[e] = __fmul_rn(beta, __fmaf_rn(-a, km, v[e]));
    y[e] = __fmul_rn(p.scale, __fmaf_rn(a, qm, __fmul_rn(dot, delta[e])));
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int d = (n * kWarps + warp) * ROWS + lane / LANES;
    if (!in || d >= p.dk) continue;
    const float k = ks[d];
#pragma unroll
    for (int e = 0; e < V; ++e) s[n][e] = __fmaf_rn(a, s[n][e], __fmul_rn(k, delta[e]));
    if constexpr (V == 4)
      *reinterpret_cast<float4*>(S + d * p.dv + c) = make_float4(s[n][0], s[n][1], s[n][2], s[n][3]);
    else
      S[d * p.dv + c] = s[n][0];
  }
  if (warp == 0 && lane < LANES && in)
#pragma unroll
    for (int e = 0; e < V; ++e) to[c + e] = from_f32<T>(y[e]);
}

template <typename T, int V, int LANES, int kWarps>
cudaError_t step(const GdeltaRows<T>& p, float* state, int64_t num_slots, const int32_t* slots, T* o,
                 int64_t ldo, cudaStream_t stream) {
  const int slices = (p.dv + V * LANES - 1) / (V * LANES);
  step_kernel<T, V, LANES, kWarps><<<static_cast<unsigned>(p.batch * p.heads_v * slices), kWarps * 32, 0, stream>>>(
      p, state, num_slots, slots, o, ldo, slices);
  return cudaGetLastError();
}

}  // namespace

template <typename T>
cudaError_t launch_gdelta_step(const GdeltaRows<T>& p, float* state, int64_t num_slots,
                               const int32_t* slots, T* o, int64_t ldo, cudaStream_t stream) {
  if (p.dv % 4 != 0 || (reinterpret_cast<uintptr_t>(state) & 15) != 0)
    return step<T, 1, 32, 8>(p, state, num_slots, slots, o, ldo, stream);
  if (p.batch * p.heads_v * ((p.dv + 127) / 128) >= 4 * kSms)
    return step<T, 4, 32, 16>(p, state, num_slots, slots, o, ldo, stream);
  return step<T, 4, 8, 8>(p, state, num_slots, slots, o, ldo, stream);
}
template cudaError_t launch_gdelta_step(const GdeltaRows<float>&, float*, int64_t, const int32_t*,
                                        float*, int64_t, cudaStream_t);
template cudaError_t launch_gdelta_step(const GdeltaRows<__nv_bfloat16>&, float*, int64_t,
                                        const int32_t*, __nv_bfloat16*, int64_t, cudaStream_t);
template cudaError_t launch_gdelta_step(const GdeltaRows<__half>&, float*, int64_t, const int32_t*,
                                        __half*, int64_t, cudaStream_t);

}  // namespace bsolve
