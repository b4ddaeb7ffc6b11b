// The part of the gated delta rule that no state enters (bs_gdelta calls): one block for each chunk
// of 64 rows and value head, all chunks at once.
//
// With b the running sum of the chunk's log decays, D_ri = e^(b_r - b_i) for i <= r and 0 above,
//   N = strict(K K^T o D),    mixing = scale (Q K^T o D),
//   inverse = (I + N diag(beta))^-1 for the forward pass, (I + diag(beta) N)^-1 for the backward one.
// The inverse of the unit lower triangular 64 x 64 system: four diagonal blocks of 16 by
// substitution, a column a lane; then two pairs of them, and the pair of these, by
// [X1 0; -X2 L21 X1, X2], in FP32. b is summed in 64 bits, in units of log 2, and kept as two FP32 numbers, so that
// a difference of neighbours is exact to its own last place behind however strong a decay; a log decay
// below -1000 (a reset, -infinity among them) counts as -1000, whose exponential is 0 as well.
//
// Blocks of four warps whose matrices take the place of q and k once the products are in registers: what bounds
// it are the barriers between the few steps, which five blocks an SM hide from each other (8 x 2,048 rows of 16 heads,
// BF16: 76 us; schedulers issue on 40% of the cycles).
#include "gdelta_tile.cuh"

namespace bsolve {
namespace {

constexpr int kThreads = 128;
constexpr int kLs = 68;  // row distance of the FP32 matrices: 16-byte aligned, banks apart
constexpr int kMs = 36;

template <int DK, int NT>
struct PrepShared {
  union {
    struct {
      __nv_bfloat16 q[NT][kChunk][DK + 8], k[NT][kChunk][DK + 8];
    } in;
    struct {
      float low[kChunk][kLs], x[kChunk][kLs], m[32][kMs];
    } solve;
  };
  float sum_hi[kChunk], sum_lo[kChunk], beta[kChunk];
  Span span;
};

// Two rows by four columns of sign a b, `depth` deep; a's rows A apart, b's B apart.
template <int A, int B, int DEPTH>
__device__ __forceinline__ void tile_product(float4 (&s)[2], const float* a, const float* b, float sign) {
  s[0] = s[1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < DEPTH; j += 4) {
    float4 v[2], w[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) v[r] = *reinterpret_cast<const float4*>(a + r * A + j);
#pragma unroll
    for (int d = 0; d < 4; ++d) w[d] = *reinterpret_cast<const float4*>(b + (j + d) * B);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const float f = sign * (d == 0 ? v[r].x : d == 1 ? v[r].y : d == 2 ? v[r].z : v[r].w);
        s[r].x = __fmaf_rn(f, w[d].x, s[r].x);
        s[r].y = __fmaf_rn(f, w[d].y, s[r].y);
        s[r].z = __fmaf_rn(f, w[d].z, s[r].z);
        s[r].w = __fmaf_rn(f, w[d].w, s[r].w);
      }
  }
}
// x21 = -x22 l21 x11 in blocks of SIZE from `base`; threads t of SIZE * SIZE / 8.
template <int SIZE, typename S>
__device__ __forceinline__ void join(S& sh, int base, int t, bool mine, float* m) {
  const int r = t / (SIZE / 4) * 2, c = t % (SIZE / 4) * 4;
  float4 s[2];
  if (mine) {
    tile_product<kLs, kLs, SIZE>(s, &sh.low[base + SIZE + r][base], &sh.x[base][base + c], 1.f);
    *reinterpret_cast<float4*>(m + r * kMs + c) = s[0];
    *reinterpret_cast<float4*>(m + (r + 1) * kMs + c) = s[1];
  }
  __syncthreads();
  if (mine) {
    tile_product<kLs, kMs, SIZE>(s, &sh.x[base + SIZE + r][base + SIZE], m + c, -1.f);
    *reinterpret_cast<float4*>(&sh.x[base + SIZE + r][base + c]) = s[0];
    *reinterpret_cast<float4*>(&sh.x[base + SIZE + r + 1][base + c]) = s[1];
  }
  __syncthreads();
}

template <typename T, int DK, bool VEC, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, 4)
prepare_kernel(GdeltaRows<T> p, Prepared* out) {
  constexpr int NT = Terms<T>::n, STRIDE = DK + 8;
  constexpr unsigned kTerm = kChunk * STRIDE * 2;
  extern __shared__ __align__(16) unsigned char raw[];
  auto& sh = *reinterpret_cast<PrepShared<DK, NT>*>(raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
  const int64_t place = blockIdx.x;
  const int h = blockIdx.y, kh = h / (p.heads_v / p.heads_k);
  if (warp == 0) {
    const Span s = chunk_at(p, place);
    if (lane == 0) sh.span = s;
  }
  __syncthreads();
  const Span span = sh.span;
  if (span.rows == 0) return;
  load_terms<T, DK, STRIDE, VEC>(&sh.in.q[0][0][0], p.q + span.row * p.ldq + kh * p.dk, p.ldq, span.rows,
                                 p.dk, threadIdx.x, kThreads);
  load_terms<T, DK, STRIDE, VEC>(&sh.in.k[0][0][0], p.k + span.row * p.ldk + kh * p.dk, p.ldk, span.rows,
                                 p.dk, threadIdx.x, kThreads);
  Prepared& o = out[place * p.heads_v + h];
  if (warp == 0) {
    double s[2];
    float beta[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * lane + e;
      const bool have = r < span.rows;
      const float gate = have ? p.g[(span.row + r) * p.ldg + h] : 0.f;
      s[e] = gate < -1000.f ? -1000.0 : static_cast<double>(gate);
      beta[e] = have ? p.beta[(span.row + r) * p.ldbeta + h] : 0.f;
    }
    s[1] += s[0];
    double run = s[1];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const double below = __shfl_up_sync(0xFFFFFFFFu, run, d);
      if (lane >= d) run += below;
    }
    const double last = __shfl_sync(0xFFFFFFFFu, run, 31), before = run - s[1];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * lane + e;
      const double b = (before + s[e]) * kLog2;
      o.sum_hi[r] = sh.sum_hi[r] = static_cast<float>(b);
      o.sum_lo[r] = sh.sum_lo[r] = static_cast<float>(b - static_cast<double>(static_cast<float>(b)));
      sh.beta[r] = beta[e];
      o.front[r] = power_of_two(static_cast<float>(b));
      o.back[r] = power_of_two(static_cast<float>(last * kLog2 - b));
      o.beta[r] = beta[e];
    }
  }
  cp_async_wait_all();
  __syncthreads();

  // A warp has 16 rows: of K K^T, and of Q K^T, or of K Q^T where the transposed products follow.
  const int mb = warp;
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[j][e] = qk[j][e] = 0.f;
  {
    const unsigned q = smem_address(&sh.in.q[0][0][0]), k = smem_address(&sh.in.k[0][0][0]);
    for (int d = 0; d < DK; d += 16) {
      unsigned a[NT][4], c[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        ldmatrix4(a[n], across(k + n * kTerm, STRIDE, mb * 16, d));
        if (!BACKWARD) ldmatrix4(c[n], across(q + n * kTerm, STRIDE, mb * 16, d));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool below = j <= mb, mixes = BACKWARD ? j >= mb : below;
        unsigned b[NT][4], e[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (below) ldmatrix4(b[n], along<STRIDE>(k + n * kTerm, j * 16, d));
          if (BACKWARD && mixes) ldmatrix4(e[n], along<STRIDE>(q + n * kTerm, j * 16, d));
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float(&x)[4] = kk[2 * j + half];
          float(&y)[4] = qk[2 * j + half];
          auto pair = [&](float(&to)[4], const unsigned(&l)[NT][4], const unsigned(&r)[NT][4]) {
            mma(to, l[0], r[0][2 * half], r[0][2 * half + 1]);
            if constexpr (NT == 2) {
              mma(to, l[0], r[1][2 * half], r[1][2 * half + 1]);
              mma(to, l[1], r[0][2 * half], r[0][2 * half + 1]);
            }
          };
          if (below) pair(x, a, b);
          if (mixes) {
            if constexpr (BACKWARD) pair(y, a, e);
            else pair(y, c, b);
          }
        }
      }
    }
  }
  __syncthreads();  // q and k give way to the matrices
  auto& m = sh.solve;
  // the decayed products: L into shared memory, the mixing matrix into its place
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k <= mb) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = mb * 16 + g + half * 8, i = k * 16 + j * 8 + t2;
          float v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float d = decay_between(sh.sum_hi, sh.sum_lo, r, i + e);
            v[e] = i + e < r ? __fmul_rn(sh.beta[BACKWARD ? r : i + e],
                                         __fmul_rn(kk[2 * k + j][2 * half + e], d)) : 0.f;
            if (!BACKWARD)
              qk[2 * k + j][2 * half + e] =
                  i + e <= r ? __fmul_rn(p.scale, __fmul_rn(qk[2 * k + j][2 * half + e], d)) : 0.f;
          }
          *reinterpret_cast<float2*>(&m.low[r][i]) = make_float2(v[0], v[1]);
        }
    }
    if (BACKWARD ? k < mb : k > mb) continue;
    if (BACKWARD)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = mb * 16 + g + (e / 2) * 8, r = k * 16 + j * 8 + t2 + (e & 1);
          const float d = decay_between(sh.sum_hi, sh.sum_lo, r, i);
          qk[2 * k + j][e] = i <= r ? __fmul_rn(p.scale, __fmul_rn(qk[2 * k + j][e], d)) : 0.f;
        }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const Split a = split(qk[2 * k][2 * half], qk[2 * k][2 * half + 1]),
                  b = split(qk[2 * k + 1][2 * half], qk[2 * k + 1][2 * half + 1]);
      o.mixing[BACKWARD ? upper_piece(mb, half, k) : lower_piece(mb, half, k)][lane] =
          make_uint4(a.hi, b.hi, a.lo, b.lo);
    }
  }
  // zeros right of the diagonal blocks, which the joins read
  for (int j = threadIdx.x; j < 32 * 16; j += kThreads)
    m.x[(j / 256) * 32 + (j / 16) % 16][(j / 256) * 32 + 16 + j % 16] = 0.f;
  __syncthreads();
  // diagonal blocks
  if (lane < 16) {
    const float* at = &m.low[warp * 16][warp * 16];
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == lane ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < r; ++j) s = __fmaf_rn(-at[r * kLs + j], x[j], s);
      x[r] = s;
      m.x[warp * 16 + r][warp * 16 + lane] = s;
    }
  }
  __syncthreads();
  // pairs of 16, then the pair of 32
  join<16>(m, threadIdx.x / 32 * 32, threadIdx.x % 32, threadIdx.x < 64, &m.m[threadIdx.x / 32 % 2 * 16][0]);
  join<32>(m, 0, threadIdx.x, true, &m.m[0][0]);
  // a warp has the pieces of two groups of columns
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (BACKWARD ? k < warp : k > warp) continue;
      const int d = k * 16 + t2, col = (2 * warp + half) * 8 + g;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int depth = d + (e & 1) + (e / 2) * 8;
        v[e] = BACKWARD ? m.x[depth][col] : m.x[col][depth];
      }
      const Split a = split(v[0], v[1]), b = split(v[2], v[3]);
      o.inverse[BACKWARD ? upper_piece(warp, half, k) : lower_piece(warp, half, k)][lane] =
          make_uint4(a.hi, b.hi, a.lo, b.lo);
    }
}

template <typename T, int DK, bool VEC>
cudaError_t prepare(const GdeltaRows<T>& p, bool for_backward, Prepared* out, cudaStream_t stream) {
  const int64_t places = gdelta_places(p.batch, p.rows);
  const size_t shared = sizeof(PrepShared<DK, Terms<T>::n>);
  auto* kernel = for_backward ? prepare_kernel<T, DK, VEC, true> : prepare_kernel<T, DK, VEC, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(shared));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(places), p.heads_v);
  kernel<<<grid, kThreads, shared, stream>>>(p, out);
  return cudaGetLastError();
}

}  // namespace

template <typename T>
cudaError_t launch_gdelta_prepare(const GdeltaRows<T>& p, bool for_backward, Prepared* out,
                                  cudaStream_t stream) {
  const bool vec = gdelta_aligned(p.q, p.ldq, p.dk) && gdelta_aligned(p.k, p.ldk, p.dk);
  if (p.dk <= 64)
    return vec ? prepare<T, 64, true>(p, for_backward, out, stream)
               : prepare<T, 64, false>(p, for_backward, out, stream);
  return vec ? prepare<T, 128, true>(p, for_backward, out, stream)
             : prepare<T, 128, false>(p, for_backward, out, stream);
}
template cudaError_t launch_gdelta_prepare(const GdeltaRows<float>&, bool, Prepared*, cudaStream_t);
template cudaError_t launch_gdelta_prepare(const GdeltaRows<__nv_bfloat16>&, bool, Prepared*,
                                           cudaStream_t);
template cudaError_t launch_gdelta_prepare(const GdeltaRows<__half>&, bool, Prepared*, cudaStream_t);

}  // namespace bsolve
