// The part of the gated delta rule that no state enters (bs_gdelta calls): one block for each chunk
// of 64 rows and key head, all chunks at once.
//
// With b the running sum of the chunk's log decays, D_ri = e^(b_r - b_i) for i <= r and 0 above,
//   N = strict(K K^T o D),    mixing = scale (Q K^T o D),
//   inverse = (I + N diag(beta))^-1 for the forward pass, (I + diag(beta) N)^-1 for the backward one.
// The inverse of the unit lower triangular 64 x 64 system: four diagonal blocks of 16 by
// substitution, a column a lane; then two pairs of them, and the pair of these, by
// [X1 0; -X2 L21 X1, X2], in FP32. K K^T and Q K^T are taken once for all value heads of the
// key head. b is summed in 64 bits and kept as two FP32 numbers, so that a difference of neighbours
// is exact to its own last place behind however strong a decay; a log decay
// below -1000 (a reset, -infinity among them) counts as -1000, whose exponential is 0 as well.
#include "gdelta_tile.cuh"

namespace bsolve {
namespace {

constexpr int kThreads = 256;
constexpr int kLs = 68;  // row distance of the FP32 matrices: 16-byte aligned, banks apart
constexpr int kMs = 36;

template <int DK, int NT>
struct PrepShared {
  __nv_bfloat16 q[NT][kChunk][DK + 8];
  __nv_bfloat16 k[NT][kChunk][DK + 8];
  float low[kChunk][kLs];
  float x[kChunk][kLs];
  float m[32][kMs];
  float sum_hi[kChunk], sum_lo[kChunk], beta[kChunk];
  Span span;
};

// out (rows x 4 columns at c) = sign * a (row r of `depth`) * b.
__device__ __forceinline__ float4 row_times(const float* a, const float* b, int b_stride, int depth,
                                            float sign) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int j = 0; j < depth; ++j) {
    const float v = sign * a[j];
    const float4 w = *reinterpret_cast<const float4*>(b + j * b_stride);
    s.x = __fmaf_rn(v, w.x, s.x);
    s.y = __fmaf_rn(v, w.y, s.y);
    s.z = __fmaf_rn(v, w.z, s.z);
    s.w = __fmaf_rn(v, w.w, s.w);
  }
  return s;
}

template <typename T, int DK, bool VEC, bool BACKWARD>
__global__ void __launch_bounds__(kThreads)
prepare_kernel(GdeltaRows<T> p, int per, Prepared* out) {
  constexpr int NT = Terms<T>::n, STRIDE = DK + 8;
  extern __shared__ __align__(16) unsigned char raw[];
  auto& sh = *reinterpret_cast<PrepShared<DK, NT>*>(raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
  const int64_t place = blockIdx.x;
  const int kh = blockIdx.y, group = p.heads_v / p.heads_k;
  if (warp == 0) {
    const Span s = chunk_at(p, place);
    if (lane == 0) sh.span = s;
  }
  __syncthreads();
  const Span span = sh.span;
  if (span.rows == 0) return;
  load_terms<T, DK, STRIDE, VEC>(&sh.q[0][0][0], p.q + span.row * p.ldq + kh * p.dk, p.ldq, span.rows,
                                 p.dk);
  load_terms<T, DK, STRIDE, VEC>(&sh.k[0][0][0], p.k + span.row * p.ldk + kh * p.dk, p.ldk, span.rows,
                                 p.dk);
  cp_async_wait_all();
  __syncthreads();

  // Warps 0 to 3: rows of K K^T; 4 to 7: of Q K^T, or of K Q^T where the transposed products follow.
  const int mb = warp & 3;
  const bool mixes = warp >= 4;
  float acc[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  {
    constexpr unsigned kTerm = kChunk * STRIDE * 2;
    const unsigned q_at = smem_addr(&sh.q[0][0][0]), k_at = smem_addr(&sh.k[0][0][0]);
    const unsigned first = mixes && !BACKWARD ? q_at : k_at, second = mixes && BACKWARD ? q_at : k_at;
    const bool upper = mixes && BACKWARD;
    for (int k = 0; k < DK; k += 16) {
      unsigned a[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
        ldmatrix4(a[n], across(first + n * kTerm, STRIDE, mb * 16, k));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (upper ? j < mb : j > mb) continue;
        unsigned b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          ldmatrix4(b[n], along<STRIDE>(second + n * kTerm, j * 16, k));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma(acc[2 * j + h], a[0], b[0][2 * h], b[0][2 * h + 1]);
          if constexpr (NT == 2) {
            mma(acc[2 * j + h], a[0], b[1][2 * h], b[1][2 * h + 1]);
            mma(acc[2 * j + h], a[1], b[0][2 * h], b[0][2 * h + 1]);
          }
        }
      }
    }
  }

  for (int h = kh * group + blockIdx.z * per, end = min(h + per, (kh + 1) * group); h < end; ++h) {
    Prepared& o = out[place * p.heads_v + h];
    __syncthreads();  // the last head's matrices are free
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
        const double b = before + s[e];
        o.sum_hi[r] = sh.sum_hi[r] = static_cast<float>(b);
        o.sum_lo[r] = sh.sum_lo[r] = static_cast<float>(b - static_cast<double>(sh.sum_hi[r]));
        sh.beta[r] = beta[e];
        o.front[r] = expf(static_cast<float>(b));
        o.back[r] = expf(static_cast<float>(last - b));
        o.beta[r] = beta[e];
      }
    } else {
      for (int j = threadIdx.x - 32; j < kChunk * kLs; j += kThreads - 32) sh.x[j / kLs][j % kLs] = 0.f;
    }
    __syncthreads();
    // the decayed products: L into shared memory, the mixing matrix into its place
    auto decay = [&](int r, int i) { return decay_between(sh.sum_hi, sh.sum_lo, r, i); };
    if (!mixes) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = mb * 16 + g + (e / 2) * 8, i = j * 8 + t2 + (e & 1);
          if (j / 2 <= mb)
            sh.low[r][i] = i < r ? __fmul_rn(sh.beta[BACKWARD ? r : i],
                                             __fmul_rn(acc[j][e], decay(r, i))) : 0.f;
        }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (BACKWARD ? k < mb : k > mb) continue;
        float v[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = mb * 16 + g + (e / 2) * 8, n = k * 16 + j * 8 + t2 + (e & 1);
            const int r = BACKWARD ? n : m, i = BACKWARD ? m : n;
            v[j][e] = i <= r ? __fmul_rn(p.scale, __fmul_rn(acc[2 * k + j][e], decay(r, i))) : 0.f;
          }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const Split a = split(v[0][2 * half], v[0][2 * half + 1]),
                      b = split(v[1][2 * half], v[1][2 * half + 1]);
          o.mixing[BACKWARD ? upper_piece(mb, half, k) : lower_piece(mb, half, k)][lane] =
              make_uint4(a.hi, b.hi, a.lo, b.lo);
        }
      }
    }
    __syncthreads();
    // diagonal blocks
    if (warp < 4 && lane < 16) {
      const float* at = &sh.low[warp * 16][warp * 16];
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float s = r == lane ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < r; ++j) s = __fmaf_rn(-at[r * kLs + j], x[j], s);
        x[r] = s;
        sh.x[warp * 16 + r][warp * 16 + lane] = s;
      }
    }
    __syncthreads();
    // pairs of 16, then the pair of 32
#pragma unroll
    for (int size = 16; size <= 32; size *= 2) {
      const int outputs = size * size / 4, pairs = 32 / size;
      const int pair = threadIdx.x / outputs, j = threadIdx.x % outputs;
      const int r = j / (size / 4), c = (j % (size / 4)) * 4, base = pair * 32;
      const bool mine = pair < pairs;
      if (mine)
        *reinterpret_cast<float4*>(&sh.m[pair * 16 + r][c]) =
            row_times(&sh.low[base + size + r][base], &sh.x[base][base + c], kLs, size, 1.f);
      __syncthreads();
      if (mine)
        *reinterpret_cast<float4*>(&sh.x[base + size + r][base + c]) =
            row_times(&sh.x[base + size + r][base + size], &sh.m[pair * 16][c], kMs, size, -1.f);
      __syncthreads();
    }
    // a warp has the pieces of one group of columns
    const int pair = warp / 2, half = warp & 1, col = warp * 8 + g;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (BACKWARD ? k < pair : k > pair) continue;
      const int d = k * 16 + t2;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int depth = d + (e & 1) + (e / 2) * 8;
        v[e] = BACKWARD ? sh.x[depth][col] : sh.x[col][depth];
      }
      const Split a = split(v[0], v[1]), b = split(v[2], v[3]);
      o.inverse[BACKWARD ? upper_piece(pair, half, k) : lower_piece(pair, half, k)][lane] =
          make_uint4(a.hi, b.hi, a.lo, b.lo);
    }
  }
}

template <typename T, int DK, bool VEC>
cudaError_t prepare(const GdeltaRows<T>& p, bool for_backward, Prepared* out, cudaStream_t stream) {
  const int64_t places = gdelta_places(p.batch, p.rows);
  const int group = p.heads_v / p.heads_k;
  // A block takes all value heads of its key head, which share K K^T and Q K^T, unless that leaves SMs
  // without a block.
  const int per = places * p.heads_k >= 2 * kSms ? group : 1;
  const size_t shared = sizeof(PrepShared<DK, Terms<T>::n>);
  auto* kernel = for_backward ? prepare_kernel<T, DK, VEC, true> : prepare_kernel<T, DK, VEC, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(shared));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(places), p.heads_k, (group + per - 1) / per);
  kernel<<<grid, kThreads, shared, stream>>>(p, per, out);
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
