// The gradients of q, k, g and beta, one block for each chunk and key head (bs_gdelta_backward_batched).
//
// With S the state in front of the chunk, M the solution's rows by beta (U = diag(beta) M), G the gradient
// of the state behind it, dU that of all uses of U, D the rows' incoming gradients, and
//   P = D S^T, Q' = dU S^T, E = M G^T (64 x dk),    H = D M^T, J = dU M^T (64 x 64),
//   x_ri = scale decay_ri beta_i H_ri (i <= r),     w_ri = -decay_ri beta_r beta_i J_ri (i < r),
//   dQ = diag(scale f) P + x K,
//   dK = x^T Q + (w + w^T) K + diag(e beta) E - diag(beta f) Q',
//   dbeta_r = J_rr, and for b, the sum of the log decays in the chunk,
//   db_r = sum_i (x qk + w kk)_ri - sum_i (x qk + w kk)_ir + scale f q.P - beta f k.Q' - e beta k.E,
// the last row's more by sum e beta k.E + f_last <G, S>; dg is db summed from the chunk's end.
// The sums over dv run over groups of 16 columns, whose operands lie in the registers' order in global memory
// and come by cp.async two groups ahead. Of the 64 x dk products a warp has all rows and an eighth of the
// columns, of the 64 x 64 ones one to four of the 20 tiles of 16 x 8 on and below the diagonal, those of the rows
// whose operands it has at hand. 8 x 2,048 rows of 16 heads 128 x 128, BF16: 445 us, more than half of it the groups
// of columns, whose products alone would take two thirds of that (with each head's first columns asked for only behind
// the last head, and db summed in 64 bits, 531). Value heads of one key head follow each other in the block, which adds
// them up in order in registers.
#include "gdelta_grad.cuh"

namespace bsolve {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kTiles = 20, kSlots = 4;  // tiles of the lower triangle, of a warp at most
constexpr int kDs = 24;                 // row distance of D's 16 columns: 16-byte pieces, banks apart
constexpr int kXs = kChunk + 8;

template <int DK, int NT>
struct GradStage {
  uint4 state[DK / 8][32], solution[4][2][32];      // S, M
  uint4 grad[DK / 8][32], solution_grad[4][2][32];  // G, dU
  __nv_bfloat16 d[NT][kChunk][kDs];
};

struct HeadRows {
  float front[kChunk], back[kChunk], beta[kChunk], sum_hi[kChunk], sum_lo[kChunk];
};

template <int DK, int NT>
struct GradShared {
  __nv_bfloat16 q[NT][kChunk][DK + 8];
  __nv_bfloat16 k[NT][kChunk][DK + 8];
  union {
    GradStage<DK, NT> stage[kStages];
    struct {
      GradStage<DK, NT> ahead[2];  // the next head's first columns come meanwhile
      __nv_bfloat16 x[2][kChunk][kXs], w[2][kChunk][kXs];  // two terms each
    } mix;
  };
  float4 qk[kSlots][kThreads], kk[kSlots][kThreads];  // of the warps' tiles
  HeadRows rows[2];  // of a head and the next one
  float dots[3][kWarps][kChunk];  // q.P, k.Q', k.E by the warps' columns
  float row_part[kTiles][16], col_part[kTiles][8];
  float product[kWarps];          // <G, S>
  Span span;
};

// Number of a tile: row block m, column group n.
__device__ __forceinline__ int tile_at(int m, int n) { return m * (m + 1) + n; }
__device__ __forceinline__ float2 two(unsigned v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float dot_terms(unsigned ahi, unsigned alo, unsigned bhi, unsigned blo) {
  const float2 a = two(ahi), c = two(alo), b = two(bhi), d = two(blo);
  return __fmaf_rn(__fadd_rn(a.x, c.x), __fadd_rn(b.x, d.x),
                   __fmul_rn(__fadd_rn(a.y, c.y), __fadd_rn(b.y, d.y)));
}
__device__ __forceinline__ void get_rows(unsigned (&hi)[4], unsigned (&lo)[4], const uint4 (&at)[2][32]) {
  const int lane = threadIdx.x & 31;
  const uint4 a = at[0][lane], b = at[1][lane];
  hi[0] = a.x, hi[1] = a.y, hi[2] = a.z, hi[3] = a.w;
  lo[0] = b.x, lo[1] = b.y, lo[2] = b.z, lo[3] = b.w;
}

template <typename T, int DK, bool VEC>
__global__ void __launch_bounds__(kThreads, 1) grad_kernel(GdeltaRows<T> p, GdeltaGrads<T> g) {
  constexpr int NT = Terms<T>::n, STRIDE = DK + 8, N8 = DK / 64, NB = DK / 8;
  using Shared = GradShared<DK, NT>;
  extern __shared__ __align__(16) unsigned char raw[];
  auto& sh = *reinterpret_cast<Shared*>(raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, gr = lane / 4, t2 = (lane & 3) * 2;
  const int64_t place = blockIdx.x;
  const int kh = blockIdx.y, group = p.heads_v / p.heads_k, groups = gdelta_groups(p.dv);
  if (warp == 0) {
    const Span s = chunk_at(p, place);
    if (lane == 0) sh.span = s;
  }
  __syncthreads();
  const Span span = sh.span;
  if (span.rows == 0) return;
  load_terms<T, DK, STRIDE, VEC>(&sh.q[0][0][0], p.q + span.row * p.ldq + kh * p.dk, p.ldq, span.rows,
                                 p.dk, threadIdx.x, kThreads);
  load_terms<T, DK, STRIDE, VEC>(&sh.k[0][0][0], p.k + span.row * p.ldk + kh * p.dk, p.ldk, span.rows,
                                 p.dk, threadIdx.x, kThreads);
  cp_async_commit();
  auto load = [&](int h, int w) {  // a group of 16 columns
    auto& st = sh.stage[w % kStages];
    const int64_t at = ((place * p.heads_v + h) * groups + w) * (kept_pieces(DK) * 32);
    constexpr int kPart = (NB + 8) * 32;
    uint4* to = &st.state[0][0] + threadIdx.x;
    const uint4 *s = g.forward + at + threadIdx.x, *d = g.backward + at + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kPart; j += kThreads) {
      cp_async_16(to + j, s + j, 16);
      cp_async_16(to + kPart + j, d + j, 16);
    }
    load_terms<T, 16, kDs, VEC>(&st.d[0][0][0], g.dout + span.row * g.lddo + h * p.dv + w * 16, g.lddo,
                                span.rows, p.dv - w * 16, threadIdx.x, kThreads);
  };
  auto begin = [&](int h) {  // a head's numbers and its first columns
    const Prepared& own = g.prepared[place * p.heads_v + h];
    HeadRows& to = sh.rows[h & 1];
    if (threadIdx.x < kChunk / 4) {
      const int r = threadIdx.x * 4;
      cp_async_16(&to.front[r], &own.front[r], 16);
      cp_async_16(&to.back[r], &own.back[r], 16);
      cp_async_16(&to.beta[r], &own.beta[r], 16);
      cp_async_16(&to.sum_hi[r], &own.sum_hi[r], 16);
      cp_async_16(&to.sum_lo[r], &own.sum_lo[r], 16);
    }
    load(h, 0);
    cp_async_commit();
    if (groups > 1) load(h, 1);
    cp_async_commit();
  };
  begin(kh * group);
  cp_async_wait_group<2>();
  __syncthreads();
  // q k and k k of the warp's tiles: a block of 16 rows, every other group of columns. The two warps of a scheduler
  // (w and w + 4) have five tiles together.
  const int rows16 = warp < 4 ? warp / 2 : 3 - (warp - 4) / 2, odd = warp & 1;
  for (int s = 0; s <= rows16; ++s) {
    float qk[4] = {0.f, 0.f, 0.f, 0.f}, kk[4] = {0.f, 0.f, 0.f, 0.f};
    for (int d = 0; d < DK; d += 16) {
      unsigned a[NT][4], b[NT][4], c[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        ldmatrix4(a[t], across(smem_address(&sh.q[t][0][0]), STRIDE, rows16 * 16, d));
        ldmatrix4(b[t], across(smem_address(&sh.k[t][0][0]), STRIDE, rows16 * 16, d));
        ldmatrix4(c[t], along<STRIDE>(smem_address(&sh.k[t][0][0]), s * 16, d));
      }
      mma(qk, a[0], odd ? c[0][2] : c[0][0], odd ? c[0][3] : c[0][1]);
      mma(kk, b[0], odd ? c[0][2] : c[0][0], odd ? c[0][3] : c[0][1]);
      if constexpr (NT == 2) {
        mma(qk, a[1], odd ? c[0][2] : c[0][0], odd ? c[0][3] : c[0][1]);
        mma(kk, b[1], odd ? c[0][2] : c[0][0], odd ? c[0][3] : c[0][1]);
        mma(qk, a[0], odd ? c[1][2] : c[1][0], odd ? c[1][3] : c[1][1]);
        mma(kk, b[0], odd ? c[1][2] : c[1][0], odd ? c[1][3] : c[1][1]);
      }
    }
    sh.qk[s][threadIdx.x] = make_float4(qk[0], qk[1], qk[2], qk[3]);
    sh.kk[s][threadIdx.x] = make_float4(kk[0], kk[1], kk[2], kk[3]);
  }

  float dq[4][N8][4], dk[4][N8][4];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int j = 0; j < N8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) dq[m][j][e] = dk[m][j][e] = 0.f;

  for (int h = kh * group; h < (kh + 1) * group; ++h) {
    const HeadRows& own = sh.rows[h & 1];
    float P[4][N8][4], R[4][N8][4], E[4][N8][4], H[kSlots][4], J[kSlots][4], product = 0.f;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int j = 0; j < N8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) P[m][j][e] = R[m][j][e] = E[m][j][e] = 0.f;
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) H[s][e] = J[s][e] = 0.f;

    for (int w = 0; w < groups; ++w) {
      cp_async_wait_group<1>();
      __syncthreads();  // this group is there, the one before the last is used
      if (w + 2 < groups) load(h, w + 2);
      cp_async_commit();
      const auto& st = sh.stage[w % kStages];
      const unsigned d = smem_address(&st.d[0][0][0]);
      uint4 S[N8], G[N8];
#pragma unroll
      for (int j = 0; j < N8; ++j) {
        S[j] = st.state[warp * N8 + j][lane];
        G[j] = st.grad[warp * N8 + j][lane];
        product = __fadd_rn(product, __fadd_rn(dot_terms(S[j].x, S[j].z, G[j].x, G[j].z),
                                               dot_terms(S[j].y, S[j].w, G[j].y, G[j].w)));
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        unsigned a[NT][4], hi[4], lo[4], mhi[4], mlo[4];
#pragma unroll
        for (int t = 0; t < NT; ++t) ldmatrix4(a[t], across(d + t * (kChunk * kDs * 2), kDs, m * 16, 0));
        get_rows(hi, lo, st.solution_grad[m]);
        get_rows(mhi, mlo, st.solution[m]);
        // the terms of one sum apart from each other: a product waits for its sum's last one
#pragma unroll
        for (int j = 0; j < N8; ++j) {
          mma(P[m][j], a[0], S[j].x, S[j].y);
          mma(R[m][j], hi, S[j].x, S[j].y);
          mma(E[m][j], mhi, G[j].x, G[j].y);
        }
#pragma unroll
        for (int j = 0; j < N8; ++j) {
          mma(P[m][j], a[0], S[j].z, S[j].w);
          mma(R[m][j], hi, S[j].z, S[j].w);
          mma(E[m][j], mhi, G[j].z, G[j].w);
        }
#pragma unroll
        for (int j = 0; j < N8; ++j) {
          if constexpr (NT == 2) mma(P[m][j], a[1], S[j].x, S[j].y);
          mma(R[m][j], lo, S[j].x, S[j].y);
          mma(E[m][j], mlo, G[j].x, G[j].y);
        }
        if (m == rows16) {
#pragma unroll
          for (int s = 0; s <= m; ++s) {
            const uint4 b = st.solution[s][0][lane], c = st.solution[s][1][lane];
            const unsigned b0 = odd ? b.y : b.x, b1 = odd ? b.w : b.z, c0 = odd ? c.y : c.x,
                           c1 = odd ? c.w : c.z;
            mma(H[s], a[0], b0, b1);
            mma(J[s], hi, b0, b1);
            mma(H[s], a[0], c0, c1);
            mma(J[s], hi, c0, c1);
            if constexpr (NT == 2) mma(H[s], a[1], b0, b1);
            mma(J[s], lo, b0, b1);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o /= 2) product += __shfl_xor_sync(0xFFFFFFFFu, product, o);
    if (lane == 0) sh.product[warp] = product;
    cp_async_wait_all();
    __syncthreads();  // the last stage gives way to x and w
    if (h + 1 < (kh + 1) * group) begin(h + 1);
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      if (s > rows16) continue;
      const int m = rows16, n = 2 * s + odd, tile = tile_at(m, n);
      const float4 q4 = sh.qk[s][threadIdx.x], k4 = sh.kk[s][threadIdx.x];
      const float qk[4] = {q4.x, q4.y, q4.z, q4.w}, kk[4] = {k4.x, k4.y, k4.z, k4.w};
      float x[4], w[4], sum[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = m * 16 + gr + (e / 2) * 8, i = n * 8 + t2 + (e & 1);
        const float decay = i <= r ? decay_between(own.sum_hi, own.sum_lo, r, i) : 0.f;
        const float b = __fmul_rn(decay, own.beta[i]);
        x[e] = i <= r ? __fmul_rn(__fmul_rn(p.scale, b), H[s][e]) : 0.f;
        w[e] = i < r ? -__fmul_rn(__fmul_rn(own.beta[r], b), J[s][e]) : 0.f;
        sum[e] = i <= r ? __fmaf_rn(x[e], qk[e], __fmul_rn(w[e], kk[e])) : 0.f;
        if (i == r && r < span.rows) g.dbeta[(span.row + r) * g.lddbeta + h] = J[s][e];
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = m * 16 + gr + half * 8, i = n * 8 + t2;
        const Split a = split(x[2 * half], x[2 * half + 1]), b = split(w[2 * half], w[2 * half + 1]);
        *reinterpret_cast<unsigned*>(&sh.mix.x[0][r][i]) = a.hi;
        *reinterpret_cast<unsigned*>(&sh.mix.x[1][r][i]) = a.lo;
        *reinterpret_cast<unsigned*>(&sh.mix.w[0][r][i]) = b.hi;
        *reinterpret_cast<unsigned*>(&sh.mix.w[1][r][i]) = b.lo;
        float v = sum[2 * half] + sum[2 * half + 1];
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
        v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
        if (t2 == 0) sh.row_part[tile][gr + half * 8] = v;
        float c = sum[half] + sum[half + 2];
#pragma unroll
        for (int o = 4; o < 32; o *= 2) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
        if (gr == 0) sh.col_part[tile][t2 + half] = c;
      }
    }
    // the rows' dots, and their parts of dq and dk
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = m * 16 + gr + half * 8;
        const float f = own.front[r], bf = __fmul_rn(own.beta[r], f), eb = __fmul_rn(own.back[r], own.beta[r]);
        float v[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < N8; ++j) {
          const int c = (warp * N8 + j) * 8 + t2;
          float2 q = two(*reinterpret_cast<const unsigned*>(&sh.q[0][r][c])),
                 k = two(*reinterpret_cast<const unsigned*>(&sh.k[0][r][c]));
          if constexpr (NT == 2) {
            const float2 ql = two(*reinterpret_cast<const unsigned*>(&sh.q[1][r][c])),
                         kl = two(*reinterpret_cast<const unsigned*>(&sh.k[1][r][c]));
            q.x += ql.x, q.y += ql.y, k.x += kl.x, k.y += kl.y;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int x = 2 * half + e;
            const float qe = e ? q.y : q.x, ke = e ? k.y : k.x;
            v[0] = __fmaf_rn(qe, P[m][j][x], v[0]);
            v[1] = __fmaf_rn(ke, R[m][j][x], v[1]);
            v[2] = __fmaf_rn(ke, E[m][j][x], v[2]);
            dq[m][j][x] = __fmaf_rn(__fmul_rn(p.scale, f), P[m][j][x], dq[m][j][x]);
            dk[m][j][x] = __fmaf_rn(eb, E[m][j][x], __fmaf_rn(-bf, R[m][j][x], dk[m][j][x]));
          }
        }
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          v[x] += __shfl_xor_sync(0xFFFFFFFFu, v[x], 1);
          v[x] += __shfl_xor_sync(0xFFFFFFFFu, v[x], 2);
          if (t2 == 0) sh.dots[x][warp][r] = v[x];
        }
      }
    __syncthreads();
    // x K, x^T Q + (w + w^T) K
    const unsigned x_at = smem_address(&sh.mix.x[0][0][0]), w_at = smem_address(&sh.mix.w[0][0][0]);
    constexpr unsigned kTerm = kChunk * kXs * 2;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
      unsigned q[NT][4], k[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        ldmatrix4_trans(q[t], across(smem_address(&sh.q[t][0][0]), STRIDE, kb * 16, warp * N8 * 8));
        ldmatrix4_trans(k[t], across(smem_address(&sh.k[t][0][0]), STRIDE, kb * 16, warp * N8 * 8));
      }
      auto add = [&](float (&c)[N8][4], const unsigned (&hi)[4], const unsigned (&lo)[4],
                     const unsigned (&b)[NT][4]) {
#pragma unroll
        for (int j = 0; j < N8; ++j) {
          mma(c[j], hi, b[0][2 * j], b[0][2 * j + 1]);
          mma(c[j], lo, b[0][2 * j], b[0][2 * j + 1]);
          if constexpr (NT == 2) mma(c[j], hi, b[1][2 * j], b[1][2 * j + 1]);
        }
      };
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        unsigned hi[4], lo[4];
        if (m >= kb) {
          ldmatrix4(hi, across(x_at, kXs, m * 16, kb * 16));
          ldmatrix4(lo, across(x_at + kTerm, kXs, m * 16, kb * 16));
          add(dq[m], hi, lo, k);
          ldmatrix4(hi, across(w_at, kXs, m * 16, kb * 16));
          ldmatrix4(lo, across(w_at + kTerm, kXs, m * 16, kb * 16));
          add(dk[m], hi, lo, k);
        }
        if (m <= kb) {
          ldmatrix4_trans(hi, along<kXs>(x_at, kb * 16, m * 16));
          ldmatrix4_trans(lo, along<kXs>(x_at + kTerm, kb * 16, m * 16));
          add(dk[m], hi, lo, q);
          ldmatrix4_trans(hi, along<kXs>(w_at, kb * 16, m * 16));
          ldmatrix4_trans(lo, along<kXs>(w_at + kTerm, kb * 16, m * 16));
          add(dk[m], hi, lo, k);
        }
      }
    }
    // dg: two rows a lane
    if (warp == 0) {
      float db[2], tail[2];  // their terms' errors are far above FP32's
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * lane + e, m = r / 16, n = r / 8;
        float sum = 0.f;
        for (int j = 0; j < 2 * m + 2; ++j) sum += sh.row_part[m * (m + 1) + j][r % 16];
        for (int j = m; j < 4; ++j) sum -= sh.col_part[j * (j + 1) + n][r % 8];
        float v[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 3; ++x)
          for (int j = 0; j < kWarps; ++j) v[x] += sh.dots[x][j][r];
        const float f = own.front[r], b = own.beta[r];
        tail[e] = __fmul_rn(__fmul_rn(own.back[r], b), v[2]);
        db[e] = sum + __fmul_rn(__fmul_rn(p.scale, f), v[0]) - __fmul_rn(__fmul_rn(b, f), v[1]) - tail[e];
      }
      float whole = tail[0] + tail[1];
#pragma unroll
      for (int o = 16; o; o /= 2) whole += __shfl_xor_sync(0xFFFFFFFFu, whole, o);
      float states = 0.f;
      for (int j = 0; j < kWarps; ++j) states += sh.product[j];
      whole += __fmul_rn(own.front[kChunk - 1], states);
      // sums from the chunk's end
      db[0] += db[1];
      float run = db[0];
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const float above = __shfl_down_sync(0xFFFFFFFFu, run, o);
        if (lane + o < 32) run += above;
      }
      const float behind = run - db[0] + whole;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * lane + e;
        if (r < span.rows) g.dg[(span.row + r) * g.lddg + h] = behind + db[e];
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = m * 16 + gr + half * 8;
      if (r >= span.rows) continue;
#pragma unroll
      for (int j = 0; j < N8; ++j) {
        const int c = (warp * N8 + j) * 8 + t2;
        T* q = g.dq + (span.row + r) * g.lddq + kh * p.dk + c;
        T* k = g.dk + (span.row + r) * g.lddk + kh * p.dk + c;
        const auto a = pair_from_f32<T>(make_float2(dq[m][j][2 * half], dq[m][j][2 * half + 1]));
        const auto b = pair_from_f32<T>(make_float2(dk[m][j][2 * half], dk[m][j][2 * half + 1]));
        if (VEC) {
          if (c < p.dk) {
            *reinterpret_cast<typename Pair<T>::type*>(q) = a;
            *reinterpret_cast<typename Pair<T>::type*>(k) = b;
          }
        } else {
          if (c < p.dk) q[0] = a.x, k[0] = b.x;
          if (c + 1 < p.dk) q[1] = a.y, k[1] = b.y;
        }
      }
    }
}

template <typename T, int DK, bool VEC>
cudaError_t grad(const GdeltaRows<T>& p, const GdeltaGrads<T>& g, cudaStream_t stream) {
  auto* kernel = grad_kernel<T, DK, VEC>;
  constexpr int kShared = sizeof(GradShared<DK, Terms<T>::n>);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(static_cast<unsigned>(gdelta_places(p.batch, p.rows)), p.heads_k), kThreads, kShared,
           stream>>>(p, g);
  return cudaGetLastError();
}

}  // namespace

template <typename T>
cudaError_t launch_gdelta_grad(const GdeltaRows<T>& p, const GdeltaGrads<T>& g, cudaStream_t stream) {
  const bool vec = gdelta_aligned(p.q, p.ldq, p.dk) && gdelta_aligned(p.k, p.ldk, p.dk) &&
                   gdelta_aligned(g.dout, g.lddo, p.dv) && gdelta_aligned(g.dq, g.lddq, p.dk) &&
                   gdelta_aligned(g.dk, g.lddk, p.dk);
  if (p.dk <= 64) return vec ? grad<T, 64, true>(p, g, stream) : grad<T, 64, false>(p, g, stream);
  return vec ? grad<T, 128, true>(p, g, stream) : grad<T, 128, false>(p, g, stream);
}
template cudaError_t launch_gdelta_grad(const GdeltaRows<float>&, const GdeltaGrads<float>&, cudaStream_t);
template cudaError_t launch_gdelta_grad(const GdeltaRows<__nv_bfloat16>&,
                                        const GdeltaGrads<__nv_bfloat16>&, cudaStream_t);
template cudaError_t launch_gdelta_grad(const GdeltaRows<__half>&, const GdeltaGrads<__half>&, cudaStream_t);

}  // namespace bsolve
