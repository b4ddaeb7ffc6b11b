// The gated delta rule's backward pass (bs_gdelta_backward_batched): the chain of the states' gradients, from
// the last chunk to the first.
//
// With G the gradient of the state behind a chunk, D the rows' incoming gradients, X = (I + diag(beta) N)^-1
// and the rest as in the forward chain, U the solution's rows and dU the gradient of all their uses,
//   dU = X^T (A^T D + diag(e) K G),     dV = diag(beta) dU,
//   G' = f_last G + (scale diag(f) Q)^T D - (diag(beta f) K)^T dU.
// The forward chain's layout: a warp has 16 columns of G, transposed, in registers, and the same number of
// products (8 x 2,048 rows of 16 heads 128 x 128, BF16: 251 us). G and dU go to the workspace as operands for
// gdelta_grad.cu.
#include "gdelta_chain.cuh"
#include "gdelta_grad.cuh"

namespace bsolve {
namespace {

template <typename T>
struct Back {
  const T* dout;
  int64_t lddo;
  T* dv;
  int64_t lddv;
  const float* dhT;
  float* dh0;
  uint4* kept;
  const Prepared* prepared;
};

template <typename T, int DK, bool VEC, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
back_kernel(GdeltaRows<T> p, Back<T> out, int slices) {
  using St = Stage<T, DK>;
  constexpr int NT = Terms<T>::n, NB = DK / 8, STRIDE = St::kStride;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ int64_t scratch[kSortedBatch + 1];
  __shared__ uint64_t full[STAGES];
  __shared__ volatile int failed;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int t2 = (lane & 3) * 2, v_stride = St::v_stride(warps), stage_bytes = St::bytes(warps);
  const Place at = place_of(p, slices, warps * 16, scratch);
  const int64_t start = at.start, end = at.end;
  const int col = at.col + warp * 16;
  const bool mine = col < p.dv;
  const int64_t state = at.head * p.dk * p.dv;
  float S[NB][4];
  load_state(S, out.dhT ? out.dhT + state : nullptr, p.dk, p.dv, col);

  const int64_t chunks = (end - start + kChunk - 1) / kChunk;
  auto rows_of = [&](int64_t c) {
    return static_cast<int>(min(end - start - c * kChunk, static_cast<int64_t>(kChunk)));
  };
  auto load = [&](int64_t c) {
    if constexpr (kBulk<T, VEC>) {
      copy_stage<T, DK>(raw + (c % STAGES) * stage_bytes, &full[c % STAGES], p, out.dout, out.lddo,
                           out.prepared + (at.chunk + c) * p.heads_v + at.h, start + c * kChunk,
                           rows_of(c), at.kh, at.h, at.col, warps * 16, v_stride);
    } else {
      load_stage<T, DK, VEC>(raw + (c % STAGES) * stage_bytes, p, out.dout, out.lddo,
                           out.prepared + (at.chunk + c) * p.heads_v + at.h, start + c * kChunk,
                           rows_of(c), at.kh, at.h, at.col, warps * 16, v_stride,
                             threadIdx.x, blockDim.x);
      cp_async_commit();
    }
  };
  if constexpr (kBulk<T, VEC>) {
    if (threadIdx.x == 0) {
      failed = 0;
      for (int s = 0; s < STAGES; ++s) barrier_init(&full[s], 1);
      barriers_ready();
    }
    if (p.dk != DK || p.dv % (warps * 16) != 0) clear_stages(raw, STAGES * stage_bytes);
    __syncthreads();
  }
  if (STAGES == 2 && chunks > 0) load(chunks - 1);
  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int n_rows = rows_of(c);
    const int64_t row = start + c * kChunk;
    if (STAGES == 1) load(c);
    if (STAGES == 2 && c > 0) {
      load(c - 1);
      if (!kBulk<T, VEC>) cp_async_wait_group<1>();
    } else if (!kBulk<T, VEC>) {
      cp_async_wait_all();
    }
    if constexpr (kBulk<T, VEC>) {
      if (!wait_for(&full[c % STAGES], (chunks - 1 - c) / STAGES & 1, &failed)) poison(S);
    }
    __syncthreads();
    if (mine) {
      unsigned char* stage = raw + (c % STAGES) * stage_bytes;
      const unsigned q = smem_address(stage), k = q + St::kQk;
      T* d = reinterpret_cast<T*>(stage + 2 * St::kQk) + warp * 16;
      const auto& own = *reinterpret_cast<const Prepared*>(stage + 2 * St::kQk +
                                                           kChunk * v_stride * sizeof(T));
      uint4* kept = out.kept + (((at.chunk + c) * p.heads_v + at.h) * gdelta_groups(p.dv) + col / 16) *
                                   (kept_pieces(DK) * 32);
      keep_pieces(kept, S);
      // (K G)^T e
      float U[8][4], R[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) U[n][e] = R[n][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < DK / 16; ++kb) {
        unsigned hi[4], lo[4];
        split_operand(hi, lo, S[2 * kb], S[2 * kb + 1]);
        along_rows<NT, STRIDE>(U, hi, lo, k, 2 * St::kTerm, kb * 16);
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(&own.back[n * 8 + t2]);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[n][e] = __fmul_rn(U[n][e], e & 1 ? f.y : f.x);
      }
      // + D^T A
      four([&](auto at_kb) {
        constexpr int kb = decltype(at_kb)::value;
        float x[2][4];
        read_transposed(x, d, v_stride, 2 * kb);
        unsigned hi[4], lo[4];
        split_operand(hi, lo, x[0], x[1]);
        by_pieces<0, 2 * kb + 2, NT == 1>(U, hi, lo, [&](int n) {
          return own.mixing[upper_piece(n / 2, n & 1, kb)][lane];
        });
      });
      // (dU)^T X
      four([&](auto at_kb) {
        constexpr int kb = decltype(at_kb)::value;
        unsigned hi[4], lo[4];
        split_operand(hi, lo, U[2 * kb], U[2 * kb + 1]);
        by_pieces<0, 2 * kb + 2, false>(R, hi, lo, [&](int n) {
          return own.inverse[upper_piece(n / 2, n & 1, kb)][lane];
        });
      });
      keep_rows(kept + NB * 32, R);
      // G^T = f_last G^T + (D^T scale f) Q - (dU^T beta f) K
      const float whole = own.front[kChunk - 1];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][e] = __fmul_rn(S[n][e], whole);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        float x[2][4], y[2][4];
        read_transposed(x, d, v_stride, 2 * kb);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = (2 * kb + j) * 8 + t2;
          const float2 f = *reinterpret_cast<const float2*>(&own.front[r]);
          const float2 b = *reinterpret_cast<const float2*>(&own.beta[r]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float fe = e & 1 ? f.y : f.x, be = e & 1 ? b.y : b.x;
            x[j][e] = __fmul_rn(x[j][e], __fmul_rn(p.scale, fe));
            R[2 * kb + j][e] = __fmul_rn(R[2 * kb + j][e], be);  // dV from here on
            y[j][e] = __fmul_rn(R[2 * kb + j][e], -fe);
          }
        }
        unsigned hi[4], lo[4], yhi[4], ylo[4];
        split_operand(hi, lo, x[0], x[1]);
        split_operand(yhi, ylo, y[0], y[1]);
        across_rows<NT, NB, STRIDE>(S, hi, lo, q, 2 * St::kTerm, kb * 16);
        across_rows<NT, NB, STRIDE>(S, yhi, ylo, k, 2 * St::kTerm, kb * 16);
      }
      store_transposed<T, VEC>(R, d, v_stride, out.dv + row * out.lddv + at.h * p.dv + col, out.lddv,
                               n_rows, p.dv - col);
    }
    if (kBulk<T, VEC>) writes_before_copies();
    __syncthreads();  // the stage is free
  }
  if (out.dh0) store_state(S, out.dh0 + state, p.dk, p.dv, col);
}

// The same chain by teams of KS warps a group of 16 columns, as in the forward pass.
template <typename T, int DK, bool VEC, int KS>
__global__ void __launch_bounds__(kMaxTeams<T, DK> * 32 * KS + kLoaders<T, DK>, 1)
team_back_kernel(GdeltaRows<T> p, Back<T> out, int slices) {
  using St = Stage<T, DK>;
  constexpr int STAGES = kTeamStages<T, DK>, NT = Terms<T>::n, NB = DK / 8, STRIDE = St::kStride;
  constexpr int OWN = NB / KS, ROWS = Team<KS>::kRows;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ int64_t scratch[kSortedBatch + 1];
  __shared__ uint64_t full[STAGES], empty[STAGES];
  __shared__ volatile int failed;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, t2 = (lane & 3) * 2;
  const int team = warp / KS, teams = (blockDim.x - kLoaders<T, DK>) / (32 * KS);
  const Team<KS> mine{warp % KS};
  const int v_stride = St::v_stride(teams), stage_bytes = St::bytes(teams);
  auto& x = reinterpret_cast<Exchange<DK>*>(raw + STAGES * stage_bytes)[team];
  const Place at = place_of(p, slices, teams * 16, scratch);
  const int64_t start = at.start, end = at.end;
  const int col = at.col + team * 16;
  const bool active = col < p.dv;
  const int64_t state = at.head * p.dk * p.dv;
  const int from = mine.j * OWN * 8;  // the warp's part of dk
  const int64_t chunks = (end - start + kChunk - 1) / kChunk;
  auto rows_of = [&](int64_t c) {
    return static_cast<int>(min(end - start - c * kChunk, static_cast<int64_t>(kChunk)));
  };
  if (threadIdx.x == 0) {
    failed = 0;
    for (int s = 0; s < STAGES; ++s) {
      barrier_init(&full[s], kLoaders<T, DK>);
      barrier_init(&empty[s], teams * KS);
    }
    barriers_ready();
  }
  __syncthreads();
  if (warp >= teams * KS) {
    bring_stages<VEC && NT == 1>(chunks, STAGES, full, empty, &failed, [&](int64_t i, int s) {
      const int64_t c = chunks - 1 - i;
      load_stage<T, DK, VEC>(raw + s * stage_bytes, p, out.dout, out.lddo,
                             out.prepared + (at.chunk + c) * p.heads_v + at.h, start + c * kChunk, rows_of(c),
                             at.kh, at.h, at.col, teams * 16, v_stride, threadIdx.x - teams * KS * 32, kLoaders<T, DK>);
    });
    return;
  }
  float S[OWN][4];
  load_state(S, out.dhT ? out.dhT + state : nullptr, p.dk, p.dv, col, from);

  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int n_rows = rows_of(c);
    const int64_t row = start + c * kChunk;
    if (active)
#pragma unroll
      for (int k = 0; k < OWN / 2; ++k) {
        unsigned hi[4], lo[4];
        split_operand(hi, lo, S[2 * k], S[2 * k + 1]);
        x.state[from / 16 + k][0][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        x.state[from / 16 + k][1][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    const int s = static_cast<int>((chunks - 1 - c) % STAGES);
    if (!wait_for(&full[s], (chunks - 1 - c) / STAGES & 1, &failed)) poison(S);
    team_sync(team, KS * 32);
    if (active) {
      unsigned char* stage = raw + s * stage_bytes;
      const unsigned q = smem_address(stage), k = q + St::kQk;
      T* d = reinterpret_cast<T*>(stage + 2 * St::kQk) + team * 16;
      const auto& own = *reinterpret_cast<const Prepared*>(stage + 2 * St::kQk +
                                                           kChunk * v_stride * sizeof(T));
      uint4* kept = out.kept + (((at.chunk + c) * p.heads_v + at.h) * gdelta_groups(p.dv) + col / 16) *
                                   (kept_pieces(DK) * 32);
      keep_pieces(kept + from / 8 * 32, S);
      // (K G)^T e of the warp's rows
      // the terms of dU apart: each a chain of at most four products
      float U[ROWS][4], R[ROWS][4], V[2][ROWS][4];
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) U[i][e] = R[i][e] = V[0][i][e] = V[1][i][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < DK / 16; ++kb) {
        unsigned hi[4], lo[4], b[ROWS / 2][4];
        get_operand(hi, lo, x.state[kb]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int i = 0; i < ROWS / 2; ++i)
            ldmatrix4(b[i], along_two<STRIDE>(k + t * 2 * St::kTerm, mine.rows(2 * i), mine.rows(2 * i + 1), kb * 16));
#pragma unroll
          for (int i = 0; i < ROWS; ++i) mma(U[i], hi, b[i / 2][(i & 1) * 2], b[i / 2][(i & 1) * 2 + 1]);
          if (t == 0)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) mma(U[i], lo, b[i / 2][(i & 1) * 2], b[i / 2][(i & 1) * 2 + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float2 f = *reinterpret_cast<const float2*>(&own.back[mine.rows(i) * 8 + t2]);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[i][e] = __fmul_rn(U[i][e], e & 1 ? f.y : f.x);
      }
      // + D^T A
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (kb < mine.rows(0) / 2) continue;
        float w[2][4];
        read_transposed(w, d, v_stride, 2 * kb);
        unsigned hi[4], lo[4];
        split_operand(hi, lo, w[0], w[1]);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const int n = mine.rows(i);
          if (kb < n / 2) continue;
          const uint4 b = own.mixing[upper_piece(n / 2, n & 1, kb)][lane];
          mma(U[i], hi, b.x, b.y);
          mma(V[0][i], hi, b.z, b.w);
          if constexpr (NT == 2) mma(V[1][i], lo, b.x, b.y);
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          U[i][e] = __fadd_rn(U[i][e], __fadd_rn(V[0][i][e], V[1][i][e]));
          V[0][i][e] = V[1][i][e] = 0.f;
        }
      // the rows' parts of the last products' operands: dU^T so far, and D^T scale f
#pragma unroll
      for (int i = 0; i < ROWS; i += 2) {
        float w[2][4];
        read_two(w[0], w[1], d, v_stride, mine.rows(i), mine.rows(i + 1));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = mine.rows(i + h);
          const float2 f = *reinterpret_cast<const float2*>(&own.front[n * 8 + t2]);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[h][e] = __fmul_rn(w[h][e], __fmul_rn(p.scale, e & 1 ? f.y : f.x));
          put_half(x.first, n, U[i + h]);
          put_half(x.second, n, w[h]);
        }
      }
      team_sync(team, KS * 32);  // d is read; the rows' parts are there
      // (dU)^T X
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (kb < mine.rows(0) / 2) continue;
        unsigned hi[4], lo[4];
        get_operand(hi, lo, x.first[kb]);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const int n = mine.rows(i);
          if (kb < n / 2) continue;
          const uint4 b = own.inverse[upper_piece(n / 2, n & 1, kb)][lane];
          mma(R[i], hi, b.x, b.y);
          mma(V[0][i], lo, b.x, b.y);
          mma(V[1][i], hi, b.z, b.w);
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int n = mine.rows(i);
#pragma unroll
        for (int e = 0; e < 4; ++e) R[i][e] = __fadd_rn(R[i][e], __fadd_rn(V[0][i][e], V[1][i][e]));
        keep_row_group(kept + NB * 32, n, R[i]);
        const float2 f = *reinterpret_cast<const float2*>(&own.front[n * 8 + t2]);
        const float2 b = *reinterpret_cast<const float2*>(&own.beta[n * 8 + t2]);
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          R[i][e] = __fmul_rn(R[i][e], e & 1 ? b.y : b.x);  // dV from here on
          y[e] = __fmul_rn(R[i][e], e & 1 ? -f.y : -f.x);
        }
        put_half(x.third, n, y);
      }
#pragma unroll
      for (int i = 0; i < ROWS; i += 2)
        store_two<T, VEC>(R[i], R[i + 1], d, v_stride, mine.rows(i), mine.rows(i + 1),
                          out.dv + row * out.lddv + at.h * p.dv + col, out.lddv, n_rows, p.dv - col);
      team_sync(team, KS * 32);
      // G^T = f_last G^T + (D^T scale f) Q - (dU^T beta f) K
      const float whole = own.front[kChunk - 1];
#pragma unroll
      for (int n = 0; n < OWN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][e] = __fmul_rn(S[n][e], whole);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        unsigned hi[4], lo[4];
        get_operand(hi, lo, x.second[kb]);
        part_across<NT, OWN, STRIDE>(S, hi, lo, q, 2 * St::kTerm, kb * 16, from);
        get_operand(hi, lo, x.third[kb]);
        part_across<NT, OWN, STRIDE>(S, hi, lo, k, 2 * St::kTerm, kb * 16, from);
      }
    }
    __syncwarp();
    if (lane == 0) barrier_arrive(&empty[s]);
  }
  if (out.dh0 && active) store_state(S, out.dh0 + state, p.dk, p.dv, col, from);
}

template <typename T, int DK, bool VEC>
cudaError_t chain(const GdeltaRows<T>& p, const Back<T>& out, cudaStream_t stream) {
  return launch_chain<T, DK, VEC>(team_back_kernel<T, DK, VEC, 4>, back_kernel<T, DK, VEC, kWarpStages<T>>, p, out,
                                  stream);
}

}  // namespace

template <typename T>
cudaError_t launch_gdelta_backward(const GdeltaRows<T>& p, const void* tape, const T* dout,
                                   int64_t lddo, const float* dhT, T* dq, int64_t lddq, T* dk,
                                   int64_t lddk, T* dv, int64_t lddv, float* dg, int64_t lddg,
                                   float* dbeta, int64_t lddbeta, float* dh0, void* work,
                                   cudaStream_t stream) {
  auto* prepared = static_cast<Prepared*>(work);
  auto* kept = reinterpret_cast<uint4*>(static_cast<char*>(work) +
                                        gdelta_workspace(p.heads_v, p.batch, p.rows));
  cudaError_t e = launch_gdelta_prepare(p, true, prepared, stream);
  if (e != cudaSuccess) return e;
  const Back<T> out{dout, lddo, dv, lddv, dhT, dh0, kept, prepared};
  const bool vec = gdelta_aligned(p.q, p.ldq, p.dk) && gdelta_aligned(p.k, p.ldk, p.dk) &&
                   gdelta_aligned(dout, lddo, p.dv) && gdelta_aligned(dv, lddv, p.dv);
  if (p.dk <= 64)
    e = vec ? chain<T, 64, true>(p, out, stream) : chain<T, 64, false>(p, out, stream);
  else
    e = vec ? chain<T, 128, true>(p, out, stream) : chain<T, 128, false>(p, out, stream);
  if (e != cudaSuccess) return e;
  return launch_gdelta_grad(p, GdeltaGrads<T>{dout, lddo, dq, lddq, dk, lddk, dg, lddg, dbeta, lddbeta,
                                              static_cast<const uint4*>(tape), kept, prepared},
                            stream);
}
#define BSOLVE_GDELTA_BACKWARD(T)                                                                    \
  template cudaError_t launch_gdelta_backward(const GdeltaRows<T>&, const void*, const T*, int64_t,  \
                                              const float*, T*, int64_t, T*, int64_t, T*, int64_t,   \
                                              float*, int64_t, float*, int64_t, float*, void*,       \
                                              cudaStream_t);
BSOLVE_GDELTA_BACKWARD(float)
BSOLVE_GDELTA_BACKWARD(__nv_bfloat16)
BSOLVE_GDELTA_BACKWARD(__half)

size_t gdelta_backward_workspace(int heads_v, int dk, int dv, int64_t batch, int64_t rows) {
  return gdelta_workspace(heads_v, batch, rows) + kept_bytes(heads_v, dk, dv, batch, rows);
}

}  // namespace bsolve
