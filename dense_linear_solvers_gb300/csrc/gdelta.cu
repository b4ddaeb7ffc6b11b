// The gated delta rule over whole sequences (bs_gdelta_batched): the chain of states from chunk to chunk.
//
// With S the state in front of a chunk (dk x dv), and the inverse X, the mixing matrix A, the
// decays f (from the chunk's start) and e (to its end) that gdelta_prep.cu has made,
//   M = X (V - diag(f) K S),   U = diag(beta) M,
//   O = scale diag(f) Q S + A U,        S' = f_last S + (diag(e) K)^T U.
// Columns of S are independent of each other, so that a warp keeps 16 of them, transposed (16 x dk, the sums of
// its products), in registers from the first chunk to the last, and nothing is exchanged between warps:
// the layout of a product's result is that of the next one's first operand, so that S^T, M^T and U^T go
// from one product into the next by way of their split into two BF16 terms. K, Q and V come through
// shared memory for the block's warps. Bound by the chain: few warps (255 registers a thread), each waiting for its
// own products. 8 x 2,048 rows of 16 heads 128 x 128, BF16: 279 us, the tensor pipe busy for 45%, schedulers issue on
// 28% of the cycles. Where there are too few columns for that many warps, teams of four warps take 16 columns (see
// gdelta_chain.cuh): one sequence of 32,768 rows of 16 heads, the whole call, 4.34 to 0.94 ms.
#include "gdelta_chain.cuh"

namespace bsolve {
namespace {

template <typename T>
struct ChainOut {
  T* o;
  int64_t ldo;
  const float* h0;
  float* hT;
  uint4* tape;
  const Prepared* prepared;
};

template <typename T, int DK, bool VEC, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
chain_kernel(GdeltaRows<T> p, ChainOut<T> out, int slices) {
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
  const bool mine = col < p.dv;  // this warp has columns
  const int64_t state = at.head * p.dk * p.dv;
  float S[NB][4];
  load_state(S, out.h0 ? out.h0 + state : nullptr, p.dk, p.dv, col);

  const int64_t chunks = (end - start + kChunk - 1) / kChunk;
  auto rows_of = [&](int64_t c) {
    return static_cast<int>(min(end - start - c * kChunk, static_cast<int64_t>(kChunk)));
  };
  auto load = [&](int64_t c) {
    if constexpr (kBulk<T, VEC>) {
      copy_stage<T, DK>(raw + (c % STAGES) * stage_bytes, &full[c % STAGES], p, p.v, p.ldv,
                           out.prepared + (at.chunk + c) * p.heads_v + at.h, start + c * kChunk,
                           rows_of(c), at.kh, at.h, at.col, warps * 16, v_stride);
    } else {
      load_stage<T, DK, VEC>(raw + (c % STAGES) * stage_bytes, p, p.v, p.ldv,
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
  if (STAGES == 2 && chunks > 0) load(0);
  for (int64_t c = 0; c < chunks; ++c) {
    const int n_rows = rows_of(c);
    const int64_t row = start + c * kChunk;
    if (STAGES == 1) load(c);
    if (STAGES == 2 && c + 1 < chunks) {
      load(c + 1);
      if (!kBulk<T, VEC>) cp_async_wait_group<1>();
    } else if (!kBulk<T, VEC>) {
      cp_async_wait_all();
    }
    if constexpr (kBulk<T, VEC>) {
      if (!wait_for(&full[c % STAGES], c / STAGES & 1, &failed)) poison(S);
    }
    __syncthreads();
    if (mine) {
      unsigned char* stage = raw + (c % STAGES) * stage_bytes;
      const unsigned q = smem_address(stage), k = q + St::kQk;
      T* v = reinterpret_cast<T*>(stage + 2 * St::kQk) + warp * 16;
      const auto& own = *reinterpret_cast<const Prepared*>(stage + 2 * St::kQk +
                                                           kChunk * v_stride * sizeof(T));
      uint4* kept = out.tape ? out.tape + (((at.chunk + c) * p.heads_v + at.h) * gdelta_groups(p.dv) +
                                           col / 16) * (kept_pieces(DK) * 32)
                             : nullptr;
      if (kept) keep_pieces(kept, S);
      // (K S)^T and (Q S)^T
      float R[8][4], O[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) R[n][e] = O[n][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < DK / 16; ++kb) {
        unsigned hi[4], lo[4];
        split_operand(hi, lo, S[2 * kb], S[2 * kb + 1]);
        along_rows<NT, STRIDE>(R, hi, lo, k, 2 * St::kTerm, kb * 16);
        along_rows<NT, STRIDE>(O, hi, lo, q, 2 * St::kTerm, kb * 16);
      }
      // R^T = V^T - (K S)^T f, O^T = scale f (Q S)^T
#pragma unroll
      for (int n = 0; n < 8; n += 2) {
        float x[2][4];
        read_transposed(x, v, v_stride, n);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = *reinterpret_cast<const float2*>(&own.front[(n + j) * 8 + t2]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float fe = e & 1 ? f.y : f.x;
            R[n + j][e] = __fmaf_rn(-fe, R[n + j][e], x[j][e]);
            O[n + j][e] = __fmul_rn(O[n + j][e], __fmul_rn(p.scale, fe));
          }
        }
      }
      // M^T = R^T X^T, U^T = M^T beta
      float U[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) U[n][e] = 0.f;
      four([&](auto at_kb) {
        constexpr int kb = decltype(at_kb)::value;
        unsigned hi[4], lo[4];
        split_operand(hi, lo, R[2 * kb], R[2 * kb + 1]);
        by_pieces<2 * kb, 8, false>(U, hi, lo, [&](int n) {
          return own.inverse[lower_piece(n / 2, n & 1, kb)][lane];
        });
      });
      if (kept) keep_rows(kept + NB * 32, U);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 b = *reinterpret_cast<const float2*>(&own.beta[n * 8 + t2]);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[n][e] = __fmul_rn(U[n][e], e & 1 ? b.y : b.x);
      }
      // O^T += U^T A^T; then S^T = f_last S^T + (U^T e) K
      const float whole = own.front[kChunk - 1];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][e] = __fmul_rn(S[n][e], whole);
      four([&](auto at_kb) {
        constexpr int kb = decltype(at_kb)::value;
        unsigned hi[4], lo[4];
        split_operand(hi, lo, U[2 * kb], U[2 * kb + 1]);
        by_pieces<2 * kb, 8, false>(O, hi, lo, [&](int n) {
          return own.mixing[lower_piece(n / 2, n & 1, kb)][lane];
        });
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = *reinterpret_cast<const float2*>(&own.back[(2 * kb + j) * 8 + t2]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            U[2 * kb + j][e] = __fmul_rn(U[2 * kb + j][e], e & 1 ? f.y : f.x);
        }
        split_operand(hi, lo, U[2 * kb], U[2 * kb + 1]);
        across_rows<NT, NB, STRIDE>(S, hi, lo, k, 2 * St::kTerm, kb * 16);
      });
      store_transposed<T, VEC>(O, v, v_stride, out.o + row * out.ldo + at.h * p.dv + col, out.ldo, n_rows,
                               p.dv - col);
    }
    if (kBulk<T, VEC>) writes_before_copies();
    __syncthreads();  // the stage is free
  }
  if (out.hT) store_state(S, out.hT + state, p.dk, p.dv, col);
}

// The same chain by teams of KS warps a group of 16 columns, `teams` groups a block.
template <typename T, int DK, bool VEC, int KS>
__global__ void __launch_bounds__(kMaxTeams<T, DK> * 32 * KS + kLoaders<T, DK>, 1)
team_kernel(GdeltaRows<T> p, ChainOut<T> out, int slices) {
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
    bring_stages<VEC && NT == 1>(chunks, STAGES, full, empty, &failed, [&](int64_t c, int s) {
      load_stage<T, DK, VEC>(raw + s * stage_bytes, p, p.v, p.ldv,
                             out.prepared + (at.chunk + c) * p.heads_v + at.h, start + c * kChunk, rows_of(c),
                             at.kh, at.h, at.col, teams * 16, v_stride, threadIdx.x - teams * KS * 32, kLoaders<T, DK>);
    });
    return;
  }
  float S[OWN][4];
  load_state(S, out.h0 ? out.h0 + state : nullptr, p.dk, p.dv, col, from);

  for (int64_t c = 0; c < chunks; ++c) {
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
    const int s = static_cast<int>(c % STAGES);
    if (!wait_for(&full[s], c / STAGES & 1, &failed)) poison(S);
    team_sync(team, KS * 32);
    if (active) {
      unsigned char* stage = raw + s * stage_bytes;
      const unsigned q = smem_address(stage), k = q + St::kQk;
      T* v = reinterpret_cast<T*>(stage + 2 * St::kQk) + team * 16;
      const auto& own = *reinterpret_cast<const Prepared*>(stage + 2 * St::kQk +
                                                           kChunk * v_stride * sizeof(T));
      uint4* kept = out.tape ? out.tape + (((at.chunk + c) * p.heads_v + at.h) * gdelta_groups(p.dv) +
                                           col / 16) * (kept_pieces(DK) * 32)
                             : nullptr;
      if (kept) keep_pieces(kept + from / 8 * 32, S);
      // (K S)^T and (Q S)^T of the warp's rows
      // the terms of U and O apart: each a chain of at most four products
      float R[ROWS][4], O[ROWS][4], U[ROWS][4], V[2][ROWS][4];
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) R[i][e] = O[i][e] = U[i][e] = V[0][i][e] = V[1][i][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < DK / 16; ++kb) {
        unsigned hi[4], lo[4], b[ROWS / 2][4], d[ROWS / 2][4];
        get_operand(hi, lo, x.state[kb]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int i = 0; i < ROWS / 2; ++i) {
            ldmatrix4(b[i], along_two<STRIDE>(k + t * 2 * St::kTerm, mine.rows(2 * i), mine.rows(2 * i + 1), kb * 16));
            ldmatrix4(d[i], along_two<STRIDE>(q + t * 2 * St::kTerm, mine.rows(2 * i), mine.rows(2 * i + 1), kb * 16));
          }
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            mma(R[i], hi, b[i / 2][(i & 1) * 2], b[i / 2][(i & 1) * 2 + 1]);
            mma(O[i], hi, d[i / 2][(i & 1) * 2], d[i / 2][(i & 1) * 2 + 1]);
          }
          if (t == 0)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
              mma(R[i], lo, b[i / 2][(i & 1) * 2], b[i / 2][(i & 1) * 2 + 1]);
              mma(O[i], lo, d[i / 2][(i & 1) * 2], d[i / 2][(i & 1) * 2 + 1]);
            }
        }
      }
      // R^T = V^T - (K S)^T f, O^T = scale f (Q S)^T
#pragma unroll
      for (int i = 0; i < ROWS; i += 2) {
        float w[2][4];
        read_two(w[0], w[1], v, v_stride, mine.rows(i), mine.rows(i + 1));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 f = *reinterpret_cast<const float2*>(&own.front[mine.rows(i + h) * 8 + t2]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float fe = e & 1 ? f.y : f.x;
            R[i + h][e] = __fmaf_rn(-fe, R[i + h][e], w[h][e]);
            O[i + h][e] = __fmul_rn(O[i + h][e], __fmul_rn(p.scale, fe));
          }
          put_half(x.first, mine.rows(i + h), R[i + h]);
        }
      }
      team_sync(team, KS * 32);
      // M^T = R^T X^T, U^T = M^T beta
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (kb > mine.rows(ROWS - 1) / 2) break;
        unsigned hi[4], lo[4];
        get_operand(hi, lo, x.first[kb]);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const int n = mine.rows(i);
          if (kb > n / 2) continue;
          const uint4 b = own.inverse[lower_piece(n / 2, n & 1, kb)][lane];
          mma(U[i], hi, b.x, b.y);
          mma(V[0][i], lo, b.x, b.y);
          mma(V[1][i], hi, b.z, b.w);
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int n = mine.rows(i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          U[i][e] = __fadd_rn(U[i][e], __fadd_rn(V[0][i][e], V[1][i][e]));
          V[0][i][e] = V[1][i][e] = 0.f;
        }
        if (kept) keep_row_group(kept + NB * 32, n, U[i]);
        const float2 b = *reinterpret_cast<const float2*>(&own.beta[n * 8 + t2]);
        const float2 f = *reinterpret_cast<const float2*>(&own.back[n * 8 + t2]);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[i][e] = __fmul_rn(U[i][e], e & 1 ? b.y : b.x);
        put_half(x.second, n, U[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[i][e] = __fmul_rn(U[i][e], e & 1 ? f.y : f.x);
        put_half(x.third, n, U[i]);
      }
      team_sync(team, KS * 32);
      // S^T = f_last S^T + (U^T e) K; O^T += U^T A^T
      const float whole = own.front[kChunk - 1];
#pragma unroll
      for (int n = 0; n < OWN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][e] = __fmul_rn(S[n][e], whole);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        unsigned hi[4], lo[4];
        get_operand(hi, lo, x.third[kb]);
        part_across<NT, OWN, STRIDE>(S, hi, lo, k, 2 * St::kTerm, kb * 16, from);
      }
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        if (kb > mine.rows(ROWS - 1) / 2) break;
        unsigned hi[4], lo[4];
        get_operand(hi, lo, x.second[kb]);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          const int n = mine.rows(i);
          if (kb > n / 2) continue;
          const uint4 b = own.mixing[lower_piece(n / 2, n & 1, kb)][lane];
          mma(O[i], hi, b.x, b.y);
          mma(V[0][i], lo, b.x, b.y);
          mma(V[1][i], hi, b.z, b.w);
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[i][e] = __fadd_rn(O[i][e], __fadd_rn(V[0][i][e], V[1][i][e]));
#pragma unroll
      for (int i = 0; i < ROWS; i += 2)
        store_two<T, VEC>(O[i], O[i + 1], v, v_stride, mine.rows(i), mine.rows(i + 1),
                          out.o + row * out.ldo + at.h * p.dv + col, out.ldo, n_rows, p.dv - col);
    }
    __syncwarp();
    if (lane == 0) barrier_arrive(&empty[s]);
  }
  if (out.hT && active) store_state(S, out.hT + state, p.dk, p.dv, col, from);
}

template <typename T, int DK, bool VEC>
cudaError_t chain(const GdeltaRows<T>& p, const ChainOut<T>& out, cudaStream_t stream) {
  return launch_chain<T, DK, VEC>(team_kernel<T, DK, VEC, 4>, chain_kernel<T, DK, VEC, kWarpStages<T>>, p, out,
                                  stream);
}

}  // namespace

template <typename T>
cudaError_t launch_gdelta(const GdeltaRows<T>& p, const float* h0, T* o, int64_t ldo, float* hT,
                          void* tape, void* work, cudaStream_t stream) {
  const cudaError_t e = launch_gdelta_prepare(p, false, static_cast<Prepared*>(work), stream);
  if (e != cudaSuccess) return e;
  const ChainOut<T> out{o, ldo, h0, hT, static_cast<uint4*>(tape), static_cast<const Prepared*>(work)};
  const bool vec = gdelta_aligned(p.q, p.ldq, p.dk) && gdelta_aligned(p.k, p.ldk, p.dk) &&
                   gdelta_aligned(p.v, p.ldv, p.dv) && gdelta_aligned(o, ldo, p.dv);
  if (p.dk <= 64)
    return vec ? chain<T, 64, true>(p, out, stream) : chain<T, 64, false>(p, out, stream);
  return vec ? chain<T, 128, true>(p, out, stream) : chain<T, 128, false>(p, out, stream);
}
template cudaError_t launch_gdelta(const GdeltaRows<float>&, const float*, float*, int64_t, float*,
                                   void*, void*, cudaStream_t);
template cudaError_t launch_gdelta(const GdeltaRows<__nv_bfloat16>&, const float*, __nv_bfloat16*,
                                   int64_t, float*, void*, void*, cudaStream_t);
template cudaError_t launch_gdelta(const GdeltaRows<__half>&, const float*, __half*, int64_t, float*,
                                   void*, void*, cudaStream_t);

size_t gdelta_workspace(int heads_v, int64_t batch, int64_t rows) {
  return gdelta_places(batch, rows) * heads_v * sizeof(Prepared);
}

size_t gdelta_tape(int heads_v, int dk, int dv, int64_t batch, int64_t rows) {
  return kept_bytes(heads_v, dk, dv, batch, rows);
}

}  // namespace bsolve
