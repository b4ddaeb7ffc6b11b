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
// shared memory for the block's warps. Bound by the rate of mma.sync and by the chain:
// one block per (sequence, head) has 1 to 8 warps.
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
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int t2 = (lane & 3) * 2, v_stride = St::v_stride(warps), stage_bytes = St::bytes(warps);
  const Place at = place_of(p, slices, scratch);
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
    load_stage<T, DK, VEC>(raw + (c % STAGES) * stage_bytes, p, p.v, p.ldv,
                           out.prepared + (at.chunk + c) * p.heads_v + at.h, start + c * kChunk,
                           rows_of(c), at.kh, at.h, at.col, v_stride);
  };
  if (STAGES == 2 && chunks > 0) load(0);
  for (int64_t c = 0; c < chunks; ++c) {
    const int n_rows = rows_of(c);
    const int64_t row = start + c * kChunk;
    if (STAGES == 1) load(c);
    if (STAGES == 2 && c + 1 < chunks) {
      load(c + 1);
      cp_async_wait_group<1>();
    } else {
      cp_async_wait_all();
    }
    __syncthreads();
    if (mine) {
      unsigned char* stage = raw + (c % STAGES) * stage_bytes;
      const unsigned q = smem_addr(stage), k = q + St::kQk;
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
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          unsigned b[4], l[4] = {0, 0, 0, 0};
          ldmatrix4(b, along<STRIDE>(k, n * 16, kb * 16));
          if constexpr (NT == 2) ldmatrix4(l, along<STRIDE>(k + 2 * St::kTerm, n * 16, kb * 16));
          mma_terms<NT>(R[2 * n], hi, lo, b[0], b[1], l[0], l[1]);
          mma_terms<NT>(R[2 * n + 1], hi, lo, b[2], b[3], l[2], l[3]);
          ldmatrix4(b, along<STRIDE>(q, n * 16, kb * 16));
          if constexpr (NT == 2) ldmatrix4(l, along<STRIDE>(q + 2 * St::kTerm, n * 16, kb * 16));
          mma_terms<NT>(O[2 * n], hi, lo, b[0], b[1], l[0], l[1]);
          mma_terms<NT>(O[2 * n + 1], hi, lo, b[2], b[3], l[2], l[3]);
        }
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
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        unsigned hi[4], lo[4];
        split_operand(hi, lo, R[2 * kb], R[2 * kb + 1]);
#pragma unroll
        for (int n = 2 * kb; n < 8; ++n) {
          const uint4 b = own.inverse[lower_piece(n / 2, n & 1, kb)][lane];
          mma_terms<2>(U[n], hi, lo, b.x, b.y, b.z, b.w);
        }
      }
      if (kept) keep_pieces(kept + NB * 32, U);
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
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        unsigned hi[4], lo[4];
        split_operand(hi, lo, U[2 * kb], U[2 * kb + 1]);
#pragma unroll
        for (int n = 2 * kb; n < 8; ++n) {
          const uint4 b = own.mixing[lower_piece(n / 2, n & 1, kb)][lane];
          mma_terms<2>(O[n], hi, lo, b.x, b.y, b.z, b.w);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = *reinterpret_cast<const float2*>(&own.back[(2 * kb + j) * 8 + t2]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            U[2 * kb + j][e] = __fmul_rn(U[2 * kb + j][e], e & 1 ? f.y : f.x);
        }
        split_operand(hi, lo, U[2 * kb], U[2 * kb + 1]);
#pragma unroll
        for (int n = 0; n < NB; n += 2) {
          unsigned b[4], l[4] = {0, 0, 0, 0};
          ldmatrix4_trans(b, across(k, STRIDE, kb * 16, n * 8));
          if constexpr (NT == 2) ldmatrix4_trans(l, across(k + 2 * St::kTerm, STRIDE, kb * 16, n * 8));
          mma_terms<NT>(S[n], hi, lo, b[0], b[1], l[0], l[1]);
          mma_terms<NT>(S[n + 1], hi, lo, b[2], b[3], l[2], l[3]);
        }
      }
      store_transposed<T, VEC>(O, v, v_stride, out.o + row * out.ldo + at.h * p.dv + col, out.ldo, n_rows,
                               p.dv - col);
    }
    __syncthreads();  // the stage is free
  }
  if (out.hT) store_state(S, out.hT + state, p.dk, p.dv, col);
}

template <typename T, int DK, bool VEC>
cudaError_t chain(const GdeltaRows<T>& p, const ChainOut<T>& out, cudaStream_t stream) {
  constexpr int STAGES = Terms<T>::n == 1 ? 2 : 1;
  const int warps = chain_warps(p), slices = (gdelta_groups(p.dv) + warps - 1) / warps;
  const int shared = STAGES * Stage<T, DK>::bytes(warps);
  auto* kernel = chain_kernel<T, DK, VEC, STAGES>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(p.batch * p.heads_v * slices), warps * 32, shared, stream>>>(p, out,
                                                                                             slices);
  return cudaGetLastError();
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
