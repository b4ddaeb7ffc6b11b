// The gated delta rule's backward pass (bs_gdelta_backward_batched): the chain of the states' gradients, from
// the last chunk to the first.
//
// With G the gradient of the state behind a chunk, D the rows' incoming gradients, X = (I + diag(beta) N)^-1
// and the rest as in the forward chain, U the solution's rows and dU the gradient of all their uses,
//   dU = X^T (A^T D + diag(e) K G),     dV = diag(beta) dU,
//   G' = f_last G + (scale diag(f) Q)^T D - (diag(beta f) K)^T dU.
// The forward chain's layout: a warp has 16 columns of G, transposed, in registers, and the same number of
// products. G and dU go to the workspace as operands for gdelta_grad.cu.
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
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int t2 = (lane & 3) * 2, v_stride = St::v_stride(warps), stage_bytes = St::bytes(warps);
  const Place at = place_of(p, slices, scratch);
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
    load_stage<T, DK, VEC>(raw + (c % STAGES) * stage_bytes, p, out.dout, out.lddo,
                           out.prepared + (at.chunk + c) * p.heads_v + at.h, start + c * kChunk,
                           rows_of(c), at.kh, at.h, at.col, v_stride);
  };
  if (STAGES == 2 && chunks > 0) load(chunks - 1);
  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int n_rows = rows_of(c);
    const int64_t row = start + c * kChunk;
    if (STAGES == 1) load(c);
    if (STAGES == 2 && c > 0) {
      load(c - 1);
      cp_async_wait_group<1>();
    } else {
      cp_async_wait_all();
    }
    __syncthreads();
    if (mine) {
      unsigned char* stage = raw + (c % STAGES) * stage_bytes;
      const unsigned q = smem_addr(stage), k = q + St::kQk;
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
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          unsigned b[4], l[4] = {0, 0, 0, 0};
          ldmatrix4(b, along<STRIDE>(k, n * 16, kb * 16));
          if constexpr (NT == 2) ldmatrix4(l, along<STRIDE>(k + 2 * St::kTerm, n * 16, kb * 16));
          mma_terms<NT>(U[2 * n], hi, lo, b[0], b[1], l[0], l[1]);
          mma_terms<NT>(U[2 * n + 1], hi, lo, b[2], b[3], l[2], l[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(&own.back[n * 8 + t2]);
#pragma unroll
        for (int e = 0; e < 4; ++e) U[n][e] = __fmul_rn(U[n][e], e & 1 ? f.y : f.x);
      }
      // + D^T A
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        float x[2][4];
        read_transposed(x, d, v_stride, 2 * kb);
        unsigned hi[4], lo[4];
        split_operand(hi, lo, x[0], x[1]);
#pragma unroll
        for (int n = 0; n < 2 * kb + 2; ++n) {
          const uint4 b = own.mixing[upper_piece(n / 2, n & 1, kb)][lane];
          mma(U[n], hi, b.x, b.y);
          mma(U[n], hi, b.z, b.w);
          if constexpr (NT == 2) mma(U[n], lo, b.x, b.y);
        }
      }
      // (dU)^T X
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        unsigned hi[4], lo[4];
        split_operand(hi, lo, U[2 * kb], U[2 * kb + 1]);
#pragma unroll
        for (int n = 0; n < 2 * kb + 2; ++n) {
          const uint4 b = own.inverse[upper_piece(n / 2, n & 1, kb)][lane];
          mma_terms<2>(R[n], hi, lo, b.x, b.y, b.z, b.w);
        }
      }
      keep_pieces(kept + NB * 32, R);
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
#pragma unroll
        for (int n = 0; n < NB; n += 2) {
          unsigned b[4], l[4] = {0, 0, 0, 0};
          ldmatrix4_trans(b, across(q, STRIDE, kb * 16, n * 8));
          if constexpr (NT == 2) ldmatrix4_trans(l, across(q + 2 * St::kTerm, STRIDE, kb * 16, n * 8));
          mma_terms<NT>(S[n], hi, lo, b[0], b[1], l[0], l[1]);
          mma_terms<NT>(S[n + 1], hi, lo, b[2], b[3], l[2], l[3]);
          ldmatrix4_trans(b, across(k, STRIDE, kb * 16, n * 8));
          if constexpr (NT == 2) ldmatrix4_trans(l, across(k + 2 * St::kTerm, STRIDE, kb * 16, n * 8));
          mma_terms<NT>(S[n], yhi, ylo, b[0], b[1], l[0], l[1]);
          mma_terms<NT>(S[n + 1], yhi, ylo, b[2], b[3], l[2], l[3]);
        }
      }
      store_transposed<T, VEC>(R, d, v_stride, out.dv + row * out.lddv + at.h * p.dv + col, out.lddv,
                               n_rows, p.dv - col);
    }
    __syncthreads();  // the stage is free
  }
  if (out.dh0) store_state(S, out.dh0 + state, p.dk, p.dv, col);
}

template <typename T, int DK, bool VEC>
cudaError_t chain(const GdeltaRows<T>& p, const Back<T>& out, cudaStream_t stream) {
  constexpr int STAGES = Terms<T>::n == 1 ? 2 : 1;
  const int warps = chain_warps(p), slices = (gdelta_groups(p.dv) + warps - 1) / warps;
  const int shared = STAGES * Stage<T, DK>::bytes(warps);
  auto* kernel = back_kernel<T, DK, VEC, STAGES>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, shared);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(p.batch * p.heads_v * slices), warps * 32, shared, stream>>>(p, out,
                                                                                             slices);
  return cudaGetLastError();
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
