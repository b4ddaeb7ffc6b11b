// The gated delta rule over whole sequences (bs_gdelta_batched): the chain of states from chunk to chunk.
//
// With S the state in front of a chunk (dk x dv), and the inverse X, the mixing matrix A, the
// decays f (from the chunk's start) and e (to its end) that gdelta_prep.cu has made,
//   R = diag(beta) (V - diag(f) K S),   U = X R,
//   O = scale diag(f) Q S + A U,        S' = f_last S + (diag(e) K)^T U.
// Columns of S are independent of each other, so that a warp keeps 16 of them, transposed (16 x dk, the sums of
// its products), in registers from the first chunk to the last, and nothing is exchanged between warps:
// the layout of a product's result is that of the next one's first operand, so that S^T, R^T and U^T go
// from one product into the next by way of their split into two BF16 terms. K, Q and V come through
// shared memory for the block's warps. Bound by the rate of mma.sync and by the chain:
// one block per (sequence, head) has 1 to 8 warps.
#include "gdelta_tile.cuh"
#include "grec_order.cuh"

namespace bsolve {
namespace {

constexpr int kMaxWarps = 8;

// Tiles of one stage for a block of `warps` warps: q, k as terms, v as stored, the prepared chunk.
template <typename T, int DK>
struct Stage {
  static constexpr int kStride = DK + 8;
  static constexpr int kTerm = kChunk * kStride;                 // BF16 elements
  static constexpr int kQk = Terms<T>::n * kTerm * 2;            // bytes of q or k
  __host__ __device__ static constexpr int v_stride(int warps) { return warps * 16 + 16 / static_cast<int>(sizeof(T)); }
  __host__ __device__ static constexpr int bytes(int warps) {
    return 2 * kQk + kChunk * v_stride(warps) * static_cast<int>(sizeof(T)) +
           static_cast<int>(sizeof(Prepared));
  }
};

template <typename T>
struct ChainOut {
  T* o;
  int64_t ldo;
  const float* h0;
  float* hT;
  uint4* tape;
  const Prepared* prepared;
};

template <typename T, int DK, bool VEC>
__device__ __forceinline__ void load_stage(unsigned char* stage, const GdeltaRows<T>& p,
                                           const Prepared* prepared, int64_t row, int n, int kh, int h,
                                           int col, int v_stride) {
  using S = Stage<T, DK>;
  auto* q = reinterpret_cast<__nv_bfloat16*>(stage);
  auto* k = reinterpret_cast<__nv_bfloat16*>(stage + S::kQk);
  T* v = reinterpret_cast<T*>(stage + 2 * S::kQk);
  auto* own = reinterpret_cast<uint4*>(stage + 2 * S::kQk + kChunk * v_stride * sizeof(T));
  load_terms<T, DK, S::kStride, VEC>(q, p.q + row * p.ldq + kh * p.dk, p.ldq, n, p.dk);
  load_terms<T, DK, S::kStride, VEC>(k, p.k + row * p.ldk + kh * p.dk, p.ldk, n, p.dk);
  const int width = min(p.dv - col, static_cast<int>(blockDim.x) / 2);
  load_rows<T, VEC>(v, v_stride, blockDim.x / 2, p.v + row * p.ldv + h * p.dv + col, p.ldv, n, width);
  for (int j = threadIdx.x; j < static_cast<int>(sizeof(Prepared) / 16); j += blockDim.x)
    cp_async_16(own + j, reinterpret_cast<const uint4*>(prepared) + j, 16);
  cp_async_commit();
}

// c += a b over one 16-deep piece: a in two terms, b in NB.
template <int NB>
__device__ __forceinline__ void mma_terms(float (&c)[4], const unsigned (&hi)[4],
                                          const unsigned (&lo)[4], unsigned b0, unsigned b1,
                                          unsigned l0, unsigned l1) {
  mma(c, hi, b0, b1);
  mma(c, lo, b0, b1);
  if constexpr (NB == 2) mma(c, hi, l0, l1);
}

template <typename T, int DK, bool VEC, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
chain_kernel(GdeltaRows<T> p, ChainOut<T> out, int slices) {
  using St = Stage<T, DK>;
  constexpr int NT = Terms<T>::n, NB = DK / 8, STRIDE = St::kStride;
  extern __shared__ __align__(16) unsigned char raw[];
  __shared__ int64_t scratch[kSortedBatch + 1];
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int g = lane / 4, t2 = (lane & 3) * 2;
  const int v_stride = St::v_stride(warps), stage_bytes = St::bytes(warps);

  const int64_t part = static_cast<int64_t>(p.heads_v) * slices;
  int64_t s = blockIdx.x / part;
  const int rest = static_cast<int>(blockIdx.x % part), h = rest / slices, slice = rest % slices;
  if (p.offsets && p.batch > 1 && p.batch <= min(kSortedBatch, static_cast<int>(blockDim.x)))
    s = nth_longest(p.offsets, static_cast<int>(p.batch), static_cast<int>(s), scratch);
  int64_t start, end;
  sequence_rows(p, s, &start, &end);
  const int kh = h / (p.heads_v / p.heads_k);
  const int block_col = slice * warps * 16, col = block_col + warp * 16;
  const int64_t place = start / kChunk + s, head = s * p.heads_v + h;
  const bool mine = col < p.dv;  // this warp has columns

  // S^T: rows g and g + 8 of the warp's columns, elements 8 n + t2, + 1 of dk
  float S[NB][4];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col + g + (e / 2) * 8, d = n * 8 + t2 + (e & 1);
      S[n][e] = out.h0 && c < p.dv && d < p.dk
                    ? out.h0[(head * p.dk + d) * p.dv + c] : 0.f;
    }

  const int64_t chunks = (end - start + kChunk - 1) / kChunk;
  auto rows_of = [&](int64_t c) {
    return static_cast<int>(min(end - start - c * kChunk, static_cast<int64_t>(kChunk)));
  };
  auto load = [&](int64_t c) {
    load_stage<T, DK, VEC>(raw + (c % STAGES) * stage_bytes, p,
                           out.prepared + (place + c) * p.heads_v + h, start + c * kChunk, rows_of(c),
                           kh, h, block_col, v_stride);
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
      T* v = reinterpret_cast<T*>(stage + 2 * St::kQk);
      const auto& own = *reinterpret_cast<const Prepared*>(stage + 2 * St::kQk +
                                                           kChunk * v_stride * sizeof(T));
      if (out.tape) {
        // the state as second operand of products over dv (rows of S): 8 x 8 blocks transposed
        uint4* at = out.tape + (((place + c) * p.heads_v + h) * ((p.dv + 15) / 16) + col / 16) *
                                   (NB * 32) + lane;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const Split a = split(S[n][0], S[n][1]), b = split(S[n][2], S[n][3]);
          at[n * 32] = make_uint4(transposed(a.hi), transposed(b.hi), transposed(a.lo), transposed(b.lo));
        }
      }
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
      // R^T = (V^T - (K S)^T f) beta, O^T = scale f (Q S)^T
#pragma unroll
      for (int n = 0; n < 8; n += 2) {
        float x[2][4];
        if constexpr (sizeof(T) == 2) {
          unsigned w[4];
          const int l7 = lane & 7;
          ldmatrix4_trans(w, smem_addr(v + (n * 8 + l7 + ((lane & 16) >> 1)) * v_stride + warp * 16 +
                                       (lane & 8)));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = to_f32(*reinterpret_cast<const typename Pair<T>::type*>(&w[j]));
            x[j / 2][(j & 1) * 2] = f.x;
            x[j / 2][(j & 1) * 2 + 1] = f.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[j][e] = to_f32(v[((n + j) * 8 + t2 + (e & 1)) * v_stride + warp * 16 + g + (e / 2) * 8]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f = *reinterpret_cast<const float2*>(&own.front[(n + j) * 8 + t2]);
          const float2 b = *reinterpret_cast<const float2*>(&own.beta[(n + j) * 8 + t2]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float fe = e & 1 ? f.y : f.x, be = e & 1 ? b.y : b.x;
            R[n + j][e] = __fmul_rn(be, __fmaf_rn(-fe, R[n + j][e], x[j][e]));
            O[n + j][e] = __fmul_rn(O[n + j][e], __fmul_rn(p.scale, fe));
          }
        }
      }
      // U^T = R^T X^T
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
          const uint4 b = own.inverse[lower_piece(n, kb)][lane];
          mma_terms<2>(U[n], hi, lo, b.x, b.y, b.z, b.w);
        }
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
          const uint4 b = own.mixing[lower_piece(n, kb)][lane];
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
      // O through the warp's columns of v's tile, which no other warp reads
      __syncwarp();
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          unsigned w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const auto pair = pair_from_f32<T>(make_float2(O[n + j / 2][(j & 1) * 2],
                                                           O[n + j / 2][(j & 1) * 2 + 1]));
            w[j] = *reinterpret_cast<const unsigned*>(&pair);
          }
          stmatrix4_trans(smem_addr(v + (n * 8 + (lane & 7) + ((lane & 16) >> 1)) * v_stride + warp * 16 +
                                    (lane & 8)), w[0], w[1], w[2], w[3]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[(n * 8 + t2 + (e & 1)) * v_stride + warp * 16 + g + (e / 2) * 8] = from_f32<T>(O[n][e]);
      }
      __syncwarp();
      T* to = out.o + row * out.ldo + h * p.dv + col;
      const T* from = v + warp * 16;
      if constexpr (VEC) {
        constexpr int kV = 16 / sizeof(T), kVecs = 16 / kV;
        for (int j = lane; j < n_rows * kVecs; j += 32) {
          const int r = j / kVecs, x = (j % kVecs) * kV;
          if (col + x < p.dv)
            *reinterpret_cast<uint4*>(to + r * out.ldo + x) =
                *reinterpret_cast<const uint4*>(from + r * v_stride + x);
        }
      } else {
        for (int j = lane; j < n_rows * 16; j += 32) {
          const int r = j / 16, x = j % 16;
          if (col + x < p.dv) to[r * out.ldo + x] = from[r * v_stride + x];
        }
      }
    }
    __syncthreads();  // the stage is free
  }
  if (out.hT) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = col + g + (e / 2) * 8, d = n * 8 + t2 + (e & 1);
        if (c < p.dv && d < p.dk) out.hT[(head * p.dk + d) * p.dv + c] = S[n][e];
      }
  }
}

template <typename T, int DK, bool VEC>
cudaError_t chain(const GdeltaRows<T>& p, const ChainOut<T>& out, cudaStream_t stream) {
  constexpr int STAGES = Terms<T>::n == 1 ? 2 : 1;
  // As many warps a block as dv has groups of 16 columns, fewer where that leaves SMs without a block.
  const int groups = (p.dv + 15) / 16;
  int warps = 1;
  while (warps < kMaxWarps && warps < groups &&
         p.batch * p.heads_v * ((groups + 2 * warps - 1) / (2 * warps)) >= kSms)
    warps *= 2;
  const int slices = (groups + warps - 1) / warps;
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
  return gdelta_places(batch, rows) * heads_v * ((dv + 15) / 16) * ((dk <= 64 ? 64 : 128) / 8) * 512;
}

}  // namespace bsolve
