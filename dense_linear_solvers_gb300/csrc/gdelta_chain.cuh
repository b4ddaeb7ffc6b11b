// What the two chains of the gated delta rule share (bs_gdelta calls): a block's stages, a warp's 16
// columns of them, its state in registers.
#pragma once

#include "gdelta_tile.cuh"
#include "grec_order.cuh"

namespace bsolve {
namespace {

constexpr int kMaxWarps = 8;

// Tiles of one stage for a block of `warps` warps: q, k as terms, v (or a gradient of its shape) as stored, the prepared chunk.
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

template <typename T, int DK, bool VEC>
__device__ __forceinline__ void load_stage(unsigned char* stage, const GdeltaRows<T>& p,
                                           const T* v_rows, int64_t ldv, const Prepared* prepared,
                                           int64_t row, int n, int kh, int h, int col, int v_stride) {
  using S = Stage<T, DK>;
  auto* q = reinterpret_cast<__nv_bfloat16*>(stage);
  auto* k = reinterpret_cast<__nv_bfloat16*>(stage + S::kQk);
  T* v = reinterpret_cast<T*>(stage + 2 * S::kQk);
  auto* own = reinterpret_cast<uint4*>(stage + 2 * S::kQk + kChunk * v_stride * sizeof(T));
  load_terms<T, DK, S::kStride, VEC>(q, p.q + row * p.ldq + kh * p.dk, p.ldq, n, p.dk);
  load_terms<T, DK, S::kStride, VEC>(k, p.k + row * p.ldk + kh * p.dk, p.ldk, n, p.dk);
  const int width = min(p.dv - col, static_cast<int>(blockDim.x) / 2);
  load_rows<T, VEC>(v, v_stride, blockDim.x / 2, v_rows + row * ldv + h * p.dv + col, ldv, n, width);
  for (int j = threadIdx.x; j < static_cast<int>(sizeof(Prepared) / 16); j += blockDim.x)
    cp_async_16(own + j, reinterpret_cast<const uint4*>(prepared) + j, 16);
  cp_async_commit();
}

// The warp's 16 columns (from `v`) of rows 8 n .. 8 n + 15 of a tile, transposed: as two neighbouring 16 x 8
// results.
template <typename T>
__device__ __forceinline__ void read_transposed(float (&x)[2][4], const T* v, int v_stride, int n) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
  if constexpr (sizeof(T) == 2) {
    unsigned w[4];
    ldmatrix4_trans(w, smem_addr(v + (n * 8 + (lane & 7) + ((lane & 16) >> 1)) * v_stride + (lane & 8)));
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
        x[j][e] = to_f32(v[((n + j) * 8 + t2 + (e & 1)) * v_stride + g + (e / 2) * 8]);
  }
}

// Rounds the warp's 64 rows (transposed results) through its own columns of a tile and stores the first
// n_rows of them, `width` columns at most.
template <typename T, bool VEC>
__device__ __forceinline__ void store_transposed(const float (&O)[8][4], T* v, int v_stride, T* to,
                                                 int64_t ld, int n_rows, int width) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
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
      stmatrix4_trans(smem_addr(v + (n * 8 + (lane & 7) + ((lane & 16) >> 1)) * v_stride + (lane & 8)),
                      w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[(n * 8 + t2 + (e & 1)) * v_stride + g + (e / 2) * 8] = from_f32<T>(O[n][e]);
  }
  __syncwarp();
  if constexpr (VEC) {
    constexpr int kV = 16 / sizeof(T), kVecs = 16 / kV;
    for (int j = lane; j < n_rows * kVecs; j += 32) {
      const int r = j / kVecs, x = (j % kVecs) * kV;
      if (x < width)
        *reinterpret_cast<uint4*>(to + r * ld + x) = *reinterpret_cast<const uint4*>(v + r * v_stride + x);
    }
  } else {
    for (int j = lane; j < n_rows * 16; j += 32) {
      const int r = j / 16, x = j % 16;
      if (x < width) to[r * ld + x] = v[r * v_stride + x];
    }
  }
}

// N results of 16 x 8, transposed, as pieces of second operands over the warp's 16 columns.
template <int N>
__device__ __forceinline__ void keep_pieces(uint4* at, const float (&x)[N][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const Split a = split(x[n][0], x[n][1]), b = split(x[n][2], x[n][3]);
    at[n * 32 + lane] = make_uint4(transposed(a.hi), transposed(b.hi), transposed(a.lo), transposed(b.lo));
  }
}

// The warp's 16 columns of a dk x dv state in and out of global memory, transposed in registers: rows g and
// g + 8 of the columns, elements 8 n + t2, + 1 of dk.
template <int NB>
__device__ __forceinline__ void load_state(float (&S)[NB][4], const float* state, int dk, int dv, int col) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col + g + (e / 2) * 8, d = n * 8 + t2 + (e & 1);
      S[n][e] = state && c < dv && d < dk ? state[d * dv + c] : 0.f;
    }
}
template <int NB>
__device__ __forceinline__ void store_state(const float (&S)[NB][4], float* state, int dk, int dv, int col) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col + g + (e / 2) * 8, d = n * 8 + t2 + (e & 1);
      if (c < dv && d < dk) state[d * dv + c] = S[n][e];
    }
}

// The sequence, head and columns of a block.
struct Place {
  int64_t start, end, chunk;  // rows; the first chunk's place
  int64_t head;               // of the states
  int sequence, h, kh, col;
};
template <typename T>
__device__ __forceinline__ Place place_of(const GdeltaRows<T>& p, int slices, int64_t* scratch) {
  const int64_t part = static_cast<int64_t>(p.heads_v) * slices;
  int64_t s = blockIdx.x / part;
  const int rest = static_cast<int>(blockIdx.x % part);
  if (p.offsets && p.batch > 1 && p.batch <= min(kSortedBatch, static_cast<int>(blockDim.x)))
    s = nth_longest(p.offsets, static_cast<int>(p.batch), static_cast<int>(s), scratch);
  Place at;
  sequence_rows(p, s, &at.start, &at.end);
  at.h = rest / slices;
  at.kh = at.h / (p.heads_v / p.heads_k);
  at.col = rest % slices * (blockDim.x / 2);
  at.chunk = at.start / kChunk + s;
  at.head = s * p.heads_v + at.h;
  return at;
}

// As many warps a block as dv has groups of 16 columns, fewer where that leaves SMs without a block.
template <typename T>
int chain_warps(const GdeltaRows<T>& p) {
  const int groups = gdelta_groups(p.dv);
  int warps = 1;
  while (warps < kMaxWarps && warps < groups &&
         p.batch * p.heads_v * ((groups + 2 * warps - 1) / (2 * warps)) >= kSms)
    warps *= 2;
  return warps;
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

}  // namespace
}  // namespace bsolve
