// What the two chains of the gated delta rule share (bs_gdelta calls): a block's stages, a warp's 16
// columns of them, its state in registers.
#pragma once

#include <cmath>
#include <type_traits>

#include "barrier.cuh"
#include "gdelta_tile.cuh"
#include "grec_order.cuh"

namespace bsolve {
namespace {

constexpr int kMaxWarps = 8;
constexpr int kMaxShared = 230000;  // bytes of dynamic shared memory, beside what the kernels declare

// Tiles of one stage for a block of `warps` warps: q, k as terms, v (or a gradient of its shape) as stored, the
// prepared chunk.
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
                                           int64_t row, int n, int kh, int h, int col, int cols,
                                           int v_stride, int thread, int threads) {
  using S = Stage<T, DK>;
  auto* q = reinterpret_cast<__nv_bfloat16*>(stage);
  auto* k = reinterpret_cast<__nv_bfloat16*>(stage + S::kQk);
  T* v = reinterpret_cast<T*>(stage + 2 * S::kQk);
  auto* own = reinterpret_cast<uint4*>(stage + 2 * S::kQk + kChunk * v_stride * sizeof(T));
  load_terms<T, DK, S::kStride, VEC>(q, p.q + row * p.ldq + kh * p.dk, p.ldq, n, p.dk, thread,
                                         threads);
  load_terms<T, DK, S::kStride, VEC>(k, p.k + row * p.ldk + kh * p.dk, p.ldk, n, p.dk, thread,
                                         threads);
  const int width = min(p.dv - col, cols);
  load_rows<T, VEC>(v, v_stride, cols, v_rows + row * ldv + h * p.dv + col, ldv, n, width, thread, threads);
  for (int j = thread; j < static_cast<int>(sizeof(Prepared) / 16); j += threads)
    cp_async_16(own + j, reinterpret_cast<const uint4*>(prepared) + j, 16);
}

// Stages of a block of single warps: FP32 and FP16 rows are split on their way, none is brought ahead.
template <typename T>
constexpr int kWarpStages = Terms<T>::n == 1 ? 2 : 1;

// Whether a stage comes by bulk copies (rows that need no other form): a row an instruction instead of 16
// bytes (16,384 rows of 16 heads 128 x 128: forward chain 286 to 279 us, backward 269 to 251).
template <typename T, bool VEC>
constexpr bool kBulk = VEC && Terms<T>::n == 1;

// Zeros in a block's stages, once, where copies leave columns behind dk or rows behind a sequence.
__device__ __forceinline__ void clear_stages(unsigned char* stages, int bytes) {
  for (int j = threadIdx.x * 16; j < bytes; j += blockDim.x * 16)
    *reinterpret_cast<uint4*>(stages + j) = make_uint4(0, 0, 0, 0);
  writes_before_copies();
}

template <typename T, int DK>
__device__ __forceinline__ void copy_stage(unsigned char* stage, uint64_t* barrier, const GdeltaRows<T>& p,
                                           const T* v_rows, int64_t ldv, const Prepared* prepared,
                                           int64_t row, int n, int kh, int h, int col, int cols,
                                           int v_stride) {
  using S = Stage<T, DK>;
  auto* q = reinterpret_cast<T*>(stage);
  auto* k = reinterpret_cast<T*>(stage + S::kQk);
  T* v = reinterpret_cast<T*>(stage + 2 * S::kQk);
  const int width = min(p.dv - col, cols), dk_bytes = p.dk * static_cast<int>(sizeof(T)),
            v_bytes = width * static_cast<int>(sizeof(T));
  if (threadIdx.x == 0)
    barrier_expect(barrier, n * (2 * dk_bytes + v_bytes) + static_cast<int>(sizeof(Prepared)));
  for (int j = threadIdx.x; j < 3 * kChunk + 1; j += blockDim.x) {
    const int r = j % kChunk, which = j / kChunk;
    if (which == 3) {
      copy_bytes(stage + 2 * S::kQk + kChunk * v_stride * sizeof(T), prepared, sizeof(Prepared), barrier);
      continue;
    }
    T* to = which == 0 ? q + r * S::kStride : which == 1 ? k + r * S::kStride : v + r * v_stride;
    const int bytes = which == 2 ? v_bytes : dk_bytes;
    if (r < n) {
      const T* from = which == 0 ? p.q + (row + r) * p.ldq + kh * p.dk
                      : which == 1 ? p.k + (row + r) * p.ldk + kh * p.dk
                                   : v_rows + (row + r) * ldv + h * p.dv + col;
      copy_bytes(to, from, bytes, barrier);
    } else {
      for (int b = 0; b < bytes; b += 16)
        *reinterpret_cast<uint4*>(reinterpret_cast<char*>(to) + b) = make_uint4(0, 0, 0, 0);
    }
  }
}

// The warp's 16 columns (from `v`) of rows 8 n .. 8 n + 15 of a tile, transposed: as two neighbouring 16 x 8
// results.
template <typename T>
__device__ __forceinline__ void read_transposed(float (&x)[2][4], const T* v, int v_stride, int n) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
  if constexpr (sizeof(T) == 2) {
    unsigned w[4];
    ldmatrix4_trans(w, smem_address(v + (n * 8 + (lane & 7) + ((lane & 16) >> 1)) * v_stride + (lane & 8)));
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
      stmatrix4_trans(smem_address(v + (n * 8 + (lane & 7) + ((lane & 16) >> 1)) * v_stride + (lane & 8)),
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
// The 64 rows as first operands over the warp's 16 columns, [16 rows][hi, lo]; all of them, or one group of eight.
__device__ __forceinline__ void keep_rows(uint4* at, const float (&x)[8][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const Split a = split(x[2 * m][0], x[2 * m][1]), b = split(x[2 * m][2], x[2 * m][3]),
                c = split(x[2 * m + 1][0], x[2 * m + 1][1]), d = split(x[2 * m + 1][2], x[2 * m + 1][3]);
    at[2 * m * 32 + lane] = make_uint4(transposed(a.hi), transposed(c.hi), transposed(b.hi), transposed(d.hi));
    at[(2 * m + 1) * 32 + lane] =
        make_uint4(transposed(a.lo), transposed(c.lo), transposed(b.lo), transposed(d.lo));
  }
}
__device__ __forceinline__ void keep_row_group(uint4* at, int n, const float (&x)[4]) {
  const Split a = split(x[0], x[1]), b = split(x[2], x[3]);
  unsigned* to = reinterpret_cast<unsigned*>(at + n / 2 * 64 + (threadIdx.x & 31)) + (n & 1);
  to[0] = transposed(a.hi);
  to[2] = transposed(b.hi);
  to[128] = transposed(a.lo);
  to[130] = transposed(b.lo);
}

// The warp's 16 columns of a dk x dv state in and out of global memory, transposed in registers: rows g and
// g + 8 of the columns, elements from + 8 n + t2, + 1 of dk.
template <int NB>
__device__ __forceinline__ void load_state(float (&S)[NB][4], const float* state, int dk, int dv, int col,
                                           int from = 0) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col + g + (e / 2) * 8, d = from + n * 8 + t2 + (e & 1);
      S[n][e] = state && c < dv && d < dk ? state[d * dv + c] : 0.f;
    }
}
template <int NB>
__device__ __forceinline__ void store_state(const float (&S)[NB][4], float* state, int dk, int dv, int col,
                                            int from = 0) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = col + g + (e / 2) * 8, d = from + n * 8 + t2 + (e & 1);
      if (c < dv && d < dk) state[d * dv + c] = S[n][e];
    }
}

// What follows from a copy that never came: NaN in every later result.
template <int NB>
__device__ __forceinline__ void poison(float (&S)[NB][4]) {
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[n][e] = __int_as_float(0x7FC00000);
}

// The sequence, head and columns of a block.
struct Place {
  int64_t start, end, chunk;  // rows; the first chunk's place
  int64_t head;               // of the states
  int sequence, h, kh, col;
};
template <typename T>
__device__ __forceinline__ Place place_of(const GdeltaRows<T>& p, int slices, int cols, int64_t* scratch) {
  const int64_t part = static_cast<int64_t>(p.heads_v) * slices;
  int64_t s = blockIdx.x / part;
  const int rest = static_cast<int>(blockIdx.x % part);
  if (p.offsets && p.batch > 1 && p.batch <= min(kSortedBatch, static_cast<int>(blockDim.x)))
    s = nth_longest(p.offsets, static_cast<int>(p.batch), static_cast<int>(s), scratch);
  Place at;
  sequence_rows(p, s, &at.start, &at.end);
  at.h = rest / slices;
  at.kh = at.h / (p.heads_v / p.heads_k);
  at.col = rest % slices * cols;
  at.chunk = at.start / kChunk + s;
  at.head = s * p.heads_v + at.h;
  return at;
}

// Products one 16-deep piece at a time, each sum's terms apart from each other.
//
// c[n] += a (rows n of a tile, along their elements from k), for all eight groups of rows.
template <int NT, int STRIDE>
__device__ __forceinline__ void along_rows(float (&c)[8][4], const unsigned (&hi)[4], const unsigned (&lo)[4],
                                           unsigned tile, unsigned term, int k) {
  unsigned b[4][4];
#pragma unroll
  for (int n = 0; n < 4; ++n) ldmatrix4(b[n], along<STRIDE>(tile, n * 16, k));
#pragma unroll
  for (int n = 0; n < 8; ++n) mma(c[n], hi, b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
#pragma unroll
  for (int n = 0; n < 8; ++n) mma(c[n], lo, b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
  if constexpr (NT == 2) {
#pragma unroll
    for (int n = 0; n < 4; ++n) ldmatrix4(b[n], along<STRIDE>(tile + term, n * 16, k));
#pragma unroll
    for (int n = 0; n < 8; ++n) mma(c[n], hi, b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
  }
}
// c[n] += a (16 rows of a tile from k), for all groups of eight of their elements.
template <int NT, int NB, int STRIDE>
__device__ __forceinline__ void across_rows(float (&c)[NB][4], const unsigned (&hi)[4], const unsigned (&lo)[4],
                                            unsigned tile, unsigned term, int k) {
#pragma unroll
  for (int first = 0; first < NB; first += 8) {
    unsigned b[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) ldmatrix4_trans(b[n], across(tile, STRIDE, k, first * 8 + n * 16));
#pragma unroll
    for (int n = 0; n < 8; ++n) mma(c[first + n], hi, b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
#pragma unroll
    for (int n = 0; n < 8; ++n) mma(c[first + n], lo, b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
    if constexpr (NT == 2) {
#pragma unroll
      for (int n = 0; n < 4; ++n) ldmatrix4_trans(b[n], across(tile + term, STRIDE, k, first * 8 + n * 16));
#pragma unroll
      for (int n = 0; n < 8; ++n) mma(c[first + n], hi, b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
    }
  }
}
// The same for a part of the elements from `first`, N groups of eight.
template <int NT, int N, int STRIDE>
__device__ __forceinline__ void part_across(float (&c)[N][4], const unsigned (&hi)[4], const unsigned (&lo)[4],
                                            unsigned tile, unsigned term, int k, int first) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    unsigned b[N / 2][4];
#pragma unroll
    for (int n = 0; n < N / 2; ++n) ldmatrix4_trans(b[n], across(tile + t * term, STRIDE, k, first + n * 16));
#pragma unroll
    for (int n = 0; n < N; ++n) mma(c[n], hi, b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
    if (t == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) mma(c[n], lo, b[n / 2][(n & 1) * 2], b[n / 2][(n & 1) * 2 + 1]);
  }
}
// c[n] += a piece(n), n from FIRST to LAST - 1; a in one term where A1.
template <int FIRST, int LAST, bool A1, typename F>
__device__ __forceinline__ void by_pieces(float (&c)[8][4], const unsigned (&hi)[4], const unsigned (&lo)[4],
                                          F&& piece) {
#pragma unroll
  for (int first = FIRST; first < LAST; first += 4) {
    uint4 b[4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
      if (first + n < LAST) b[n] = piece(first + n);
#pragma unroll
    for (int n = 0; n < 4; ++n)
      if (first + n < LAST) mma(c[first + n], hi, b[n].x, b[n].y);
#pragma unroll
    for (int n = 0; n < 4; ++n)
      if (first + n < LAST) mma(c[first + n], hi, b[n].z, b[n].w);
    if constexpr (!A1) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
        if (first + n < LAST) mma(c[first + n], lo, b[n].x, b[n].y);
    }
  }
}
// Calls f with 0, 1, 2, 3 as constants.
template <typename F>
__device__ __forceinline__ void four(F&& f) {
  f(std::integral_constant<int, 0>());
  f(std::integral_constant<int, 1>());
  f(std::integral_constant<int, 2>());
  f(std::integral_constant<int, 3>());
}

// ---------------------------------------------------------------------------- several warps a group of columns
// KS warps share 16 columns: each keeps an equal part of dk of the transposed state and works out
// the chunk's rows in its 8 / KS groups of eight. What all of them need as first operands of the next products goes
// through shared memory, split and in the registers' order.
template <int KS>
struct Team {
  static constexpr int kRows = 8 / KS;  // groups of rows of a warp
  int j;                                // the warp's place
  // Group i of the warp: low and high numbers together, since the triangles grow with them.
  __device__ __forceinline__ int rows(int i) const {
    return 2 * KS * (i / 2) + (i & 1 ? 2 * KS - 1 - j : j);
  }
};
template <int DK>
struct Exchange {
  uint4 state[DK / 16][2][32];  // [16 of dk][hi, lo]
  uint4 first[4][2][32];        // [16 rows]
  uint4 second[4][2][32];
  uint4 third[4][2][32];
};
// One group of eight rows (a 16 x 8 result) as half of a first operand over 16 rows.
__device__ __forceinline__ void put_half(uint4 (&at)[4][2][32], int n, const float (&x)[4]) {
  const int lane = threadIdx.x & 31;
  const Split a = split(x[0], x[1]), b = split(x[2], x[3]);
  reinterpret_cast<uint2*>(&at[n / 2][0][lane])[n & 1] = make_uint2(a.hi, b.hi);
  reinterpret_cast<uint2*>(&at[n / 2][1][lane])[n & 1] = make_uint2(a.lo, b.lo);
}
__device__ __forceinline__ void get_operand(unsigned (&hi)[4], unsigned (&lo)[4], const uint4 (&at)[2][32]) {
  const int lane = threadIdx.x & 31;
  const uint4 a = at[0][lane], b = at[1][lane];
  hi[0] = a.x, hi[1] = a.y, hi[2] = a.z, hi[3] = a.w;
  lo[0] = b.x, lo[1] = b.y, lo[2] = b.z, lo[3] = b.w;
}
// ldmatrix addresses of two groups of eight rows, n and m: as second operand over the rows' elements, and transposed as
// two 16 x 8 results.
template <int STRIDE>
__device__ __forceinline__ unsigned along_two(unsigned tile, int n, int m, int k) {
  const int lane = threadIdx.x & 31;
  return tile + 2 * (((lane & 16 ? m : n) * 8 + (lane & 7)) * STRIDE + k + (lane & 8));
}
template <typename T>
__device__ __forceinline__ void read_two(float (&x)[4], float (&y)[4], const T* v, int v_stride, int n, int m) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
  if constexpr (sizeof(T) == 2) {
    unsigned w[4];
    ldmatrix4_trans(w, smem_address(v + ((lane & 16 ? m : n) * 8 + (lane & 7)) * v_stride + (lane & 8)));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 a = to_f32(*reinterpret_cast<const typename Pair<T>::type*>(&w[j])),
                   b = to_f32(*reinterpret_cast<const typename Pair<T>::type*>(&w[2 + j]));
      x[2 * j] = a.x, x[2 * j + 1] = a.y, y[2 * j] = b.x, y[2 * j + 1] = b.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = to_f32(v[(n * 8 + t2 + (e & 1)) * v_stride + g + (e / 2) * 8]);
      y[e] = to_f32(v[(m * 8 + t2 + (e & 1)) * v_stride + g + (e / 2) * 8]);
    }
  }
}
// Rounds two groups of eight rows through the warp's own rows and columns of a tile and stores those below
// n_rows, `width` columns at most.
template <typename T, bool VEC>
__device__ __forceinline__ void store_two(const float (&x)[4], const float (&y)[4], T* v, int v_stride, int n,
                                          int m, T* to, int64_t ld, int n_rows, int width) {
  const int lane = threadIdx.x & 31, g = lane / 4, t2 = (lane & 3) * 2;
  __syncwarp();
  if constexpr (sizeof(T) == 2) {
    unsigned w[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const auto a = pair_from_f32<T>(make_float2(x[2 * j], x[2 * j + 1])),
                 b = pair_from_f32<T>(make_float2(y[2 * j], y[2 * j + 1]));
      w[j] = *reinterpret_cast<const unsigned*>(&a);
      w[2 + j] = *reinterpret_cast<const unsigned*>(&b);
    }
    stmatrix4_trans(smem_address(v + ((lane & 16 ? m : n) * 8 + (lane & 7)) * v_stride + (lane & 8)), w[0], w[1],
                    w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[(n * 8 + t2 + (e & 1)) * v_stride + g + (e / 2) * 8] = from_f32<T>(x[e]);
      v[(m * 8 + t2 + (e & 1)) * v_stride + g + (e / 2) * 8] = from_f32<T>(y[e]);
    }
  }
  __syncwarp();
  constexpr int kV = VEC ? 16 / static_cast<int>(sizeof(T)) : 1, kVecs = 16 / kV;
#pragma unroll
  for (int j = lane; j < 16 * kVecs; j += 32) {
    const int r = j / kVecs, c = (j % kVecs) * kV, row = (r < 8 ? n : m) * 8 + (r & 7);
    if (row >= n_rows || c >= width) continue;
    if constexpr (VEC)
      *reinterpret_cast<uint4*>(to + row * ld + c) = *reinterpret_cast<const uint4*>(v + row * v_stride + c);
    else
      to[row * ld + c] = v[row * v_stride + c];
  }
}
// A block's stages: three where two teams' fit (32,768 BF16 rows of 16 heads 128 x 128, the whole call: 1,072 to 940
// us). Four more warps for O, which the next chunk does not wait for, gained nothing beside them.
template <typename T, int DK>
constexpr int kTeamStages =
    3 * Stage<T, DK>::bytes(2) + 2 * static_cast<int>(sizeof(Exchange<DK>)) <= kMaxShared ? 3 : 2;
template <typename T, int DK>
constexpr int team_bytes(int teams) {
  return kTeamStages<T, DK> * Stage<T, DK>::bytes(teams) + teams * static_cast<int>(sizeof(Exchange<DK>));
}
// Teams of a block at most, and the threads behind them that bring the stages: the same registers a thread are left
// where one team's stages are all that fits, and its rows have to be split on their way (3 x 1,023 unaligned FP32 rows of
// 5 heads 93 x 77: 105 us with 128 such threads, 82 with 256; 32,768 BF16 rows, which are only copied, 940 and 1,003).
template <typename T, int DK>
constexpr int kMaxTeams = team_bytes<T, DK>(2) <= kMaxShared ? 2 : 1;
template <typename T, int DK>
constexpr int kLoaders = kMaxTeams<T, DK> == 2 ? 128 : 256;
// How a chain's blocks are made up: teams of four warps (`teams` a block), or one warp a group of columns.
struct Blocks {
  int teams, warps;
};
// A chunk's time in a block, 0.01 us, where every SM has one: of one team and of two; of four single warps, and with two
// such blocks on an SM; of eight. Measured over 2,048 and 4,096 rows of 152 or 304 heads with as many columns as the
// block has, the mean of both passes (BF16, 128: forward 1.6, 2.4, 5.3 and 6.8 us). 0: does not fit. ALIGNED: rows
// that come in pieces of 16 bytes; others come by elements.
struct ChunkTimes {
  int teams[2], four[2], eight;
};
template <typename T, int DK, bool ALIGNED>
constexpr ChunkTimes chunk_times() {
  constexpr bool kLong = DK == 128;
  if constexpr (Terms<T>::n == 1) {
    if (ALIGNED) return kLong ? ChunkTimes{{170, 256}, {568, 0}, 719} : ChunkTimes{{147, 204}, {449, 566}, 557};
    return kLong ? ChunkTimes{{1462, 1564}, {2151, 0}, 1776} : ChunkTimes{{823, 923}, {1422, 1594}, 1307};
  } else if constexpr (sizeof(T) == 2) {
    if (ALIGNED) return kLong ? ChunkTimes{{310, 0}, {963, 1143}, 1172} : ChunkTimes{{299, 345}, {630, 776}, 877};
    return kLong ? ChunkTimes{{864, 0}, {2467, 2684}, 2169} : ChunkTimes{{839, 945}, {1555, 1741}, 1484};
  } else {
    if (ALIGNED) return kLong ? ChunkTimes{{457, 0}, {1645, 1843}, 1556} : ChunkTimes{{451, 491}, {966, 1135}, 1010};
    return kLong ? ChunkTimes{{578, 0}, {1882, 2160}, 1925} : ChunkTimes{{554, 688}, {1325, 1504}, 1416};
  }
}
constexpr int kTurnTime = 400;  // what a turn costs beside its chunks: the same runs, extended to none
// The least time. Equal sequences run in turns of what the GPU holds, a turn as long as its blocks. Uneven ones fill
// each other's gaps, but the longest, about 1 + ln(batch) times the average where they were cut at random, cannot take less
// than its own chunks. A team takes the chain's products apart, so that a chunk takes less than half of one warp's
// time, but its warps exchange their parts, so that blocks of eight single warps do more in all.
template <typename T, int DK, bool ALIGNED>
Blocks chain_blocks(const GdeltaRows<T>& p) {
  constexpr ChunkTimes kTimes = chunk_times<T, DK, ALIGNED>();
  static_assert((kTimes.teams[1] != 0) == (kMaxTeams<T, DK> == 2), "a time for every block that fits");
  const int groups = gdelta_groups(p.dv);
  const double average = std::fmax(1.0, static_cast<double>(p.rows) / (static_cast<double>(p.batch) * kChunk));
  const double chunks = p.offsets ? average : std::ceil(average);
  Blocks best{1, 0};
  double least = 0;
  // blocks of so many groups, `one` a chunk with one of them on an SM, `two` with two (0: there is no room)
  auto offer = [&](int a_block, int one, int two, Blocks b) {
    if (one == 0) return;
    const double blocks = static_cast<double>(p.batch * p.heads_v * ((groups + a_block - 1) / a_block));
    const double held = two ? 2.0 * kSms : kSms;
    auto turn = [&](int time) { return chunks * time + kTurnTime; };
    double cost;
    if (p.offsets) {
      const int time = two && blocks > kSms ? two : one;
      cost = std::fmax(blocks / (time == one ? kSms : held) * turn(time),
                       chunks * (1.0 + std::log(static_cast<double>(p.batch))) * time);
    } else {
      const double turns = std::floor(blocks / held), rest = blocks - turns * held;
      cost = turns * turn(two ? two : one) + (rest > kSms ? turn(two) : rest > 0 ? turn(one) : 0);
    }
    if (least == 0 || cost < least) least = cost, best = b;
  };
  offer(1, kTimes.teams[0], 0, {1, 0});
  if (groups > 1) offer(2, kTimes.teams[1], 0, {2, 0});
  if (groups > 2) offer(4, kTimes.four[0], kTimes.four[1], {0, 4});
  if (groups > 4) offer(8, kTimes.eight, 0, {0, 8});
  return best;
}
// Launches a chain in the blocks that chain_blocks() gives, by its kernel for teams or the one for single warps. The
// limit of shared memory belongs to the kernel and the device, not to a host thread: it is the kernel's
// largest, since a call that set its own size could lower it between another thread's setting and launch.
template <typename T, int DK, bool ALIGNED, typename Out>
cudaError_t launch_chain(void (*by_teams)(GdeltaRows<T>, Out, int), void (*by_warps)(GdeltaRows<T>, Out, int),
                         const GdeltaRows<T>& p, const Out& out, cudaStream_t stream) {
  const auto [teams, warps] = chain_blocks<T, DK, ALIGNED>(p);
  auto* kernel = teams ? by_teams : by_warps;
  const int groups = teams ? teams : warps, slices = (gdelta_groups(p.dv) + groups - 1) / groups;
  const int threads = teams ? teams * 128 + kLoaders<T, DK> : warps * 32;
  const int shared = teams ? team_bytes<T, DK>(teams) : kWarpStages<T> * Stage<T, DK>::bytes(warps);
  const int most = teams ? team_bytes<T, DK>(kMaxTeams<T, DK>) : kWarpStages<T> * Stage<T, DK>::bytes(kMaxWarps);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(p.batch * p.heads_v * slices), threads, shared, stream>>>(p, out, slices);
  return cudaGetLastError();
}
// The warps behind the teams bring the stages: `load` for each chunk in its order, two stages ahead at most.
template <bool ASYNC, typename F>
__device__ __forceinline__ void bring_stages(int64_t chunks, int stages, uint64_t* full, uint64_t* empty,
                                             volatile int* failed, F&& load) {
  for (int64_t i = 0; i < chunks; ++i) {
    const int s = static_cast<int>(i % stages);
    if (!wait_for(&empty[s], (i / stages & 1) ^ 1, failed)) return;
    load(i, s);
    if constexpr (ASYNC) {
      arrive_behind_copies(&full[s]);
    } else {
      cp_async_wait_all();
      barrier_arrive(&full[s]);
    }
  }
  cp_async_wait_all();
}
__device__ __forceinline__ void team_sync(int team, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

}  // namespace
}  // namespace bsolve
