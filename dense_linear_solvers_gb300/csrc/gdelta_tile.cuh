// Tiles of the gated delta rule's kernels (bs_gdelta calls): matrix products of BF16 terms in registers,
// rows brought into shared memory, chunks of a sequence and their places in workspaces.
//
// Products run on mma.sync m16n8k16 with BF16 operands and FP32 sums. What is not a BF16 number by
// itself (states, solutions, decayed products; inputs in FP16 and FP32) is split into two
// BF16 terms, x = hi + lo up to 2^-18 |x| (two roundings to eight bits), and a product of two split
// operands takes hi hi + hi lo + lo hi; lo lo is below 2^-18 too. BF16 and not FP16 or TF32: the
// terms keep FP32's range, and a product of two terms costs half of one in TF32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "barrier.cuh"
#include "common.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {

constexpr int kChunk = 64;  // rows of a sequence that are solved together

// Rows 0, 64, 128, ... of a sequence start its chunks. Sequence s that starts at row a has its chunks at
// places a / 64 + s, ...: ceil(length / 64) of them fit in front of the next one's.
constexpr int64_t gdelta_places(int64_t batch, int64_t rows) { return rows / kChunk + batch; }

template <typename T>
struct Terms { static constexpr int n = 2; };   // BF16 terms of an input
template <>
struct Terms<__nv_bfloat16> { static constexpr int n = 1; };

// ---------------------------------------------------------------------------- products
__device__ __forceinline__ void mma(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(unsigned (&r)[4], unsigned at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(unsigned (&r)[4], unsigned at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void stmatrix4_trans(unsigned at, unsigned a, unsigned b, unsigned c,
                                                unsigned d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at),
               "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// An 8 x 8 matrix of 16-bit elements, transposed across the warp.
__device__ __forceinline__ unsigned transposed(unsigned v) {
  unsigned r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Two values as two BF16 terms each.
struct Split {
  unsigned hi, lo;
};
__device__ __forceinline__ unsigned pack_bf16(float x, float y) {
  const __nv_bfloat162 v = __float22bfloat162_rn(make_float2(x, y));
  return *reinterpret_cast<const unsigned*>(&v);
}
__device__ __forceinline__ Split split(float x, float y) {
  Split s;
  s.hi = pack_bf16(x, y);
  s.lo = pack_bf16(__fsub_rn(x, __uint_as_float(s.hi << 16)),
                   __fsub_rn(y, __uint_as_float(s.hi & 0xFFFF0000u)));
  return s;
}
// The first operand of a product, 16 x 16, from two neighbouring 16 x 8 results.
__device__ __forceinline__ void split_operand(unsigned (&hi)[4], unsigned (&lo)[4],
                                              const float (&x)[4], const float (&y)[4]) {
  const Split a = split(x[0], x[1]), b = split(x[2], x[3]), c = split(y[0], y[1]),
              d = split(y[2], y[3]);
  hi[0] = a.hi, hi[1] = b.hi, hi[2] = c.hi, hi[3] = d.hi;
  lo[0] = a.lo, lo[1] = b.lo, lo[2] = c.lo, lo[3] = d.lo;
}

// ---------------------------------------------------------------------------- chunks
// The chunk at a place, and the sequences of a call.
struct Span {
  int64_t row;  // the first row
  int rows;     // 0: there is none
  int sequence;
};
template <typename T>
__device__ __forceinline__ void sequence_rows(const GdeltaRows<T>& p, int64_t s, int64_t* start,
                                              int64_t* end) {
  if (!p.offsets) {
    *start = s * p.length;
    *end = *start + p.length;
    return;
  }
  int64_t a = p.offsets[s], b = p.offsets[s + 1];
  a = a < 0 ? 0 : a > p.rows ? p.rows : a;
  b = b < a ? a : b > p.rows ? p.rows : b;
  *start = a;
  *end = b;
}
// Looks for the last sequence whose first place is not behind `place`; 32 probes a turn, by one warp.
template <typename T>
__device__ __forceinline__ Span chunk_at(const GdeltaRows<T>& p, int64_t place) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, n = p.batch;  // the answer is one of lo .. lo + n - 1
  while (n > 1) {
    const int64_t step = (n + 31) / 32, s = lo + lane * step;
    bool before = false;
    if (lane * step < n) {
      int64_t a, b;
      sequence_rows(p, s, &a, &b);
      before = a / kChunk + s <= place;
    }
    const unsigned yes = __ballot_sync(0xFFFFFFFFu, before);
    const int last = yes ? 31 - __clz(yes) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  int64_t a, b;
  sequence_rows(p, lo, &a, &b);
  const int64_t row = a + (place - (a / kChunk + lo)) * kChunk;
  Span s;
  s.sequence = static_cast<int>(lo);
  s.row = row;
  s.rows = row >= a && row < b ? static_cast<int>(min(b - row, static_cast<int64_t>(kChunk))) : 0;
  return s;
}

// ---------------------------------------------------------------------------- rows in shared memory
// Brings `n` rows of `width` elements (row j at src + j ld) into a tile of 64 rows of COLS elements, row
// distance STRIDE, as BF16 terms, one tile a term, zeros elsewhere. VEC: rows aligned to 16 bytes.
// BF16 rows come by cp.async: commit and wait behind it. By `threads` threads, this one number `thread`.
template <typename T, int COLS, int STRIDE, bool VEC>
__device__ __forceinline__ void load_terms(__nv_bfloat16* tile, const T* src, int64_t ld, int n,
                                           int width, int thread, int threads) {
  constexpr int kTerm = kChunk * STRIDE;
  // where they have to be split, or are not aligned, several loads are asked for before the first is used
  if constexpr (VEC && Terms<T>::n == 1) {
    constexpr int kV = 16 / sizeof(T), kVecs = COLS / kV;
    for (int j = thread; j < kChunk * kVecs; j += threads) {
      const int r = j / kVecs, c = (j % kVecs) * kV;
      const int have = r < n ? min(max(width - c, 0), kV) : 0;  // width is a multiple of kV here
      cp_async_16(tile + r * STRIDE + c, have ? src + r * ld + c : src, have * static_cast<int>(sizeof(T)));
    }
  } else if constexpr (VEC) {
    constexpr int kV = 16 / sizeof(T), kVecs = COLS / kV, kAtOnce = 4;
    for (int first = thread; first < kChunk * kVecs; first += kAtOnce * threads) {
      uint4 v[kAtOnce];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int j = first + a * threads, r = j / kVecs, c = (j % kVecs) * kV;
        v[a] = j < kChunk * kVecs && r < n && c < width ? *reinterpret_cast<const uint4*>(src + r * ld + c)
                                                        : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int j = first + a * threads;
        if (j >= kChunk * kVecs) break;
        unsigned* at = reinterpret_cast<unsigned*>(tile + j / kVecs * STRIDE + (j % kVecs) * kV);
        const auto* pairs = reinterpret_cast<const typename Pair<T>::type*>(&v[a]);
#pragma unroll
        for (int e = 0; e < kV / 2; ++e) {
          const float2 f = to_f32(pairs[e]);
          const Split s = split(f.x, f.y);
          at[e] = s.hi;
          at[kTerm / 2 + e] = s.lo;
        }
      }
    }
  } else {
    constexpr int kPairs = COLS / 2, kAtOnce = 8;
    for (int first = thread; first < kChunk * kPairs; first += kAtOnce * threads) {
      float2 v[kAtOnce];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int j = first + a * threads, r = j / kPairs, c = (j % kPairs) * 2;
        const bool row = j < kChunk * kPairs && r < n;
        const T* from = src + r * ld + c;
        v[a].x = row && c < width ? to_f32(from[0]) : 0.f;
        v[a].y = row && c + 1 < width ? to_f32(from[1]) : 0.f;
      }
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int j = first + a * threads;
        if (j >= kChunk * kPairs) break;
        unsigned* at = reinterpret_cast<unsigned*>(tile + j / kPairs * STRIDE + (j % kPairs) * 2);
        const Split s = split(v[a].x, v[a].y);
        at[0] = s.hi;  // a BF16 number itself
        if constexpr (Terms<T>::n == 2) at[kTerm / 2] = s.lo;
      }
    }
  }
}

// The same, as stored: `cols` elements a row.
template <typename T, bool VEC>
__device__ __forceinline__ void load_rows(T* tile, int stride, int cols, const T* src, int64_t ld,
                                          int n, int width, int thread, int threads) {
  if constexpr (VEC) {
    constexpr int kV = 16 / sizeof(T);
    const int vecs = cols / kV;
    for (int j = thread; j < kChunk * vecs; j += threads) {
      const int r = j / vecs, c = (j % vecs) * kV;
      const int have = r < n ? min(max(width - c, 0), kV) : 0;
      cp_async_16(tile + r * stride + c, have ? src + r * ld + c : src,
                  have * static_cast<int>(sizeof(T)));
    }
  } else {
    constexpr int kAtOnce = 8;
    for (int first = thread; first < kChunk * cols; first += kAtOnce * threads) {
      T v[kAtOnce];
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int j = first + a * threads, r = j / cols, c = j % cols;
        v[a] = r < n && c < width ? src[r * ld + c] : from_f32<T>(0.f);
      }
#pragma unroll
      for (int a = 0; a < kAtOnce; ++a) {
        const int j = first + a * threads;
        if (j < kChunk * cols) tile[j / cols * stride + j % cols] = v[a];
      }
    }
  }
}

// Addresses of ldmatrix in a tile of rows STRIDE apart, for a lane: the second operand of a product over
// the rows' elements (its columns the rows n, two groups of eight, 16 elements from k), and over
// the rows themselves (16 rows from k, two groups of eight elements from n).
template <int STRIDE>
__device__ __forceinline__ unsigned along(unsigned tile, int n, int k) {
  const int lane = threadIdx.x & 31;
  return tile + 2 * ((n + (lane & 7) + ((lane & 16) >> 1)) * STRIDE + k + (lane & 8));
}
__device__ __forceinline__ unsigned across(unsigned tile, int stride, int k, int n) {
  const int lane = threadIdx.x & 31;
  return tile + 2 * ((k + (lane & 15)) * stride + n + ((lane & 16) >> 1));
}

// ---------------------------------------------------------------------------- prepared chunks
// What a chunk's chain needs of each value head, made from q, k, g, beta alone: the inverse and the mixing matrix,
// lower triangular, as second operands in registers' order (20 pieces of 8 columns and 16 deep, hi and lo, 16 bytes
// a lane), and by row the decay from the chunk's start, beta, the decay to its end, and the log decays' sum.
constexpr int kPieces = 20;
struct Prepared {
  uint4 inverse[kPieces][32];
  uint4 mixing[kPieces][32];
  float front[kChunk], beta[kChunk], back[kChunk];
  float sum_hi[kChunk], sum_lo[kChunk];  // the running sum of the log decays, in units of log 2
};
static_assert(sizeof(Prepared) % 16 == 0, "copied in pieces of 16 bytes");
// Where a piece of the lower triangle is: columns (2 pair + half) * 8 .. + 7, which are rows of the matrix, depth
// k * 16 .. + 15, k <= pair; and of the upper one, k >= pair, for the transposed products.
__host__ __device__ constexpr int lower_piece(int pair, int half, int k) {
  return pair * (pair + 1) + half * (pair + 1) + k;
}
__host__ __device__ constexpr int upper_piece(int pair, int half, int k) {
  return pair * (9 - pair) + half * (4 - pair) + k - pair;
}

constexpr double kLog2 = 1.4426950408889634;  // 1 / log 2
// 2^v, within two units in the last place; 0 below 2^-126.
__device__ __forceinline__ float power_of_two(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// e^(b_r - b_i) from the sums' two parts, in units of log 2.
__device__ __forceinline__ float decay_between(const float* hi, const float* lo, int r, int i) {
  return power_of_two(__fadd_rn(__fsub_rn(hi[r], hi[i]), __fsub_rn(lo[r], lo[i])));
}

// What the chains leave for the gradients of a chunk, by value head and 16 columns of dv: a state (or its
// gradient) as second operand of products over dv, in pieces as above, and 64 rows as first operand of such.
__host__ __device__ constexpr int gdelta_groups(int dv) { return (dv + 15) / 16; }
constexpr int gdelta_deep(int dk) { return dk <= 64 ? 64 : 128; }   // dk as the kernels pad it
__host__ __device__ constexpr int64_t kept_pieces(int deep) { return deep / 8 + kChunk / 8; }
inline size_t kept_bytes(int heads_v, int dk, int dv, int64_t batch, int64_t rows) {
  return gdelta_places(batch, rows) * heads_v * gdelta_groups(dv) * kept_pieces(gdelta_deep(dk)) * 512;
}

template <typename T>
cudaError_t launch_gdelta_prepare(const GdeltaRows<T>& p, bool for_backward, Prepared* out,
                                  cudaStream_t stream);

}  // namespace bsolve
