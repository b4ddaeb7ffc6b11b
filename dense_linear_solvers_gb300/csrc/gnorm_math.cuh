// The gate of the norms around a block and the staging of their rows (bs_gnorm calls).
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "common.cuh"
#include "grec_math.cuh"
#include "row_types.cuh"

namespace bsolve {

// act(z) and its derivative, for H pairs of elements; KIND: a bs_gate. sigma(z) = 1 / (1 + e^-z),
// 1 - sigma(z) = e^-z sigma(z) with e^-z kept finite there. The approximate exponential and
// reciprocal are within 2 ulp.
template <int KIND, bool SLOPE, int H>
__device__ __forceinline__ void gate_kind(const float2 (&z)[H], float2 (&act)[H], float2 (&slope)[H]) {
#pragma unroll
  for (int k = 0; k < H; ++k) {
    if constexpr (KIND == 2) {
      act[k] = z[k];
      slope[k] = both(1.f);
    } else {
      float2 e = z[k] * both(-kLog2e);
      e = make_float2(ex2(e.x), ex2(e.y));
      float2 s = e + both(1.f);
      s = make_float2(rcp(s.x), rcp(s.y));
      act[k] = KIND == 1 ? s : z[k] * s;
      if constexpr (SLOPE) {
        const float2 c = make_float2(fminf(e.x, 0x1p126f), fminf(e.y, 0x1p126f)) * s;
        slope[k] = KIND == 1 ? s * c : fma2(act[k], c, s);
      }
    }
  }
}
// The kind's branch once for all of them, so that their instructions interleave.
template <bool SLOPE, int H>
__device__ __forceinline__ void gate_of(const float2 (&z)[H], int kind, float2 (&act)[H],
                                        float2 (&slope)[H]) {
  if (kind == 0) {
    gate_kind<0, SLOPE>(z, act, slope);
  } else if (kind == 1) {
    gate_kind<1, SLOPE>(z, act, slope);
  } else {
    gate_kind<2, SLOPE>(z, act, slope);
  }
}
// One element.
struct Gate {
  float act, slope;
};
__device__ __forceinline__ Gate gate_of(float z, int kind) {
  const float2 v[1] = {both(z)};
  float2 act[1], slope[1];
  gate_of<true>(v, kind, act, slope);
  return {act[0].x, slope[0].x};
}

// A thread's elements of a row, VE of them a vector. ALIGNED: whole vectors, thread t the vectors t,
// t + threads, ...; otherwise single elements, t, t + threads, ..., so that a warp's stores are
// still one stretch.
template <typename T>
constexpr int kVecElements = 16 / static_cast<int>(sizeof(T));

template <int VE, int THREADS, bool ALIGNED>
__device__ __forceinline__ int row_element(int t, int k, int e) {
  return ALIGNED ? (k * THREADS + t) * VE + e : (k * VE + e) * THREADS + t;
}

// Bytes that a row of `elements` takes in shared memory. Where it is not aligned it is staged from the
// 16-byte boundary at or below its first element, one piece more.
template <typename T, int ELEMENTS, bool ALIGNED>
constexpr int kStagedRow = ELEMENTS * static_cast<int>(sizeof(T)) + (ALIGNED ? 0 : 16);

// Row `row` of an operand (rows and row distances in bytes fit 32 bits, their product need not).
template <typename T>
__device__ __forceinline__ T* row_of(T* base, unsigned row, int64_t ld) {
  using C = typename std::conditional<std::is_const<T>::value, const char, char>::type;
  return reinterpret_cast<T*>(reinterpret_cast<C*>(base) +
                              static_cast<uint64_t>(row) *
                                  (static_cast<unsigned>(ld) * static_cast<unsigned>(sizeof(T))));
}

// Copies piece `piece` (16 bytes) of the first `bytes` of a row into smem, zeros behind them (bytes ==
// 0: a row of zeros, nothing is read). Nothing in front of the operand is read.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void stage_piece(char* smem, const T* base, unsigned row, int64_t ld,
                                            int bytes, int piece) {
  const char* src = reinterpret_cast<const char*>(row_of(base, row, ld));
  const int shift = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
  const char* from = src - shift + piece * 16;
  int left = bytes == 0 ? 0 : bytes + shift - piece * 16;
  left = left < 0 ? 0 : (left > 16 ? 16 : left);
  if (ALIGNED || left == 0 || from >= reinterpret_cast<const char*>(base)) {
    cp_async_16(smem + piece * 16, from, left);
  } else {  // the boundary lies in front of the operand: its first elements one by one
    for (int b = shift; b < 16; b += static_cast<int>(sizeof(T)))
      *reinterpret_cast<T*>(smem + b) =
          b < shift + bytes ? *reinterpret_cast<const T*>(from + b) : from_f32<T>(0.f);
  }
}

// Stages one operand's ROWS rows for a group of threads, VE elements a thread and vector, row i at
// smem + i * distance. Where a vector has 8 bytes, two threads share a 16-byte piece and each copies
// one of their two vectors' pieces, so that with ALIGNED data a thread reads what its own warp copied.
template <typename T, int VE, int THREADS, int K, int ROWS, bool ALIGNED>
__device__ __forceinline__ void stage_rows(char* smem, int distance, const T* base, unsigned row0,
                                           unsigned rows, int64_t ld, int bytes, int t) {
  constexpr int kShare = 16 / (VE * static_cast<int>(sizeof(T)));  // threads of a piece: 1 or 2
  constexpr int kPieces = THREADS * K / kShare;                    // of a row
  static_assert(kShare == 1 || (ROWS == 1 && K == 2), "a thread for every piece");
  if constexpr (kShare == 1) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int n = row0 + i < rows ? bytes : 0;
#pragma unroll
      for (int k = 0; k < K; ++k)
        stage_piece<T, ALIGNED>(smem + i * distance, base, row0 + i, ld, n, k * THREADS + t);
      if (!ALIGNED && t == 0)
        stage_piece<T, ALIGNED>(smem + i * distance, base, row0 + i, ld, n, kPieces);
    }
  } else {
    // one row, each of the two threads the half of its vectors
    const int n = row0 < rows ? bytes : 0;
    stage_piece<T, ALIGNED>(smem, base, row0, ld, n, ((t & 1) * THREADS + t) / 2);
    if (!ALIGNED && t == 0) stage_piece<T, ALIGNED>(smem, base, row0, ld, n, kPieces);
  }
}

// H pairs of elements as stored.
template <typename T, int H>
struct alignas(sizeof(T) * 2 * H) PairVec {
  typename Pair<T>::type p[H];
};

// The thread's vector k of a staged row in FP32; `row` the row's address (its low bits are used).
template <typename T, int THREADS, bool ALIGNED, int H>
__device__ __forceinline__ void staged_vector(const char* smem, unsigned row, int t, int k,
                                              float2 (&v)[H]) {
  if constexpr (ALIGNED) {
    const auto q = *reinterpret_cast<const PairVec<T, H>*>(
        smem + (k * THREADS + t) * static_cast<int>(sizeof(PairVec<T, H>)));
#pragma unroll
    for (int e = 0; e < H; ++e) v[e] = to_f32(q.p[e]);
  } else {
    const T* at = reinterpret_cast<const T*>(smem + (row & 15u));
#pragma unroll
    for (int e = 0; e < H; ++e)
      v[e] = make_float2(to_f32(at[row_element<2 * H, THREADS, false>(t, k, 2 * e)]),
                         to_f32(at[row_element<2 * H, THREADS, false>(t, k, 2 * e + 1)]));
  }
}

template <typename T, int THREADS, bool ALIGNED, int H>
__device__ __forceinline__ void store_vector(T* row, int t, int k, int width,
                                             const float2 (&v)[H]) {
  const int at = row_element<2 * H, THREADS, ALIGNED>(t, k, 0);
  PairVec<T, H> q;
#pragma unroll
  for (int e = 0; e < H; ++e) q.p[e] = pair_from_f32<T>(v[e]);
  if (ALIGNED && at + 2 * H <= width) {
    *reinterpret_cast<PairVec<T, H>*>(row + at) = q;
    return;
  }
#pragma unroll
  for (int e = 0; e < H; ++e) {
    const int c = row_element<2 * H, THREADS, ALIGNED>(t, k, 2 * e),
              d = row_element<2 * H, THREADS, ALIGNED>(t, k, 2 * e + 1);
    if (c < width) row[c] = q.p[e].x;
    if (d < width) row[d] = q.p[e].y;
  }
}

// The vector's parameters (`fill` where they are absent, 0 behind the row's end); they stay in the
// first cache level over the rows that a block walks.
template <int THREADS, bool ALIGNED, int H>
__device__ __forceinline__ void load_params(const float* w, float fill, int t, int k, int width,
                                            float2 (&v)[H]) {
  const int at = row_element<2 * H, THREADS, ALIGNED>(t, k, 0);
  if (ALIGNED && w != nullptr && at + 2 * H <= width) {
#pragma unroll
    for (int e = 0; e < H; e += 2) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(w + at + 2 * e));
      v[e] = make_float2(q.x, q.y);
      v[e + 1] = make_float2(q.z, q.w);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < H; ++e) {
    const int c = row_element<2 * H, THREADS, ALIGNED>(t, k, 2 * e),
              d = row_element<2 * H, THREADS, ALIGNED>(t, k, 2 * e + 1);
    v[e].x = w == nullptr ? fill : (c < width ? __ldg(w + c) : 0.f);
    v[e].y = w == nullptr ? fill : (d < width ? __ldg(w + d) : 0.f);
  }
}

}  // namespace bsolve
