// The gate of the norms around a block and the rows' register layout (bs_gnorm calls).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "grec_math.cuh"
#include "row_types.cuh"

namespace bsolve {

struct Gate {
  float act, slope;  // act(z) and its derivative
};

// kind: a bs_gate. sigma(z) = 1 / (1 + e^-z); 1 - sigma(z) = e^-z sigma(z), and 1 where e^-z
// is beyond FP32. The approximate exponential and reciprocal are within 2 ulp.
__device__ __forceinline__ Gate gate_of(float z, int kind) {
  if (kind == 2) return {z, 1.f};
  const float e = ex2(z * -kLog2e);
  const float s = rcp(1.f + e);
  const float c = z < -80.f ? 1.f : e * s;
  if (kind == 1) return {s, s * c};
  return {z * s, fmaf(z * s, c, s)};
}

// A thread's elements of a row in registers: VE of them, K times, as stored. ALIGNED: 16-byte
// vectors, thread t the vectors t, t + threads, ...; otherwise single elements, thread t the
// elements t, t + threads, ..., so that a warp's loads are still one stretch.
template <typename T>
constexpr int kVecElements = 16 / static_cast<int>(sizeof(T));

template <typename T>
struct alignas(16) RowVec {
  T e[kVecElements<T>];
};

__device__ __forceinline__ uint4 load_streamed(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The element of the row that slot e of the thread's vector k holds.
template <typename T, int THREADS, bool ALIGNED>
__device__ __forceinline__ int row_element(int t, int k, int e) {
  constexpr int VE = kVecElements<T>;
  return ALIGNED ? (k * THREADS + t) * VE + e : (k * VE + e) * THREADS + t;
}

// Zeros where the row is absent or ends.
template <typename T, int THREADS, bool ALIGNED>
__device__ __forceinline__ RowVec<T> load_row(const T* row, int t, int k, int width) {
  constexpr int VE = kVecElements<T>;
  RowVec<T> v;
  const int at = row_element<T, THREADS, ALIGNED>(t, k, 0);
  if (ALIGNED && row != nullptr && at + VE <= width) {
    *reinterpret_cast<uint4*>(&v) = load_streamed(row + at);
    return v;
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const int c = row_element<T, THREADS, ALIGNED>(t, k, e);
    v.e[e] = row != nullptr && c < width ? row[c] : from_f32<T>(0.f);
  }
  return v;
}

template <typename T, int THREADS, bool ALIGNED>
__device__ __forceinline__ void store_row(T* row, int t, int k, int width, const float* v) {
  constexpr int VE = kVecElements<T>;
  const int at = row_element<T, THREADS, ALIGNED>(t, k, 0);
  RowVec<T> q;
#pragma unroll
  for (int e = 0; e < VE; ++e) q.e[e] = from_f32<T>(v[e]);
  if (ALIGNED && at + VE <= width) {
    *reinterpret_cast<uint4*>(row + at) = *reinterpret_cast<const uint4*>(&q);
    return;
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const int c = row_element<T, THREADS, ALIGNED>(t, k, e);
    if (c < width) row[c] = q.e[e];
  }
}

// The vector's parameters (`fill` where the vector is absent, 0 behind the row's end); they stay
// in the first cache level over the rows that a block walks.
template <typename T, int THREADS, bool ALIGNED>
__device__ __forceinline__ void load_params(const float* w, float fill, int t, int k, int width,
                                            float* v) {
  constexpr int VE = kVecElements<T>;
  const int at = row_element<T, THREADS, ALIGNED>(t, k, 0);
  if (ALIGNED && w != nullptr && at + VE <= width) {
#pragma unroll
    for (int e = 0; e < VE; e += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(w + at + e));
      v[e] = q.x, v[e + 1] = q.y, v[e + 2] = q.z, v[e + 3] = q.w;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const int c = row_element<T, THREADS, ALIGNED>(t, k, e);
    v[e] = w == nullptr ? fill : (c < width ? __ldg(w + c) : 0.f);
  }
}

}  // namespace bsolve
