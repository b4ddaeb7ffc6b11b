// Element types of the row operators (bs_grec, bs_gnorm): storage in FP32, BF16 or FP16,
// arithmetic in FP32, one rounding (to nearest even) on the way out.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace bsolve {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// The low bits of an address.
__device__ __forceinline__ unsigned low_bits(const void* p) {
  return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p));
}

// Asynchronous copy to shared memory: 16 bytes of which the first `bytes` are read, the others zero (both addresses 16-byte aligned);
// past the first cache level.
__device__ __forceinline__ void cp_async_16(void* smem, const void* gmem, int bytes) {
  const unsigned d = static_cast<unsigned>(__cvta_generic_to_shared(smem));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(d), "l"(gmem), "r"(bytes)
               : "memory");
}

// Two neighbouring elements: as one value of twice the size, and in FP32.
template <typename T>
struct Pair;
template <>
struct Pair<float> {
  using type = float2;
};
template <>
struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
};
template <>
struct Pair<__half> {
  using type = __half2;
};

__device__ __forceinline__ float2 to_f32(float2 v) { return v; }
// A BF16 number is the upper half of the FP32 number of its value: one shift, one mask.
__device__ __forceinline__ float2 to_f32(__nv_bfloat162 v) {
  const unsigned u = *reinterpret_cast<const unsigned*>(&v);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ float2 to_f32(__half2 v) { return __half22float2(v); }

template <typename T>
__device__ __forceinline__ typename Pair<T>::type pair_from_f32(float2 v);
template <>
__device__ __forceinline__ float2 pair_from_f32<float>(float2 v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat162 pair_from_f32<__nv_bfloat16>(float2 v) {
  return __float22bfloat162_rn(v);
}
template <>
__device__ __forceinline__ __half2 pair_from_f32<__half>(float2 v) {
  return __float22half2_rn(v);
}

}  // namespace bsolve
