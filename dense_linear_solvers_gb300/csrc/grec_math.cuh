// The gates of the gated linear recurrence (bs_grec calls) and the tape's layout.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bsolve {

constexpr int kTapeRows = 64;  // rows of a sequence between two states on the tape

// First tape row of the sequence that starts at row `start` and is number s: the sequences'
// parts do not overlap, since floor(b / 64) - floor(a / 64) + 1 >= ceil((b - a) / 64).
__host__ __device__ __forceinline__ int64_t tape_base(int64_t start, int64_t s) {
  return start / kTapeRows + s;
}

// Rows [start, end) of sequence s, clamped to the operand's rows.
__device__ __forceinline__ void sequence_rows(const int64_t* offsets, int64_t s, int64_t length,
                                              int64_t rows, int64_t* start, int64_t* end) {
  if (offsets == nullptr) {
    *start = s * length;
    *end = *start + length;
    return;
  }
  int64_t a = offsets[s], b = offsets[s + 1];
  a = a < 0 ? 0 : (a > rows ? rows : a);
  b = b < a ? a : (b > rows ? rows : b);
  *start = a;
  *end = b;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Minimum and maximum that hand a NaN on.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

constexpr float kLog2e = 1.44269504088896341f;

// Per channel: the rate K = kappa softplus(lam), so that l = -K sigma(r).
__device__ __forceinline__ float grec_rate(float lam, float kappa) {
  return kappa * (fmaxf(lam, 0.f) + log1pf(expf(-fabsf(lam))));
}

// d log(K) / d lam = sigma(lam) / softplus(lam): what turns the sum of D = dL/dl * l into the
// gradient of lam. Below -15 both functions are e^lam to FP32 accuracy.
__device__ __forceinline__ float grec_rate_slope(float lam) {
  if (lam < -15.f) return 1.f;
  const float e = expf(-fabsf(lam));
  const float sp = fmaxf(lam, 0.f) + log1pf(e);
  return (lam >= 0.f ? 1.f : e) / ((1.f + e) * sp);
}

// What one element's gates give.
//   er = e^-r, ei = e^-i, each at most 2^60, share one reciprocal of (1 + er)(1 + ei):
//     sigma(r) = (1 + ei) d,  1 - sigma(r) = er sigma(r), without cancellation. The bound keeps
//     the product finite; sigma(r) is taken 2^-60 lower, so that a gate of -inf closes (a = 1,
//     s = 0 up to 2^-40: the row hands its state on).
//   a = exp(l) and 1 - a^2 both come from E = exp(l) - 1, since near a = 1 (long memory)
//     1 - a^2 = -E (1 + a) keeps its digits while 1 - a*a loses them: l = n ln 2 + f with
//     |f| <= ln 2 / 2, E = 2^n (e^f - 1) + (2^n - 1), e^f - 1 by its Taylor sum to f^7 (the
//     next term is f^8 / 40320, 2e-8 of f at the end of the range). l is bounded at -80, where
//     a is 2e-35.
//   s = sqrt(1 - a^2) = w rsqrt(w), l / s = l rsqrt(w) with w >= 2^-80, where both are below
//     2^-40 of full scale.
// The approximate exponential, reciprocal and root are within 2 ulp of FP32 (2^-22), two
// orders below a 16-bit output's rounding and near that of one FP32 operation.
// Two neighbouring channels at a time: the products and sums are FP32 pair instructions.
struct Gates {
  float2 a, s, sr, si, er, ei, l, rs;
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 operator*(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 operator+(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return __ffma2_rn(a, b, c);
}

// e^-v, at most 2^60.
__device__ __forceinline__ float2 bounded_exp_neg(float2 v) {
  v = v * both(-kLog2e);
  return make_float2(ex2(min_nan(v.x, 60.f)), ex2(min_nan(v.y, 60.f)));
}

// From er and ei; neg_rate: -K of the two channels.
__device__ __forceinline__ Gates grec_gates_from(float2 er, float2 ei, float2 neg_rate) {
  Gates g;
  g.er = er;
  g.ei = ei;
  const float2 p = g.er + both(1.f), q = g.ei + both(1.f);
  float2 d = p * q;
  d = make_float2(rcp(d.x), rcp(d.y));
  g.sr = fma2(q, d, both(-0x1p-60f));
  g.si = p * d;
  g.l = neg_rate * g.sr;
  g.l = make_float2(max_nan(g.l.x, -80.f), max_nan(g.l.y, -80.f));
  const float2 t = fma2(g.l, both(kLog2e), both(12582912.f));  // 1.5 * 2^23: n in the low bits
  const float2 n = t + both(-12582912.f);
  float2 f = fma2(n, both(-0.693359375f), g.l);  // ln 2 in two parts, the first exact * n
  f = fma2(n, both(2.12194440e-4f), f);
  float2 e = fma2(f, both(1.f / 5040.f), both(1.f / 720.f));
  e = fma2(f, e, both(1.f / 120.f));
  e = fma2(f, e, both(1.f / 24.f));
  e = fma2(f, e, both(1.f / 6.f));
  e = fma2(f, e, both(0.5f));
  e = fma2(f * f, e, f);
  const float2 two_n = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                                   __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));
  const float2 E = fma2(two_n, e, two_n + both(-1.f));
  g.a = E + both(1.f);
  float2 w = fma2(E, g.a, E);  // E (1 + a) = a^2 - 1
  w = make_float2(max_nan(-w.x, 0x1p-80f), max_nan(-w.y, 0x1p-80f));
  g.rs = make_float2(rsqrt_fast(w.x), rsqrt_fast(w.y));
  g.s = w * g.rs;
  return g;
}

__device__ __forceinline__ Gates grec_gates(float2 r, float2 i, float2 neg_rate) {
  return grec_gates_from(bounded_exp_neg(r), bounded_exp_neg(i), neg_rate);
}

}  // namespace bsolve
