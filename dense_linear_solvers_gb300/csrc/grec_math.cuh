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
struct Gates {
  float a, s, sr, si, er, ei, l, rs;
};

__device__ __forceinline__ Gates grec_gates(float r, float i, float rate) {
  Gates g;
  g.er = ex2(min_nan(r * -kLog2e, 60.f));
  g.ei = ex2(min_nan(i * -kLog2e, 60.f));
  const float p = 1.f + g.er, q = 1.f + g.ei;
  const float d = rcp(p * q);
  g.sr = fmaf(q, d, -0x1p-60f);
  g.si = p * d;
  g.l = max_nan(-rate * g.sr, -80.f);
  const float t = fmaf(g.l, kLog2e, 12582912.f);  // 1.5 * 2^23: n in the low bits
  const float n = t - 12582912.f;
  float f = fmaf(n, -0.693359375f, g.l);          // ln 2 in two parts, the first exact * n
  f = fmaf(n, 2.12194440e-4f, f);
  float e = fmaf(f, 1.f / 5040.f, 1.f / 720.f);
  e = fmaf(f, e, 1.f / 120.f);
  e = fmaf(f, e, 1.f / 24.f);
  e = fmaf(f, e, 1.f / 6.f);
  e = fmaf(f, e, 0.5f);
  e = fmaf(f * f, e, f);
  const float two_n = __int_as_float((__float_as_int(t) << 23) + 0x3f800000);
  const float E = fmaf(two_n, e, two_n - 1.f);
  g.a = 1.f + E;
  const float w = max_nan(-E * (1.f + g.a), 0x1p-80f);
  g.rs = rsqrt_fast(w);
  g.s = w * g.rs;
  return g;
}

}  // namespace bsolve
