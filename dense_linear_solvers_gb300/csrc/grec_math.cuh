// The gates of the gated linear recurrence (bs_grec calls) and the tape's layout.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bsolve {

constexpr int kTapeRows = 32;  // rows of a sequence between two states on the tape

// First tape row of the sequence that starts at row `start` and is number s: the sequences'
// parts do not overlap, since floor(b / 32) - floor(a / 32) + 1 >= ceil((b - a) / 32).
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
// The minimum, or NaN where either is one.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
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

// What one element's gates give, with l = -t:
//   sigma(r) = 1 / (1 + e^-r); 1 - sigma(r) = e^-r sigma(r), without cancellation where e^-r is
//     kept finite (grec_exp_neg<true>, at most 2^100: the sigma below is then 2^-100, not 0).
//   1 - a^2 comes from m = 1 - e^-t, since near a = 1 (long memory) 1 - a^2 = m (1 + a) keeps its
//     digits while 1 - a*a loses them. SMALL (rate at most kSmallRate, so that a >= 0.6): m =
//     t - t^2 q(t), q the polynomial of degree 3 with the least relative error of m on [0, 0.5],
//     2^-24, and a = 1 - m. Otherwise t = n ln 2 + f with |f| <= ln 2 / 2 (Cody and Waite: n rounded
//     by adding 1.5 * 2^23, ln 2 in two parts), e = 1 - e^-f = f - f^2 q(f), q of degree 4 (2^-27),
//     m = (1 - 2^-n) + 2^-n e and a = 2^-n - 2^-n e: taken from m, a small a would keep the
//     digits of 1 only (6% off at t = 16, 0 from t = 17 on). t is bounded at 80, where a is 2e-35.
//     On 16,384 x 4,096 BF16 rows the two forward passes take 119 and 129 us, 28 and 35
//     instructions an element (m and a in paired instructions, the sign of e in one of its own: 134 us).
//   2^-124 more in t, which no other value notices, keeps the root below away from 0 / 0:
//   s = sqrt(1 - a^2) = w rsqrt(w), t / s = t rsqrt(w).
// The approximate exponential, reciprocal and root are within 2 ulp of FP32 (2^-22), two
// orders below a 16-bit output's rounding and near that of one FP32 operation.
constexpr float kSmallRate = 0.5f;

// Two neighbouring channels at a time: the products and sums are FP32 pair instructions.
struct Gates {
  float2 a, s, sr, si, t, rs;  // decay, root, sigma(r), sigma(i), -l, 1 / root
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 operator*(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 operator+(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return __ffma2_rn(a, b, c);
}

// e^-v; BOUNDED: at most 2^100.
template <bool BOUNDED>
__device__ __forceinline__ float2 grec_exp_neg(float2 v) {
  v = v * both(-kLog2e);
  if (BOUNDED) v = make_float2(min_nan(v.x, 100.f), min_nan(v.y, 100.f));
  return make_float2(ex2(v.x), ex2(v.y));
}

// From e^-r, e^-i and the rates K of the two channels.
template <bool SMALL>
__device__ __forceinline__ Gates grec_gates(float2 er, float2 ei, float2 rate) {
  Gates g;
  const float2 p = er + both(1.f), q = ei + both(1.f);
  g.sr = make_float2(rcp(p.x), rcp(p.y));
  g.si = make_float2(rcp(q.x), rcp(q.y));
  g.t = fma2(rate, g.sr, both(0x1p-124f));
  float2 m;
  if constexpr (SMALL) {
    const float2 t = g.t;
    float2 c = fma2(t, both(6.7512975e-3f), both(-4.0983321e-2f));  // -q(t)
    c = fma2(t, c, both(1.6654362e-1f));
    c = fma2(t, c, both(-4.9999245e-1f));
    m = fma2(t * t, c, t);
    g.a = fma2(m, both(-1.f), both(1.f));
  } else {
    g.t = make_float2(min_nan(g.t.x, 80.f), min_nan(g.t.y, 80.f));
    const float2 k = fma2(g.t, both(-kLog2e), both(12582912.f));  // 1.5 * 2^23: -n in the low bits
    const float2 n = k + both(-12582912.f);
    float2 f = fma2(n, both(0.693359375f), g.t);  // ln 2 in two parts, the first exact * n
    f = fma2(n, both(-2.12194440e-4f), f);
    float2 c = fma2(f, both(-1.3459974e-3f), both(8.3572877e-3f));  // -q(f)
    c = fma2(f, c, both(-4.1672192e-2f));
    c = fma2(f, c, both(1.6666666e-1f));
    c = fma2(f, c, both(-0.5f));
    const float2 e = fma2(f * f, c, f);
    const float2 two_n = make_float2(__int_as_float((__float_as_int(k.x) << 23) + 0x3f800000),
                                     __int_as_float((__float_as_int(k.y) << 23) + 0x3f800000));
    m = make_float2(fmaf(two_n.x, e.x, 1.f - two_n.x), fmaf(two_n.y, e.y, 1.f - two_n.y));
    g.a = make_float2(fmaf(-two_n.x, e.x, two_n.x), fmaf(-two_n.y, e.y, two_n.y));
  }
  const float2 w = fma2(m, g.a, m);
  g.rs = make_float2(rsqrt_fast(w.x), rsqrt_fast(w.y));
  g.s = w * g.rs;
  return g;
}

}  // namespace bsolve
