// The norms around a block with its gate and residual scale (bs_gnorm calls of bsolve.h): kernels and
// launchers, one instance a row type (gnorm_f32.cu, gnorm_bf16.cu, gnorm_f16.cu).
//
// A row belongs to a group of 8 to 1024 threads, each with K vectors of it; a group takes ROWS rows
// at a time, and persistent blocks walk all of them. Each thread copies its own vectors of the rows of the
// next turn into shared memory with cp.async while it works on these, so that the loads need no
// registers and no barrier, and reads them as often as it needs them; the rows' sums go through shuffles
// and, for groups of several warps, one barrier for all rows of the turn, the last sums of a turn
// together with the first of the next. The parameters stay in the first cache level. The backward pass
// keeps its three sums over rows in registers, every thread those of its own columns, and each
// block writes one part of them at its end; a second kernel adds the parts in order. Rows too long for
// that run the looped kernels at the end, which read a row once for each mean and once for the
// outputs.
//
// 16,384 x 4,096 BF16: forward 112 us (6.0 TB/s of its five operands, 89% of a copy's rate), backward 233
// us (4.6 TB/s of its eight; one block of 512 threads an SM, which waits at its two reductions a turn).
// Measured without gain there: every sum in one reduction by expanding sum y^2 (296 against 279 at the
// time), four elements a thread and twice the warps (279), two vectors a thread and one row (340).
#pragma once

#include <type_traits>

#include <cuda_fp8.h>

#include "gnorm_math.cuh"
#include "gnorm_shapes.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {
namespace {

constexpr int kTurns = 2;  // turns of rows in shared memory: this one and the next

// Sums of N values (a power of two) over a group's threads, the same bits in all of them. While
// lanes hold several values, a step hands half of them to the lanes across and keeps the other
// half, so that N values take few more shuffles than one; then lane part k of a warp holds value k's
// sum. The warps' sums meet in `red`, [2][WARPS][N] and, behind that, [WARPS][N]; consecutive calls
// take its two halves in turn, so that one barrier a call is enough.
template <int N, int THREADS>
constexpr int kRedFloats = THREADS > 32 ? 3 * N * (THREADS / 32) : 1;

template <int N, int THREADS>
__device__ __forceinline__ void group_sums(float (&v)[N], float* red, int& turn) {
  constexpr int LANES = THREADS < 32 ? THREADS : 32, WARPS = THREADS / LANES;
  constexpr unsigned kAll = 0xFFFFFFFFu;
  static_assert(N <= LANES, "a lane part for every value");
  const int lane = threadIdx.x & 31;
  int m = LANES / 2;
#pragma unroll
  for (int n = N / 2; n > 0; n >>= 1, m >>= 1) {
    const bool high = lane & m;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float keep = high ? v[k + n] : v[k], give = high ? v[k] : v[k + n];
      v[k] = keep + __shfl_xor_sync(kAll, give, m);
    }
  }
  float s = v[0];
#pragma unroll
  for (; m > 0; m >>= 1) s += __shfl_xor_sync(kAll, s, m);
  if constexpr (WARPS == 1) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      v[k] = N == 1 ? s : __shfl_sync(kAll, s, (lane & ~(LANES - 1)) + k * (LANES / N));
  } else {
    const int warp = threadIdx.x >> 5;
    float* r = red + turn * (WARPS * N);
    turn ^= 1;
    if (lane % (32 / N) == 0) r[warp * N + lane / (32 / N)] = s;
    __syncthreads();
    constexpr int PARTS = 32 / N;  // lanes that add up one value
    const int value = lane % N, part = lane / N;
    s = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; w += PARTS)
      if (WARPS % PARTS == 0 || w + part < WARPS) s += r[(w + part) * N + value];
#pragma unroll
    for (int q = N; q < 32; q <<= 1) s += __shfl_xor_sync(kAll, s, q);
    if constexpr (N <= 2) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = N == 1 ? s : __shfl_sync(kAll, s, k);
    } else {
      float* own = red + (2 * WARPS + warp) * N;
      if (lane < N) own[lane] = s;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const float4 q = *reinterpret_cast<const float4*>(own + k);
        v[k] = q.x, v[k + 1] = q.y, v[k + 2] = q.z, v[k + 3] = q.w;
      }
    }
  }
}

// 1 / sqrt(v) for v > 0: the approximate root with one Newton step. Below 2^-100 (rows of zeros under a
// small eps, subnormal numbers included) that of v 2^100, so that neither the root, which takes a
// subnormal number for 0, nor the step loses digits.
__device__ __forceinline__ float inverse_root(float v) {
  const bool low = v < 0x1p-100f;
  if (low) v *= 0x1p100f;
  const float r = rsqrt_fast(v);
  const float s = r == 0.f ? r : fmaf(r * 0.5f, fmaf(-v * r, r, 1.f), r);  // 0 where v overflowed
  return low ? s * 0x1p50f : s;
}

template <int THREADS>
struct Group {
  static constexpr int kBlock = THREADS <= 32 ? 128 : THREADS;
  static constexpr int kGroups = kBlock / THREADS;
};

// How a call's operands lie. kFull: every operand there, 16-byte bases, row distances and widths; kAligned:
// 16-byte bases and row distances; kAny.
enum Mode : int { kFull = 0, kAligned = 1, kAny = 2 };

// ------------------------------------------------------------------ output in 8 bits
// bs_gnorm_q8_batched: the row's last value v (u, or y without a norm behind it) as e4m3 numbers v / s under
// one scale s = max(max |v|, 2^-100) / 448 for each 128 elements. The largest magnitude goes through integer
// maxima of the numbers' bits, which order them and keep a NaN.
constexpr int kScaled = 128;  // elements under one scale

__device__ __forceinline__ unsigned magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ float scale_of(unsigned top) {
  return __fdiv_rn(__uint_as_float(max(top, __float_as_uint(0x1p-100f))), 448.f);
}
// Quotients by the scale that is stored: a product with the rounded inverse alone would put values near the middle of
// two e4m3 numbers on the other side. The product is corrected once by its remainder (Markstein's method), two
// instructions for two numbers (16,384 x 4,096 BF16, all operands: 109.8 us, 107.8 without, 122.2 with __fdiv_rn).
struct Divisor {
  float s, inverse;
};
// (an infinite scale: the inverse is 0, and with 0 for the scale the remainder of a finite number is none of NaN)
__device__ __forceinline__ Divisor divisor(float s) {
  return {s == __int_as_float(0x7F800000) ? 0.f : s, __fdiv_rn(1.f, s)};
}
__device__ __forceinline__ float2 quotient(float2 v, const Divisor& by) {
  const float2 q = v * both(by.inverse), rest = fma2(q, both(-by.s), v);
  return fma2(rest, both(by.inverse), q);
}
__device__ __forceinline__ unsigned as_e4m3(float2 v) {
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

// The numbers of ROWS rows and where they go. `tops`, [ROWS][blocks], is shared memory of the group, used
// where a thread's elements lie apart (kAny).
template <int H, int K, int THREADS, int MODE>
struct Quantise {
  static constexpr int VE = 2 * H;
  static constexpr int kBlocks = THREADS * K * VE < kScaled ? 1 : THREADS * K * VE / kScaled;
  static constexpr int kLanes = kScaled / VE < THREADS ? kScaled / VE : THREADS;  // of a scale

  // Threads of a group wait for each other.
  static __device__ __forceinline__ void meet() {
    if (THREADS > 32) __syncthreads(); else __syncwarp();
  }

  template <int ROWS>
  static __device__ __forceinline__ void put(const Bytes8& out, unsigned row0, unsigned rows, int t,
                                             int width, const float2 (&v)[ROWS][K][H],
                                             unsigned* tops) {
    if constexpr (MODE != kAny) {
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          unsigned top = 0;
#pragma unroll
          for (int e = 0; e < H; ++e)
            top = max(top, max(magnitude(v[i][k][e].x), magnitude(v[i][k][e].y)));
#pragma unroll
          for (int m = 1; m < kLanes; m *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
          const float s = scale_of(top);
          const Divisor by = divisor(s);
          const int at = (k * THREADS + t) * VE;
          if (row0 + i >= rows || at >= width) continue;
          const unsigned row = row0 + i;
          if (at % kScaled == 0) out.s[row * out.lds + at / kScaled] = s;
          unsigned w[H / 2];
#pragma unroll
          for (int e = 0; e < H; e += 2)
            w[e / 2] = as_e4m3(quotient(v[i][k][e], by)) | as_e4m3(quotient(v[i][k][e + 1], by)) << 16;
          uint8_t* to = out.q + row * out.ldq + at;
          if (MODE == kFull || at + VE <= width) {
            if constexpr (H == 4) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<unsigned*>(to) = w[0];
          } else {
            for (int e = 0; e < width - at; ++e) to[e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e % 4)));
          }
        }
    } else {
      for (int j = t; j < ROWS * kBlocks; j += THREADS) tops[j] = 0;
      meet();
#pragma unroll
      for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float x = e & 1 ? v[i][k][e / 2].y : v[i][k][e / 2].x;
            const int c = row_element<VE, THREADS, false>(t, k, e);
            if (c < width) atomicMax(&tops[i * kBlocks + c / kScaled], magnitude(x));
          }
      meet();
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        if (row0 + i >= rows) continue;
        const unsigned row = row0 + i;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float x = e & 1 ? v[i][k][e / 2].y : v[i][k][e / 2].x;
            const int c = row_element<VE, THREADS, false>(t, k, e);
            if (c >= width) continue;
            const float s = scale_of(tops[i * kBlocks + c / kScaled]);
            out.q[row * out.ldq + c] = static_cast<uint8_t>(as_e4m3(make_float2(__fdiv_rn(x, s), 0.f)));
            if (c % kScaled == 0) out.s[row * out.lds + c / kScaled] = s;
          }
      }
      meet();
    }
  }
};

// ------------------------------------------------------------------ forward

// One group's thread and its part of a row: VE = 2 H elements a vector, K vectors.
template <typename T, int H, int K, int THREADS, int ROWS, int MODE>
struct Part {
  static constexpr bool kAl = MODE != kAny;
  static constexpr int VE = 2 * H;
  // a thread reads its own copies; otherwise its warp's, or (kAny) its block's
  static constexpr bool kPrivate = kAl && VE * sizeof(T) == 16;
  static constexpr int kRow = kStagedRow<T, VE * THREADS * K, kAl>;

  // Stages ROWS rows of one operand from row `from`, `distance` apart.
  static __device__ __forceinline__ void stage(char* to, int distance, const T* base, unsigned from,
                                               unsigned rows, int64_t ld, int bytes, int t) {
    if constexpr (MODE == kFull && kPrivate) {
      const unsigned pitch = static_cast<unsigned>(ld) * static_cast<unsigned>(sizeof(T));
      if (from + ROWS <= rows) {
        const char* src = reinterpret_cast<const char*>(base) + t * 16 +
                          static_cast<uint64_t>(from) * pitch;
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const int at = (k * THREADS + t) * 16;
            cp_async_16(to + i * distance + at, src + i * static_cast<uint64_t>(pitch) + k * THREADS * 16,
                        at < bytes ? 16 : 0);
          }
        return;
      }
    }
    if (MODE == kFull || base)
      stage_rows<T, VE, THREADS, K, ROWS, kAl>(to, distance, base, from, rows, ld, bytes, t);
  }

  // Asks for a turn's rows of one operand to come into the second cache level, a line (128 bytes) a
  // thread.
  static __device__ __forceinline__ void prefetch(const T* base, unsigned from, unsigned rows,
                                                  int64_t ld, int bytes, int t) {
    if (MODE != kFull && !base) return;
    constexpr int kLines = THREADS * K * VE * static_cast<int>(sizeof(T)) / 128;
    if constexpr (kLines >= 1) {
      const int i = ROWS == 2 ? t / (THREADS / 2) : 0, line = t % (THREADS / ROWS);
      if (line < kLines && line * 128 < bytes && from + i < rows)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            reinterpret_cast<const char*>(row_of(base, from + i, ld)) + line * 128));
    }
  }

  // Parameters of vector k; `fill` where the vector is absent, 0 behind the row's end.
  static __device__ __forceinline__ void params(const float* w, float fill, int t, int k, int width,
                                                float2 (&v)[H]) {
    if constexpr (MODE == kFull) {
      const int at = (k * THREADS + t) * VE;
      if (at < width) {
#pragma unroll
        for (int e = 0; e < H; e += 2) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(w + at + 2 * e));
          v[e] = make_float2(q.x, q.y);
          v[e + 1] = make_float2(q.z, q.w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < H; ++e) v[e] = both(0.f);
      }
    } else {
      load_params<THREADS, kAl>(w, fill, t, k, width, v);
    }
  }

  static __device__ __forceinline__ void store(T* base, unsigned row, int64_t ld, int t, int k,
                                               int width, const float2 (&v)[H]) {
    if constexpr (MODE == kFull) {
      const int at = (k * THREADS + t) * VE;
      PairVec<T, H> q;
#pragma unroll
      for (int e = 0; e < H; ++e) q.p[e] = pair_from_f32<T>(v[e]);
      if (at < width) *reinterpret_cast<PairVec<T, H>*>(row_of(base + at, row, ld)) = q;
    } else {
      store_vector<T, THREADS, kAl>(row_of(base, row, ld), t, k, width, v);
    }
  }

  // Waits between copies and reads, and between reads and the copies that overwrite them.
  static __device__ __forceinline__ void meet() {
    if constexpr (!kPrivate) {
      if (!kAl && THREADS > 32) __syncthreads(); else __syncwarp();
    }
  }
};

// Q8: u goes out in 8 bits, to `bytes8`.
template <typename T, int H, int K, int THREADS, int ROWS, int MODE, bool Q8>
__global__ void __launch_bounds__(Group<THREADS>::kBlock, 1024 / Group<THREADS>::kBlock)
gnorm_kernel(GnormRows<T> p, T* __restrict__ y, int64_t ldy, T* __restrict__ u, int64_t ldu,
             Bytes8 bytes8) {
  using G = Group<THREADS>;
  using P = Part<T, H, K, THREADS, ROWS, MODE>;
  constexpr int kRow = P::kRow;
  constexpr bool kAll = MODE == kFull;
  __shared__ __align__(16) float red[kRedFloats<2 * ROWS, THREADS>];
  extern __shared__ __align__(16) char shared[];
  const int t = threadIdx.x % THREADS, group = threadIdx.x / THREADS;
  char* mine = shared + group * (kTurns * ROWS * 3 * kRow);
  const float inv = 1.f / p.width;
  const int bytes = p.width * static_cast<int>(sizeof(T));
  const unsigned rows = static_cast<unsigned>(p.rows);  // at most 2^30
  const unsigned turn_rows = gridDim.x * (G::kGroups * ROWS);
  unsigned row0 = (blockIdx.x * G::kGroups + group) * ROWS;
  int turn = 0;

  auto one = [&](char* to, const T* base, int64_t ld, unsigned from) {
    P::stage(to, 3 * kRow, base, from, rows, ld, bytes, t);
  };
  auto stage = [&](unsigned from, int slot) {
    char* to = mine + slot * ROWS * 3 * kRow;
    one(to, p.f, p.ldf, from);
    one(to + kRow, p.z, p.ldz, from);
    one(to + 2 * kRow, p.x, p.ldx, from);
    cp_async_commit();
  };
  // sum f^2 of the rows of a turn
  auto squares = [&](int slot, unsigned from, float* out) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      float2 sum = both(0.f);
      if (kAll || p.w_post)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float2 v[H];
          staged_vector<T, THREADS, P::kAl>(mine + (slot * ROWS + i) * 3 * kRow,
                                            low_bits(row_of(p.f, from + i, p.ldf)), t, k, v);
#pragma unroll
          for (int e = 0; e < H; ++e) sum = fma2(v[e], v[e], sum);
        }
      out[i] = sum.x + sum.y;
    }
  };
  // One reduction a turn: this turn's sum y^2 goes with the next turn's sum f^2.
  stage(row0, 0);
  stage(row0 + turn_rows, 1);
  cp_async_wait_group<1>();
  P::meet();
  float s[2 * ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) s[i] = 0.f;
  squares(0, row0, s + ROWS);
  group_sums<2 * ROWS, THREADS>(s, red, turn);
  int slot = 0;
  // the same number of turns for all groups of a block: the shuffles take whole warps
  for (unsigned at = blockIdx.x * (G::kGroups * ROWS); at < rows; at += turn_rows, row0 += turn_rows) {
    const char* in = mine + slot * ROWS * 3 * kRow;
    float r1[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      r1[i] = kAll || p.w_post ? inverse_root(fmaf(s[ROWS + i], inv, p.eps)) : 1.f;
    float2 v[ROWS][K][H];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 w[H], c[H];
      P::params(p.w_post, 1.f, t, k, p.width, w);
      P::params(p.scale, 1.f, t, k, p.width, c);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const char* at_row = in + i * 3 * kRow;
        float2 q[H];
        staged_vector<T, THREADS, P::kAl>(at_row, low_bits(row_of(p.f, row0 + i, p.ldf)), t, k, q);
#pragma unroll
        for (int e = 0; e < H; ++e) v[i][k][e] = q[e] * both(r1[i]) * w[e];
        if (kAll || p.z) {
          staged_vector<T, THREADS, P::kAl>(at_row + kRow, low_bits(row_of(p.z, row0 + i, p.ldz)), t,
                                             k, q);
          float2 act[H], none[H];
          gate_of<false>(q, p.gate, act, none);
#pragma unroll
          for (int e = 0; e < H; ++e) v[i][k][e] = v[i][k][e] * act[e];
        }
        if (kAll || p.x) {
          staged_vector<T, THREADS, P::kAl>(at_row + 2 * kRow, low_bits(row_of(p.x, row0 + i, p.ldx)),
                                             t, k, q);
#pragma unroll
          for (int e = 0; e < H; ++e) v[i][k][e] = fma2(v[i][k][e], c[e], q[e]);
        } else {
#pragma unroll
          for (int e = 0; e < H; ++e) v[i][k][e] = v[i][k][e] * c[e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      float2 sum = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < H; ++e) sum = fma2(v[i][k][e], v[i][k][e], sum);
        if ((kAll || y) && row0 + i < rows)
          P::store(y, row0 + i, ldy, t, k, p.width, v[i][k]);
      }
      s[i] = sum.x + sum.y;
    }
    cp_async_wait_group<0>();
    P::meet();
    squares(slot ^ 1, row0 + turn_rows, s + ROWS);
    group_sums<2 * ROWS, THREADS>(s, red, turn);
    P::meet();  // every thread has read its rows before they are overwritten
    stage(row0 + 2 * turn_rows, slot);
    slot ^= 1;
    if constexpr (Q8) {
      if (kAll || p.w_pre) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float2 w[H];
          P::params(p.w_pre, 1.f, t, k, p.width, w);
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            const float r = inverse_root(fmaf(s[i], inv, p.eps));
#pragma unroll
            for (int e = 0; e < H; ++e) v[i][k][e] = v[i][k][e] * (both(r) * w[e]);
          }
        }
      }
      using Q = Quantise<H, K, THREADS, MODE>;
      __shared__ unsigned tops[MODE == kAny ? G::kGroups * ROWS * Q::kBlocks : 1];
      Q::template put<ROWS>(bytes8, row0, rows, t, p.width, v,
                            tops + (MODE == kAny ? group * ROWS * Q::kBlocks : 0));
      continue;
    }
    if (!kAll && !u) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 w[H];
      P::params(p.w_pre, 1.f, t, k, p.width, w);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float r = inverse_root(fmaf(s[i], inv, p.eps));
        float2 q[H];
#pragma unroll
        for (int e = 0; e < H; ++e) q[e] = v[i][k][e] * (both(r) * w[e]);
        if (row0 + i < rows) P::store(u, row0 + i, ldu, t, k, p.width, q);
      }
    }
  }
  cp_async_wait_all();
}

// ------------------------------------------------------------------ backward
//
// With n = f r1 (r1 = 1 / rms(f)), t = n w_post act(z), y = x + scale t, q = r2 = 1 / rms(y):
//   dx = dy + q du w_pre - y q^3 mean(du w_pre y),     dt = dx scale,
//   dz = dt n w_post act'(z),  dn = dt act(z) w_post,  df = r1 (dn - n mean(dn n)),
//   dw_pre = sum du y q,  dscale = sum dx t,  dw_post = sum dt act(z) n.
template <typename T, int H, int K, int THREADS, int ROWS, int MODE>
__global__ void __launch_bounds__(Group<THREADS>::kBlock,
                                  (K * ROWS * H == 8 ? 512 : 1024) / Group<THREADS>::kBlock)
gnorm_backward_kernel(GnormRows<T> p, GnormGrads<T> g, float* __restrict__ partial) {
  using G = Group<THREADS>;
  using P = Part<T, H, K, THREADS, ROWS, MODE>;
  constexpr int kRow = P::kRow;
  constexpr bool kAll = MODE == kFull;
  __shared__ __align__(16) float red[kRedFloats<2 * ROWS, THREADS>];
  __shared__ __align__(16) float red2[kRedFloats<2 * ROWS, THREADS>];
  extern __shared__ __align__(16) char shared[];
  const int t = threadIdx.x % THREADS, group = threadIdx.x / THREADS;
  char* mine = shared + group * (kTurns * ROWS * 5 * kRow);
  const float inv = 1.f / p.width;
  const int bytes = p.width * static_cast<int>(sizeof(T));
  const unsigned rows = static_cast<unsigned>(p.rows);  // at most 2^30
  const unsigned turn_rows = gridDim.x * (G::kGroups * ROWS);
  unsigned row0 = (blockIdx.x * G::kGroups + group) * ROWS;
  int turn = 0, turn2 = 0;
  float2 sw[K][H], sc[K][H], sp[K][H];  // the sums dw_post, dscale, dw_pre
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < H; ++e) sw[k][e] = sc[k][e] = sp[k][e] = both(0.f);

  auto one = [&](char* to, const T* base, int64_t ld, unsigned from) {
    P::stage(to, 5 * kRow, base, from, rows, ld, bytes, t);
  };
  auto stage = [&](unsigned from, int slot) {
    char* to = mine + slot * ROWS * 5 * kRow;
    one(to, p.f, p.ldf, from);
    one(to + kRow, p.z, p.ldz, from);
    one(to + 2 * kRow, p.x, p.ldx, from);
    one(to + 3 * kRow, g.dy, g.lddy, from);
    one(to + 4 * kRow, g.du, g.lddu, from);
    cp_async_commit();
  };
  auto squares = [&](int slot, unsigned from, float* out) {  // sum f^2 of the rows of a turn
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      float2 sum = both(0.f);
      if (kAll || p.w_post)
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float2 v[H];
          staged_vector<T, THREADS, P::kAl>(mine + (slot * ROWS + i) * 5 * kRow,
                                            low_bits(row_of(p.f, from + i, p.ldf)), t, k, v);
#pragma unroll
          for (int e = 0; e < H; ++e) sum = fma2(v[e], v[e], sum);
        }
      out[i] = sum.x + sum.y;
    }
  };
  // Two reductions a turn: the second's sum dn n goes with the next turn's sum f^2.
  stage(row0, 0);
  stage(row0 + turn_rows, 1);
  cp_async_wait_group<1>();
  P::meet();
  float s[2 * ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) s[i] = 0.f;
  squares(0, row0, s + ROWS);
  group_sums<2 * ROWS, THREADS>(s, red, turn);
  int slot = 0;
  for (unsigned at = blockIdx.x * (G::kGroups * ROWS); at < rows; at += turn_rows, row0 += turn_rows) {
    const char* in = mine + slot * ROWS * 5 * kRow;
    if constexpr (THREADS >= 512) {
      // The one block that an SM holds asks for a turn's rows only when the last turn's are read, so late
      // that it waits for them; from the second cache level it does not (16,384 x 4,096 BF16: 275
      // to 239 us; with more blocks an SM, or in the forward pass, this costs 3 to 10%).
      const unsigned later = row0 + 2 * turn_rows;
      P::prefetch(p.f, later, rows, p.ldf, bytes, t);
      P::prefetch(p.z, later, rows, p.ldz, bytes, t);
      P::prefetch(p.x, later, rows, p.ldx, bytes, t);
      P::prefetch(g.dy, later, rows, g.lddy, bytes, t);
      P::prefetch(g.du, later, rows, g.lddu, bytes, t);
    }
    auto read = [&](int operand, const T* base, int64_t ld, int i, int k, float2 (&v)[H]) {
      staged_vector<T, THREADS, P::kAl>(in + (i * 5 + operand) * kRow,
                                         low_bits(row_of(base, row0 + i, ld)), t, k, v);
    };
    float r1[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      r1[i] = kAll || p.w_post ? inverse_root(fmaf(s[ROWS + i], inv, p.eps)) : 1.f;
    float2 y[ROWS][K][H];
    float r2[ROWS], back[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) r2[i] = back[i] = 0.f;
    if (kAll || g.du) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float2 w[H], c[H];
        P::params(p.w_post, 1.f, t, k, p.width, w);
        P::params(p.scale, 1.f, t, k, p.width, c);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          float2 q[H];
          read(0, p.f, p.ldf, i, k, q);
#pragma unroll
          for (int e = 0; e < H; ++e) y[i][k][e] = q[e] * both(r1[i]) * w[e];
          if (kAll || p.z) {
            read(1, p.z, p.ldz, i, k, q);
            float2 act[H], none[H];
            gate_of<false>(q, p.gate, act, none);
#pragma unroll
            for (int e = 0; e < H; ++e) y[i][k][e] = y[i][k][e] * act[e];
          }
          if (kAll || p.x) {
            read(2, p.x, p.ldx, i, k, q);
#pragma unroll
            for (int e = 0; e < H; ++e) y[i][k][e] = fma2(y[i][k][e], c[e], q[e]);
          } else {
#pragma unroll
            for (int e = 0; e < H; ++e) y[i][k][e] = y[i][k][e] * c[e];
          }
        }
      }
      float sums[2 * ROWS];
      float2 sq[ROWS], dot[ROWS];
#pragma unroll
      for (int i = 0; i < ROWS; ++i) sq[i] = dot[i] = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float2 w[H];
        P::params(p.w_pre, 0.f, t, k, p.width, w);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          float2 q[H];
          read(4, g.du, g.lddu, i, k, q);
#pragma unroll
          for (int e = 0; e < H; ++e) {
            sq[i] = fma2(y[i][k][e], y[i][k][e], sq[i]);
            dot[i] = fma2(q[e] * w[e], y[i][k][e], dot[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        sums[2 * i] = sq[i].x + sq[i].y;
        sums[2 * i + 1] = dot[i].x + dot[i].y;
      }
      group_sums<2 * ROWS, THREADS>(sums, red2, turn2);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        r2[i] = inverse_root(fmaf(sums[2 * i], inv, p.eps));
        back[i] = sums[2 * i + 1] * inv * r2[i] * r2[i] * r2[i];
      }
    }
    float2 dn[ROWS][K][H];
    float2 dot[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) dot[i] = both(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 w[H];
      P::params(p.w_pre, 0.f, t, k, p.width, w);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {  // dn holds dx for now
        if (kAll || g.dy) {
          read(3, g.dy, g.lddy, i, k, dn[i][k]);
        } else {
#pragma unroll
          for (int e = 0; e < H; ++e) dn[i][k][e] = both(0.f);
        }
        if (kAll || g.du) {
          float2 q[H];
          read(4, g.du, g.lddu, i, k, q);
#pragma unroll
          for (int e = 0; e < H; ++e) {
            const float2 ur = q[e] * both(r2[i]);
            dn[i][k][e] = fma2(ur, w[e], fma2(y[i][k][e], both(-back[i]), dn[i][k][e]));
            sp[k][e] = fma2(ur, y[i][k][e], sp[k][e]);
          }
        }
        if ((kAll || g.dx) && row0 + i < rows)
          P::store(g.dx, row0 + i, g.lddx, t, k, p.width, dn[i][k]);
      }
      float2 c[H];
      P::params(p.w_post, 1.f, t, k, p.width, w);
      P::params(p.scale, 1.f, t, k, p.width, c);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        float2 f[H], act[H], slope[H], dz[H];
        if (kAll || p.z) {
          read(1, p.z, p.ldz, i, k, f);
          gate_of<true>(f, p.gate, act, slope);
        } else {
#pragma unroll
          for (int e = 0; e < H; ++e) act[e] = both(1.f), slope[e] = both(0.f);
        }
        read(0, p.f, p.ldf, i, k, f);
#pragma unroll
        for (int e = 0; e < H; ++e) {
          const float2 n = f[e] * both(r1[i]), nw = n * w[e];
          const float2 d = dn[i][k][e];
          sc[k][e] = fma2(d * nw, act[e], sc[k][e]);
          const float2 dt = d * c[e], da = dt * act[e];
          dz[e] = dt * nw * slope[e];
          sw[k][e] = fma2(da, n, sw[k][e]);
          dn[i][k][e] = da * w[e];
          dot[i] = fma2(dn[i][k][e], n, dot[i]);
        }
        if ((kAll || g.dz) && row0 + i < rows)
          P::store(g.dz, row0 + i, g.lddz, t, k, p.width, dz);
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s[i] = dot[i].x + dot[i].y;
    cp_async_wait_group<0>();
    P::meet();
    squares(slot ^ 1, row0 + turn_rows, s + ROWS);
    group_sums<2 * ROWS, THREADS>(s, red, turn);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        if (kAll || p.w_post) {  // r1 (dn - f r1 mean)
          float2 f[H];
          read(0, p.f, p.ldf, i, k, f);
          const float m = -r1[i] * (s[i] * inv);
#pragma unroll
          for (int e = 0; e < H; ++e)
            dn[i][k][e] = both(r1[i]) * fma2(f[e], both(m), dn[i][k][e]);
        }
        if (row0 + i < rows)
          P::store(g.df, row0 + i, g.lddf, t, k, p.width, dn[i][k]);
      }
    P::meet();  // every thread has read its rows before they are overwritten
    stage(row0 + 2 * turn_rows, slot);
    slot ^= 1;
  }
  cp_async_wait_all();
  if (!partial) return;
  // the block's part, [3][width]; the sums of several groups in order
  float* sums = reinterpret_cast<float*>(shared);
  auto put = [&](int which, float2 (&v)[K][H]) {
    float* part = partial + (static_cast<int64_t>(blockIdx.x) * 3 + which) * p.width;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 2 * H; ++e) {
        const int c = row_element<2 * H, THREADS, P::kAl>(t, k, e);
        float sum = e % 2 ? v[k][e / 2].y : v[k][e / 2].x;
        if constexpr (G::kGroups > 1) {
          __syncthreads();
          sums[threadIdx.x] = sum;
          __syncthreads();
          if (group == 0)
            for (int q = 1; q < G::kGroups; ++q) sum += sums[q * THREADS + t];
        }
        if (group == 0 && c < p.width) part[c] = sum;
      }
  };
  __syncthreads();
  put(0, sw);
  put(1, sc);
  put(2, sp);
}

// ------------------------------------------------------------------ long rows
__device__ __forceinline__ float block_sum(float v, float* red, int& turn) {
  float s[1] = {v};
  group_sums<1, kLong>(s, red, turn);
  return s[0];
}

template <typename T>
__device__ __forceinline__ float new_residual(const GnormRows<T>& p, int64_t row, int c, float r1) {
  float t = to_f32(p.f[row * p.ldf + c]);
  if (p.w_post) t = t * r1 * p.w_post[c];
  if (p.z) t *= gate_of(to_f32(p.z[row * p.ldz + c]), p.gate).act;
  return fmaf(t, p.scale ? p.scale[c] : 1.f, p.x ? to_f32(p.x[row * p.ldx + c]) : 0.f);
}

template <typename T>
__device__ __forceinline__ float post_norm(const GnormRows<T>& p, int64_t row, float* red,
                                           int& turn) {
  if (!p.w_post) return 1.f;
  float sum = 0.f;
  for (int c = threadIdx.x; c < p.width; c += kLong) {
    const float v = to_f32(p.f[row * p.ldf + c]);
    sum = fmaf(v, v, sum);
  }
  return inverse_root(fmaf(block_sum(sum, red, turn), 1.f / p.width, p.eps));
}

template <typename T, bool Q8>
__global__ void __launch_bounds__(kLong)
gnorm_long_kernel(GnormRows<T> p, T* __restrict__ y, int64_t ldy, T* __restrict__ u, int64_t ldu,
                  Bytes8 bytes8) {
  __shared__ float red[kRedFloats<1, kLong>];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float r1 = post_norm(p, row, red, turn);
    float r2 = 1.f;
    if (Q8 ? p.w_pre != nullptr : u != nullptr) {
      float sum = 0.f;
      for (int c = threadIdx.x; c < p.width; c += kLong) {
        const float v = new_residual(p, row, c, r1);
        sum = fmaf(v, v, sum);
      }
      r2 = inverse_root(fmaf(block_sum(sum, red, turn), 1.f / p.width, p.eps));
    }
    if constexpr (Q8) {  // the 128 elements under a scale by one warp
      const int lane = threadIdx.x & 31;
      for (int block = threadIdx.x / 32; block * kScaled < p.width; block += kLong / 32) {
        float v[kScaled / 32];
        unsigned top = 0;
#pragma unroll
        for (int j = 0; j < kScaled / 32; ++j) {
          const int c = block * kScaled + j * 32 + lane;
          v[j] = 0.f;
          if (c >= p.width) continue;
          v[j] = new_residual(p, row, c, r1);
          if (y) y[row * ldy + c] = from_f32<T>(v[j]);
          if (p.w_pre) v[j] *= r2 * p.w_pre[c];
          top = max(top, magnitude(v[j]));
        }
        const float s = scale_of(__reduce_max_sync(0xFFFFFFFFu, top));
        if (lane == 0) bytes8.s[row * bytes8.lds + block] = s;
#pragma unroll
        for (int j = 0; j < kScaled / 32; ++j) {
          const int c = block * kScaled + j * 32 + lane;
          if (c < p.width)
            bytes8.q[row * bytes8.ldq + c] =
                static_cast<uint8_t>(as_e4m3(make_float2(__fdiv_rn(v[j], s), 0.f)));
        }
      }
    } else {
      for (int c = threadIdx.x; c < p.width; c += kLong) {
        const float v = new_residual(p, row, c, r1);
        if (y) y[row * ldy + c] = from_f32<T>(v);
        if (u) u[row * ldu + c] = from_f32<T>(v * (r2 * p.w_pre[c]));
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kLong, 2)
gnorm_long_backward_kernel(GnormRows<T> p, GnormGrads<T> g, float* __restrict__ partial) {
  __shared__ float red[kRedFloats<1, kLong>];
  int turn = 0;
  const float inv = 1.f / p.width;
  float* part = partial + static_cast<int64_t>(blockIdx.x) * 3 * p.width;
  if (partial)  // a thread touches its own columns only
    for (int j = 0; j < 3; ++j)
      for (int c = threadIdx.x; c < p.width; c += kLong) part[j * p.width + c] = 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float r1 = post_norm(p, row, red, turn);
    float r2 = 0.f, back = 0.f;
    if (g.du) {
      float sum = 0.f, dot = 0.f;
      for (int c = threadIdx.x; c < p.width; c += kLong) {
        const float v = new_residual(p, row, c, r1);
        sum = fmaf(v, v, sum);
        dot = fmaf(to_f32(g.du[row * g.lddu + c]) * p.w_pre[c], v, dot);
      }
      r2 = inverse_root(fmaf(block_sum(sum, red, turn), inv, p.eps));
      back = block_sum(dot, red, turn) * inv * r2 * r2 * r2;
    }
    float dot = 0.f;
    for (int c = threadIdx.x; c < p.width; c += kLong) {
      const float v = new_residual(p, row, c, r1);
      float d = g.dy ? to_f32(g.dy[row * g.lddy + c]) : 0.f;
      if (g.du) {
        const float du = to_f32(g.du[row * g.lddu + c]);
        d = fmaf(-v, back, fmaf(du * p.w_pre[c], r2, d));
        if (g.dw_pre) part[2 * p.width + c] += du * v * r2;
      }
      if (g.dx) g.dx[row * g.lddx + c] = from_f32<T>(d);
      const float n = to_f32(p.f[row * p.ldf + c]) * r1;
      const float w = p.w_post ? p.w_post[c] : 1.f;
      const Gate q = p.z ? gate_of(to_f32(p.z[row * p.ldz + c]), p.gate) : Gate{1.f, 0.f};
      if (g.dscale) part[p.width + c] += d * (n * w) * q.act;
      const float dt = p.scale ? d * p.scale[c] : d;
      if (g.dz) g.dz[row * g.lddz + c] = from_f32<T>(dt * (n * w) * q.slope);
      const float da = dt * q.act;
      if (g.dw_post) part[c] += da * n;
      dot = fmaf(da * w, n, dot);
    }
    const float mean = p.w_post ? block_sum(dot, red, turn) * inv : 0.f;
    for (int c = threadIdx.x; c < p.width; c += kLong) {
      float d = g.dy ? to_f32(g.dy[row * g.lddy + c]) : 0.f;
      if (g.du)
        d = fmaf(-new_residual(p, row, c, r1), back,
                 fmaf(to_f32(g.du[row * g.lddu + c]) * p.w_pre[c], r2, d));
      if (p.scale) d *= p.scale[c];
      if (p.z) d *= gate_of(to_f32(p.z[row * p.ldz + c]), p.gate).act;
      if (p.w_post)
        d = r1 * fmaf(-(to_f32(p.f[row * p.ldf + c]) * r1), mean, d * p.w_post[c]);
      g.df[row * g.lddf + c] = from_f32<T>(d);
    }
  }
}

// ------------------------------------------------------------------ launches

inline bool vec16(const void* p, int64_t bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(bytes)) & 15) == 0;
}

// Calls f with a shape as compile-time values.
template <int PAIRS, int K, int THREADS, int ROWS>
struct Config {
  static constexpr int pairs = PAIRS, vectors = K, threads = THREADS, rows = ROWS;
};
template <int PAIRS, int ROWS, typename F>
cudaError_t with_threads(int threads, F&& f) {
  switch (threads) {
    case 8: return f(Config<PAIRS, 1, 8, ROWS>());
    case 16: return f(Config<PAIRS, 1, 16, ROWS>());
    case 32: return f(Config<PAIRS, 1, 32, ROWS>());
    case 64: return f(Config<PAIRS, 1, 64, ROWS>());
    case 128: return f(Config<PAIRS, 1, 128, ROWS>());
    case 256: return f(Config<PAIRS, 1, 256, ROWS>());
    default: return f(Config<PAIRS, 1, 512, ROWS>());
  }
}

template <typename T, int MODE, bool Q8>
cudaError_t launch_forward(const Shape& s, const GnormRows<T>& p, T* y, int64_t ldy, T* u,
                           int64_t ldu, const Bytes8& bytes8, cudaStream_t stream) {
  constexpr int H = kVecElements<T> / 2;
  auto run = [&](auto c) {
    using C = decltype(c);
    using P = Part<T, H, C::vectors, C::threads, C::rows, MODE>;
    constexpr int kShared = Group<C::threads>::kGroups * kTurns * C::rows * 3 * P::kRow;
    auto* kernel = gnorm_kernel<T, H, C::vectors, C::threads, C::rows, MODE, Q8>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
    if (e != cudaSuccess) return e;
    kernel<<<blocks_for(s, p.rows), Group<C::threads>::kBlock, kShared, stream>>>(p, y, ldy, u, ldu,
                                                                                 bytes8);
    return cudaGetLastError();
  };
  if (s.threads < 1024) return with_threads<H, 2>(s.threads, run);
  return s.vectors == 1 ? run(Config<H, 1, 1024, 1>()) : run(Config<H, 2, 1024, 1>());
}

template <typename T, int MODE>
cudaError_t launch_backward(const Shape& s, const GnormRows<T>& p, const GnormGrads<T>& g,
                            float* partial, int parts, cudaStream_t stream) {
  auto run = [&](auto c) {
    using C = decltype(c);
    using P = Part<T, C::pairs, C::vectors, C::threads, C::rows, MODE>;
    constexpr int kShared = Group<C::threads>::kGroups * kTurns * C::rows * 5 * P::kRow;
    auto* kernel = gnorm_backward_kernel<T, C::pairs, C::vectors, C::threads, C::rows, MODE>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
    if (e != cudaSuccess) return e;
    kernel<<<parts, Group<C::threads>::kBlock, kShared, stream>>>(p, g, partial);
    return cudaGetLastError();
  };
  constexpr int H = kVecElements<T> / 2;
  if (s.threads < 1024) return with_threads<H, sizeof(T) == 2 ? 2 : 1>(s.threads, run);
  return run(Config<2, sizeof(T) == 2 ? 2 : 1, 1024, 1>());
}

// Whether an operand is there (or need not be) and lies on 16-byte boundaries.
template <typename T>
struct Lies {
  bool all = true, aligned = true;
  template <typename V>
  Lies& with(const V* p, int64_t ld) {
    all = all && p != nullptr;
    aligned = aligned && vec16(p, ld * static_cast<int64_t>(sizeof(V)));
    return *this;
  }
  Mode mode(int width) const {
    if (!aligned) return kAny;
    return all && width * sizeof(T) % 16 == 0 ? kFull : kAligned;
  }
};

}  // namespace

template <typename T>
cudaError_t launch_gnorm(const GnormRows<T>& p, T* y, int64_t ldy, T* u, int64_t ldu,
                         cudaStream_t stream) {
  const Shape s = forward_shape(p.width, sizeof(T));
  if (s.threads == 0) {
    gnorm_long_kernel<T, false><<<blocks_for(s, p.rows, 2 * kLong), kLong, 0, stream>>>(p, y, ldy, u,
                                                                                       ldu, {});
    return cudaGetLastError();
  }
  const Mode mode = Lies<T>()
                        .with(p.f, p.ldf).with(p.z, p.ldz).with(p.x, p.ldx).with(y, ldy)
                        .with(u, ldu).with(p.w_post, 0).with(p.scale, 0).with(p.w_pre, 0)
                        .mode(p.width);
  auto* launch = mode == kFull      ? launch_forward<T, kFull, false>
                 : mode == kAligned ? launch_forward<T, kAligned, false>
                                    : launch_forward<T, kAny, false>;
  return launch(s, p, y, ldy, u, ldu, {}, stream);
}

template <typename T>
cudaError_t launch_gnorm_q8(const GnormRows<T>& p, T* y, int64_t ldy, const Bytes8& out,
                            cudaStream_t stream) {
  const Shape s = forward_shape(p.width, sizeof(T));
  if (s.threads == 0) {
    gnorm_long_kernel<T, true><<<blocks_for(s, p.rows, 2 * kLong), kLong, 0, stream>>>(p, y, ldy, nullptr,
                                                                                      0, out);
    return cudaGetLastError();
  }
  const Mode mode = Lies<T>()
                        .with(p.f, p.ldf).with(p.z, p.ldz).with(p.x, p.ldx).with(y, ldy)
                        .with(out.q, out.ldq).with(p.w_post, 0).with(p.scale, 0).with(p.w_pre, 0)
                        .mode(p.width);
  auto* launch = mode == kFull      ? launch_forward<T, kFull, true>
                 : mode == kAligned ? launch_forward<T, kAligned, true>
                                    : launch_forward<T, kAny, true>;
  return launch(s, p, y, ldy, nullptr, 0, out, stream);
}

template <typename T>
cudaError_t launch_gnorm_backward(const GnormRows<T>& p, const GnormGrads<T>& g, void* work,
                                  cudaStream_t stream) {
  const bool sums = g.dw_post || g.dscale || g.dw_pre;
  float* partial = sums ? static_cast<float*>(work) : nullptr;
  const Shape s = backward_shape(p.width, sizeof(T));
  const int parts = backward_blocks(p.width, sizeof(T), p.rows);
  if (parts > 0) {
    cudaError_t e;
    if (s.threads == 0) {
      gnorm_long_backward_kernel<T><<<parts, kLong, 0, stream>>>(p, g, partial);
      e = cudaGetLastError();
    } else {
      const Mode mode = Lies<T>()
                            .with(p.f, p.ldf).with(p.z, p.ldz).with(p.x, p.ldx)
                            .with(g.dy, g.lddy).with(g.du, g.lddu).with(g.df, g.lddf)
                            .with(g.dz, g.lddz).with(g.dx, g.lddx).with(p.w_post, 0)
                            .with(p.scale, 0).with(p.w_pre, 0)
                            .mode(p.width);
      auto* launch = mode == kFull      ? launch_backward<T, kFull>
                     : mode == kAligned ? launch_backward<T, kAligned>
                                        : launch_backward<T, kAny>;
      e = launch(s, p, g, partial, parts, stream);
    }
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  return launch_gnorm_sums(p.width, parts, partial, g.dw_post, g.dscale, g.dw_pre, stream);
}

#define BSOLVE_GNORM(T)                                                                         \
  template cudaError_t launch_gnorm<T>(const GnormRows<T>&, T*, int64_t, T*, int64_t,           \
                                       cudaStream_t);                                           \
  template cudaError_t launch_gnorm_backward<T>(const GnormRows<T>&, const GnormGrads<T>&,      \
                                                void*, cudaStream_t);
#define BSOLVE_GNORM_Q8(T)                                                                      \
  template cudaError_t launch_gnorm_q8<T>(const GnormRows<T>&, T*, int64_t, const Bytes8&,      \
                                          cudaStream_t);

}  // namespace bsolve
