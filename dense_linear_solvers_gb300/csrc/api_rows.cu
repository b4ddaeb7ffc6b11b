// C ABI of the row operators (bs_grec and bs_gnorm calls of bsolve.h): argument checks and
// dispatch to the kernel launchers.
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bsolve.h"
#include "kernels.h"

namespace {

constexpr int kMaxChannels = 1 << 20;
constexpr int kMaxWidth = 65536;
constexpr int64_t kMaxRows = int64_t(1) << 30;  // a row's number, and a step beyond, fits 32 bits
constexpr int64_t kMaxLd = int64_t(1) << 21;

int element_size(bs_dtype dtype) {
  switch (dtype) {
    case BS_FP32: return 4;
    case BS_BF16:
    case BS_FP16: return 2;
    default: return 0;
  }
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// An operand of a call: `rows` pieces of `width` bytes, `pitch` bytes apart (null: absent).
struct Operand {
  const void* base;
  int64_t rows, width, pitch;
};

// Whether two operands share a byte. Operands of one pitch may interleave as column windows
// of one matrix: their windows are then compared within a row.
bool share(const Operand& a, const Operand& b) {
  if (!a.base || !b.base || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0)
    return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.base), y = reinterpret_cast<uintptr_t>(b.base);
  const uintptr_t xe = x + static_cast<uintptr_t>((a.rows - 1) * a.pitch + a.width);
  const uintptr_t ye = y + static_cast<uintptr_t>((b.rows - 1) * b.pitch + b.width);
  if (xe <= y || ye <= x) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t pitch = a.pitch;
  const int64_t d = x <= y ? static_cast<int64_t>((y - x) % pitch)      // b's window starts d
                           : (pitch - static_cast<int64_t>((x - y) % pitch)) % pitch;  // after a's
  return d < a.width || d + b.width > pitch;
}

// Whether no output shares a byte with an input or another output.
bool apart(std::initializer_list<Operand> outs, std::initializer_list<Operand> ins) {
  for (auto a = outs.begin(); a != outs.end(); ++a) {
    for (auto b = a + 1; b != outs.end(); ++b)
      if (share(*a, *b)) return false;
    for (const Operand& b : ins)
      if (share(*a, b)) return false;
  }
  return true;
}

bs_status done(cudaError_t e) {
  if (e == cudaSuccess) return BS_OK;
  bsolve::record_cuda_error(e);
  return BS_ERR_CUDA;
}

bool bad_ld(int64_t ld, int width) { return ld < width; }

bool grec_ok(bs_dtype dtype, int channels) {
  return element_size(dtype) != 0 && channels >= 1 && channels <= kMaxChannels;
}

bool gnorm_ok(bs_dtype dtype, int width) {
  return element_size(dtype) != 0 && width >= 1 && width <= kMaxWidth;
}

// The checks the three bs_grec calls share; sets *empty when there is nothing to do.
bs_status grec_sizes(bs_dtype dtype, int channels, int64_t batch, int64_t rows, double kappa,
                     std::initializer_list<int64_t> lds) {
  if (channels < 0 || batch < 0 || rows < 0) return BS_ERR_INVALID_ARG;
  if (!(kappa > 0.0) || !std::isfinite(static_cast<float>(kappa))) return BS_ERR_INVALID_ARG;
  if (!grec_ok(dtype, channels) || batch > 0x7FFFFFFF || rows > kMaxRows)
    return BS_ERR_UNSUPPORTED;
  for (int64_t ld : lds) {
    if (bad_ld(ld, channels)) return BS_ERR_INVALID_ARG;
    if (ld > kMaxLd) return BS_ERR_UNSUPPORTED;
  }
  return BS_OK;
}

template <typename T>
bsolve::GrecRows<T> grec_rows(int channels, int64_t batch, int64_t rows, const int64_t* offsets,
                              const void* x, int64_t ldx, const void* r, int64_t ldr,
                              const void* i, int64_t ldi) {
  return {channels, batch, rows, offsets || batch == 0 ? 0 : rows / batch, offsets,
          static_cast<const T*>(x), static_cast<const T*>(r), static_cast<const T*>(i),
          ldx, ldr, ldi};
}

// Calls f with a value of the row type.
template <typename F>
cudaError_t with_type(bs_dtype dtype, F&& f) {
  switch (dtype) {
    case BS_FP32: return f(float());
    case BS_BF16: return f(__nv_bfloat16());
    default: return f(__half());
  }
}

}  // namespace

extern "C" {

bs_status bs_grec_batched(bs_dtype dtype, int channels, int64_t batch, int64_t rows,
                          const int64_t* offsets, const void* x, int64_t ldx, const void* r,
                          int64_t ldr, const void* i, int64_t ldi, const float* lam, double kappa,
                          const float* h0, void* h, int64_t ldh, float* hT, float* tape,
                          void* stream) {
  const bs_status st = grec_sizes(dtype, channels, batch, rows, kappa, {ldx, ldr, ldi, ldh});
  if (st != BS_OK) return st;
  if (batch == 0) return BS_OK;
  if (!offsets && rows % batch != 0) return BS_ERR_INVALID_ARG;
  if (!lam || (rows > 0 && (!x || !r || !i || !h))) return BS_ERR_INVALID_ARG;
  const uintptr_t es = element_size(dtype);
  if (!aligned(x, es) || !aligned(r, es) || !aligned(i, es) || !aligned(h, es) ||
      !aligned(lam, 4) || !aligned(h0, 4) || !aligned(hT, 4) || !aligned(tape, 4) ||
      !aligned(offsets, 8))
    return BS_ERR_INVALID_ARG;
  const int64_t w = channels * int64_t(es), sw = channels * int64_t(4);
  const Operand oh{h, rows, w, ldh * int64_t(es)}, ohT{hT, batch, sw, sw},
      otape{tape, bs_grec_tape_rows(batch, rows), sw, sw}, ox{x, rows, w, ldx * int64_t(es)},
      orr{r, rows, w, ldr * int64_t(es)}, oi{i, rows, w, ldi * int64_t(es)}, ol{lam, 1, sw, sw},
      oh0{hT == h0 ? nullptr : h0, batch, sw, sw},
      oo{offsets, 1, (batch + 1) * 8, (batch + 1) * 8};
  if (!apart({oh, ohT, otape}, {ox, orr, oi, ol, oh0, oo})) return BS_ERR_INVALID_ARG;
  if (h0 && hT == h0 && !apart({oh, otape}, {ohT})) return BS_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    return bsolve::launch_grec<T>(
        grec_rows<T>(channels, batch, rows, offsets, x, ldx, r, ldr, i, ldi), lam,
        static_cast<float>(kappa), h0, static_cast<T*>(h), ldh, hT, tape, s);
  }));
}

bs_status bs_grec_backward_batched(bs_dtype dtype, int channels, int64_t batch, int64_t rows,
                                   const int64_t* offsets, const void* x, int64_t ldx,
                                   const void* r, int64_t ldr, const void* i, int64_t ldi,
                                   const float* lam, double kappa, const float* tape,
                                   const void* dh, int64_t lddh, const float* dhT, void* dx,
                                   int64_t lddx, void* dr, int64_t lddr, void* di, int64_t lddi,
                                   float* dlam, float* dh0, void* work, size_t work_bytes,
                                   void* stream) {
  const bs_status st = grec_sizes(dtype, channels, batch, rows, kappa,
                                  {ldx, ldr, ldi, lddh, lddx, lddr, lddi});
  if (st != BS_OK) return st;
  if (batch > 0 && !offsets && rows % batch != 0) return BS_ERR_INVALID_ARG;
  if (!lam || !dlam) return BS_ERR_INVALID_ARG;
  if (batch > 0 && (!tape || !work ||
                    (rows > 0 && (!x || !r || !i || !dh || !dx || !dr || !di))))
    return BS_ERR_INVALID_ARG;
  const uintptr_t es = element_size(dtype);
  for (const void* p : {x, r, i, dh, static_cast<const void*>(dx), static_cast<const void*>(dr),
                        static_cast<const void*>(di)})
    if (!aligned(p, es)) return BS_ERR_INVALID_ARG;
  if (!aligned(lam, 4) || !aligned(tape, 4) || !aligned(dhT, 4) || !aligned(dlam, 4) ||
      !aligned(dh0, 4) || !aligned(offsets, 8) || !aligned(work, 16))
    return BS_ERR_INVALID_ARG;
  const size_t need = bs_grec_backward_workspace(channels, batch, rows);
  if (work_bytes < need) return BS_ERR_INVALID_ARG;
  const int64_t e = es, w = channels * e, sw = channels * int64_t(4);
  if (!apart({{dx, rows, w, lddx * e}, {dr, rows, w, lddr * e}, {di, rows, w, lddi * e},
              {dlam, 1, sw, sw}, {dh0, batch, sw, sw},
              {work, 1, static_cast<int64_t>(need), static_cast<int64_t>(need)}},
             {{x, rows, w, ldx * e}, {r, rows, w, ldr * e}, {i, rows, w, ldi * e},
              {dh, rows, w, lddh * e}, {lam, 1, sw, sw}, {dhT, batch, sw, sw},
              {tape, bs_grec_tape_rows(batch, rows), sw, sw},
              {offsets, 1, (batch + 1) * 8, (batch + 1) * 8}}))
    return BS_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    return bsolve::launch_grec_backward<T>(
        grec_rows<T>(channels, batch, rows, offsets, x, ldx, r, ldr, i, ldi), lam,
        static_cast<float>(kappa), tape, static_cast<const T*>(dh), lddh, dhT,
        static_cast<T*>(dx), lddx, static_cast<T*>(dr), lddr, static_cast<T*>(di), lddi, dlam,
        dh0, work, s);
  }));
}

bs_status bs_grec_step_batched(bs_dtype dtype, int channels, int64_t batch, const void* x,
                               int64_t ldx, const void* r, int64_t ldr, const void* i,
                               int64_t ldi, const float* lam, double kappa, float* state,
                               int64_t num_slots, const int32_t* slots, void* y, int64_t ldy,
                               void* stream) {
  if (num_slots < 0) return BS_ERR_INVALID_ARG;
  const bs_status st = grec_sizes(dtype, channels, batch, batch, kappa, {ldx, ldr, ldi, ldy});
  if (st != BS_OK) return st;
  if (num_slots > kMaxRows) return BS_ERR_UNSUPPORTED;
  if (batch == 0) return BS_OK;
  if (!x || !r || !i || !lam || !y || (num_slots > 0 && !state)) return BS_ERR_INVALID_ARG;
  const uintptr_t es = element_size(dtype);
  if (!aligned(x, es) || !aligned(r, es) || !aligned(i, es) || !aligned(y, es) ||
      !aligned(lam, 4) || !aligned(state, 4) || !aligned(slots, 4))
    return BS_ERR_INVALID_ARG;
  const int64_t e = es, w = channels * e, sw = channels * int64_t(4);
  if (!apart({{y, batch, w, ldy * e}, {state, num_slots, sw, sw}},
             {{x, batch, w, ldx * e}, {r, batch, w, ldr * e}, {i, batch, w, ldi * e},
              {lam, 1, sw, sw}, {slots, 1, batch * 4, batch * 4}}))
    return BS_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    return bsolve::launch_grec_step<T>(
        grec_rows<T>(channels, batch, batch, nullptr, x, ldx, r, ldr, i, ldi), lam,
        static_cast<float>(kappa), state, num_slots, slots, static_cast<T*>(y), ldy, s);
  }));
}

int64_t bs_grec_tape_rows(int64_t batch, int64_t rows) {
  return batch < 0 || rows < 0 ? 0 : rows / 32 + batch;
}

size_t bs_grec_backward_workspace(int channels, int64_t batch, int64_t rows) {
  if (channels < 1 || channels > kMaxChannels || batch < 0 || batch > 0x7FFFFFFF || rows < 0)
    return 0;
  return bsolve::grec_backward_workspace(channels, batch, rows);
}

int bs_grec_supported(bs_dtype dtype, int channels) { return grec_ok(dtype, channels) ? 1 : 0; }

bs_status bs_gnorm_batched(bs_dtype dtype, int64_t rows, int width, const void* f, int64_t ldf,
                           const void* z, int64_t ldz, const void* x, int64_t ldx,
                           const float* w_post, const float* scale, const float* w_pre,
                           double eps, bs_gate gate, void* y, int64_t ldy, void* u, int64_t ldu,
                           void* stream) {
  if (rows < 0 || width < 0) return BS_ERR_INVALID_ARG;
  if (!(static_cast<float>(eps) > 0.f) || !std::isfinite(static_cast<float>(eps)) ||
      gate < BS_GATE_SILU || gate > BS_GATE_LINEAR)
    return BS_ERR_INVALID_ARG;
  if (!gnorm_ok(dtype, width) || rows > kMaxRows) return BS_ERR_UNSUPPORTED;
  if (bad_ld(ldf, width) || (z && bad_ld(ldz, width)) || (x && bad_ld(ldx, width)) ||
      (y && bad_ld(ldy, width)) || (u && bad_ld(ldu, width)))
    return BS_ERR_INVALID_ARG;
  if (ldf > kMaxLd || (z && ldz > kMaxLd) || (x && ldx > kMaxLd) || (y && ldy > kMaxLd) ||
      (u && ldu > kMaxLd))
    return BS_ERR_UNSUPPORTED;
  if (rows == 0) return BS_OK;
  if (!f || (!y && !u) || (u == nullptr) != (w_pre == nullptr)) return BS_ERR_INVALID_ARG;
  const uintptr_t es = element_size(dtype);
  if (!aligned(f, es) || !aligned(z, es) || !aligned(x, es) || !aligned(y, es) ||
      !aligned(u, es) || !aligned(w_post, 4) || !aligned(scale, 4) || !aligned(w_pre, 4))
    return BS_ERR_INVALID_ARG;
  const int64_t e = es, w = width * e, sw = width * int64_t(4);
  if (!apart({{y, rows, w, ldy * e}, {u, rows, w, ldu * e}},
             {{f, rows, w, ldf * e}, {z, rows, w, ldz * e}, {x, rows, w, ldx * e},
              {w_post, 1, sw, sw}, {scale, 1, sw, sw}, {w_pre, 1, sw, sw}}))
    return BS_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    const bsolve::GnormRows<T> p{rows, width, static_cast<const T*>(f), static_cast<const T*>(z),
                                 static_cast<const T*>(x), ldf, ldz, ldx, w_post, scale, w_pre,
                                 static_cast<float>(eps), static_cast<int>(gate)};
    return bsolve::launch_gnorm<T>(p, static_cast<T*>(y), ldy, static_cast<T*>(u), ldu, s);
  }));
}

bs_status bs_gnorm_backward_batched(bs_dtype dtype, int64_t rows, int width, const void* f,
                                    int64_t ldf, const void* z, int64_t ldz, const void* x,
                                    int64_t ldx, const float* w_post, const float* scale,
                                    const float* w_pre, double eps, bs_gate gate, const void* dy,
                                    int64_t lddy, const void* du, int64_t lddu, void* df,
                                    int64_t lddf, void* dz, int64_t lddz, void* dx, int64_t lddx,
                                    float* dw_post, float* dscale, float* dw_pre, void* work,
                                    size_t work_bytes, void* stream) {
  if (rows < 0 || width < 0) return BS_ERR_INVALID_ARG;
  if (!(static_cast<float>(eps) > 0.f) || !std::isfinite(static_cast<float>(eps)) ||
      gate < BS_GATE_SILU || gate > BS_GATE_LINEAR)
    return BS_ERR_INVALID_ARG;
  if (!gnorm_ok(dtype, width) || rows > kMaxRows) return BS_ERR_UNSUPPORTED;
  const uintptr_t es = element_size(dtype);
  const int64_t e = es, w = width * e, sw = width * int64_t(4);
  const std::pair<const void*, int64_t> lds[] = {{f, ldf},   {z, ldz},   {x, ldx},   {dy, lddy},
                                                 {du, lddu}, {df, lddf}, {dz, lddz}, {dx, lddx}};
  for (const auto& q : lds) {
    if (!q.first) continue;
    if (bad_ld(q.second, width) || !aligned(q.first, es)) return BS_ERR_INVALID_ARG;
    if (q.second > kMaxLd) return BS_ERR_UNSUPPORTED;
  }
  for (const float* q : {w_post, scale, w_pre, static_cast<const float*>(dw_post),
                         static_cast<const float*>(dscale), static_cast<const float*>(dw_pre)})
    if (!aligned(q, 4)) return BS_ERR_INVALID_ARG;
  if ((dw_post && !w_post) || (dscale && !scale) || (dw_pre && !w_pre)) return BS_ERR_INVALID_ARG;
  if (rows > 0) {
    if (!f || !df || (!dy && !du) || (du == nullptr) != (w_pre == nullptr) || (dz && !z) ||
        (dx && !x))
      return BS_ERR_INVALID_ARG;
  }
  const bool sums = dw_post || dscale || dw_pre;
  const size_t need = sums ? bs_gnorm_backward_workspace(width, rows) : 0;
  if (need > 0 && (!work || !aligned(work, 16) || work_bytes < need)) return BS_ERR_INVALID_ARG;
  if (!apart({{df, rows, w, lddf * e}, {dz, rows, w, lddz * e}, {dx, rows, w, lddx * e},
              {dw_post, 1, sw, sw}, {dscale, 1, sw, sw}, {dw_pre, 1, sw, sw},
              {work, 1, static_cast<int64_t>(need), static_cast<int64_t>(need)}},
             {{f, rows, w, ldf * e}, {z, rows, w, ldz * e}, {x, rows, w, ldx * e},
              {dy, rows, w, lddy * e}, {du, rows, w, lddu * e}, {w_post, 1, sw, sw},
              {scale, 1, sw, sw}, {w_pre, 1, sw, sw}}))
    return BS_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    const bsolve::GnormRows<T> p{rows, width, static_cast<const T*>(f), static_cast<const T*>(z),
                                 static_cast<const T*>(x), ldf, ldz, ldx, w_post, scale, w_pre,
                                 static_cast<float>(eps), static_cast<int>(gate)};
    const bsolve::GnormGrads<T> g{static_cast<const T*>(dy), static_cast<const T*>(du), lddy, lddu,
                                  static_cast<T*>(df), static_cast<T*>(dz), static_cast<T*>(dx),
                                  lddf, lddz, lddx, dw_post, dscale, dw_pre};
    return bsolve::launch_gnorm_backward<T>(p, g, work, s);
  }));
}

size_t bs_gnorm_backward_workspace(int width, int64_t rows) {
  if (width < 1 || width > kMaxWidth || rows < 0) return 0;
  return bsolve::gnorm_backward_workspace(width, rows);
}

int bs_gnorm_supported(bs_dtype dtype, int width) { return gnorm_ok(dtype, width) ? 1 : 0; }

}  // extern "C"
