// C ABI of the gated delta rule (bs_gdelta calls of bsolve.h): argument checks and dispatch to the
// kernel launchers.
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "api_rows.cuh"

namespace {

constexpr int kMaxDk = 128;
constexpr int kMaxDv = 1024;
constexpr int64_t kMaxStates = int64_t(1) << 24;

bool gdelta_ok(bs_dtype dtype, int heads_k, int heads_v, int dk, int dv) {
  return element_size(dtype) != 0 && heads_k >= 1 && heads_v >= heads_k && heads_v % heads_k == 0 &&
         heads_v <= 65535 && dk >= 1 && dk <= kMaxDk && dv >= 1 && dv <= kMaxDv;
}
bool gdelta_counts(int64_t batch, int heads_v, int64_t rows) {
  return rows <= kMaxRows && batch <= kMaxStates && batch * heads_v <= kMaxStates;
}

// A row operand of a call: its base, row distance, elements a row, and their size.
struct RowArg {
  const void* base;
  int64_t ld, width;
  int size;
};

// The checks the bs_gdelta calls share: sizes, row distances, null and aligned row operands.
bs_status gdelta_sizes(bs_dtype dtype, int heads_k, int heads_v, int dk, int dv, int64_t batch,
                       int64_t rows, double scale, std::initializer_list<RowArg> operands) {
  if (heads_k < 0 || heads_v < 0 || dk < 0 || dv < 0 || batch < 0 || rows < 0)
    return BS_ERR_INVALID_ARG;
  if (!std::isfinite(static_cast<float>(scale))) return BS_ERR_INVALID_ARG;
  if (heads_k > 0 && heads_v % heads_k != 0) return BS_ERR_INVALID_ARG;
  if (!gdelta_ok(dtype, heads_k, heads_v, dk, dv) || !gdelta_counts(batch, heads_v, rows))
    return BS_ERR_UNSUPPORTED;
  for (const RowArg& r : operands) {
    if (r.ld < r.width || !aligned(r.base, r.size)) return BS_ERR_INVALID_ARG;
    if (r.ld > kMaxLd) return BS_ERR_UNSUPPORTED;
    if (rows > 0 && batch > 0 && !r.base) return BS_ERR_INVALID_ARG;
  }
  return BS_OK;
}

Operand operand(const RowArg& r, int64_t rows) {
  return {r.base, rows, r.width * r.size, r.ld * r.size};
}
// A contiguous operand of so many bytes.
Operand block(const void* base, int64_t bytes) { return {base, 1, bytes, bytes}; }

template <typename T>
bsolve::GdeltaRows<T> gdelta_rows(int heads_k, int heads_v, int dk, int dv, int64_t batch,
                                  int64_t rows, const int64_t* offsets, const RowArg& q,
                                  const RowArg& k, const RowArg& v, const RowArg& g,
                                  const RowArg& beta, double scale) {
  return {heads_k, heads_v, dk, dv, batch, rows, offsets || batch == 0 ? 0 : rows / batch, offsets,
          static_cast<const T*>(q.base), static_cast<const T*>(k.base),
          static_cast<const T*>(v.base), q.ld, k.ld, v.ld, static_cast<const float*>(g.base),
          static_cast<const float*>(beta.base), g.ld, beta.ld, static_cast<float>(scale)};
}

}  // namespace

extern "C" {

bs_status bs_gdelta_batched(bs_dtype dtype, int heads_k, int heads_v, int dk, int dv, int64_t batch,
                            int64_t rows, const int64_t* offsets, const void* q, int64_t ldq,
                            const void* k, int64_t ldk, const void* v, int64_t ldv, const float* g,
                            int64_t ldg, const float* beta, int64_t ldbeta, double scale,
                            const float* h0, void* o, int64_t ldo, float* hT, void* tape,
                            void* work, size_t work_bytes, void* stream) {
  const int es = element_size(dtype);
  const int64_t wk = int64_t(heads_k) * dk, wv = int64_t(heads_v) * dv;
  const RowArg aq{q, ldq, wk, es}, ak{k, ldk, wk, es}, av{v, ldv, wv, es}, ag{g, ldg, heads_v, 4},
      ab{beta, ldbeta, heads_v, 4}, ao{o, ldo, wv, es};
  const bs_status st = gdelta_sizes(dtype, heads_k, heads_v, dk, dv, batch, rows, scale,
                                    {aq, ak, av, ag, ab, ao});
  if (st != BS_OK) return st;
  if (batch == 0) return BS_OK;
  if (!offsets && rows % batch != 0) return BS_ERR_INVALID_ARG;
  if (!aligned(h0, 4) || !aligned(hT, 4) || !aligned(tape, 16) || !aligned(work, 16) ||
      !aligned(offsets, 8))
    return BS_ERR_INVALID_ARG;
  const size_t need = bs_gdelta_workspace(heads_v, batch, rows);
  if (!work || work_bytes < need) return BS_ERR_INVALID_ARG;
  const int64_t state = batch * heads_v * dk * dv * 4;
  const Operand ohT = block(hT, state), owork = block(work, need), oo = operand(ao, rows),
                otape = block(tape, bs_gdelta_tape(heads_v, dk, dv, batch, rows));
  if (!apart({oo, ohT, otape, owork},
             {operand(aq, rows), operand(ak, rows), operand(av, rows), operand(ag, rows),
              operand(ab, rows), block(hT == h0 ? nullptr : h0, state),
              block(offsets, (batch + 1) * 8)}))
    return BS_ERR_INVALID_ARG;
  return done(with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    return bsolve::launch_gdelta<T>(
        gdelta_rows<T>(heads_k, heads_v, dk, dv, batch, rows, offsets, aq, ak, av, ag, ab, scale), h0,
        static_cast<T*>(o), ldo, hT, tape, work, static_cast<cudaStream_t>(stream));
  }));
}

bs_status bs_gdelta_backward_batched(bs_dtype dtype, int heads_k, int heads_v, int dk, int dv,
                                     int64_t batch, int64_t rows, const int64_t* offsets,
                                     const void* q, int64_t ldq, const void* k, int64_t ldk,
                                     const void* v, int64_t ldv, const float* g, int64_t ldg,
                                     const float* beta, int64_t ldbeta, double scale,
                                     const void* tape, const void* d_o, int64_t lddo,
                                     const float* dhT, void* dq, int64_t lddq, void* d_k,
                                     int64_t lddk, void* d_v, int64_t lddv, float* dg, int64_t lddg,
                                     float* dbeta, int64_t lddbeta, float* dh0, void* work,
                                     size_t work_bytes, void* stream) {
  const int es = element_size(dtype);
  const int64_t wk = int64_t(heads_k) * dk, wv = int64_t(heads_v) * dv;
  const RowArg aq{q, ldq, wk, es}, ak{k, ldk, wk, es}, av{v, ldv, wv, es}, ag{g, ldg, heads_v, 4},
      ab{beta, ldbeta, heads_v, 4}, ao{d_o, lddo, wv, es}, bq{dq, lddq, wk, es},
      bk{d_k, lddk, wk, es}, bv{d_v, lddv, wv, es}, bg{dg, lddg, heads_v, 4},
      bb{dbeta, lddbeta, heads_v, 4};
  const bs_status st = gdelta_sizes(dtype, heads_k, heads_v, dk, dv, batch, rows, scale,
                                    {aq, ak, av, ag, ab, ao, bq, bk, bv, bg, bb});
  if (st != BS_OK) return st;
  if (batch == 0) return BS_OK;
  if (!offsets && rows % batch != 0) return BS_ERR_INVALID_ARG;
  if (!aligned(dhT, 4) || !aligned(dh0, 4) || !aligned(tape, 16) || !aligned(work, 16) ||
      !aligned(offsets, 8))
    return BS_ERR_INVALID_ARG;
  const size_t need = bs_gdelta_backward_workspace(heads_v, dk, dv, batch, rows);
  if (!tape || !work || work_bytes < need) return BS_ERR_INVALID_ARG;
  const int64_t state = batch * heads_v * dk * dv * 4;
  if (!apart({operand(bq, rows), operand(bk, rows), operand(bv, rows), operand(bg, rows),
              operand(bb, rows), block(dh0, state), block(work, need)},
             {operand(aq, rows), operand(ak, rows), operand(av, rows), operand(ag, rows),
              operand(ab, rows), operand(ao, rows), block(dhT == dh0 ? nullptr : dhT, state),
              block(tape, bs_gdelta_tape(heads_v, dk, dv, batch, rows)),
              block(offsets, (batch + 1) * 8)}))
    return BS_ERR_INVALID_ARG;
  return done(with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    return bsolve::launch_gdelta_backward<T>(
        gdelta_rows<T>(heads_k, heads_v, dk, dv, batch, rows, offsets, aq, ak, av, ag, ab, scale),
        tape, static_cast<const T*>(d_o), lddo, dhT, static_cast<T*>(dq), lddq,
        static_cast<T*>(d_k), lddk, static_cast<T*>(d_v), lddv, dg, lddg, dbeta, lddbeta, dh0, work,
        static_cast<cudaStream_t>(stream));
  }));
}

bs_status bs_gdelta_step_batched(bs_dtype dtype, int heads_k, int heads_v, int dk, int dv,
                                 int64_t batch, const void* q, int64_t ldq, const void* k,
                                 int64_t ldk, const void* v, int64_t ldv, const float* g,
                                 int64_t ldg, const float* beta, int64_t ldbeta, double scale,
                                 float* state, int64_t num_slots, const int32_t* slots, void* o,
                                 int64_t ldo, void* stream) {
  const int es = element_size(dtype);
  const int64_t wk = int64_t(heads_k) * dk, wv = int64_t(heads_v) * dv;
  const RowArg aq{q, ldq, wk, es}, ak{k, ldk, wk, es}, av{v, ldv, wv, es}, ag{g, ldg, heads_v, 4},
      ab{beta, ldbeta, heads_v, 4}, ao{o, ldo, wv, es};
  if (num_slots < 0) return BS_ERR_INVALID_ARG;
  const bs_status st = gdelta_sizes(dtype, heads_k, heads_v, dk, dv, batch, batch, scale,
                                    {aq, ak, av, ag, ab, ao});
  if (st != BS_OK) return st;
  if (num_slots > kMaxRows) return BS_ERR_UNSUPPORTED;
  if (batch == 0) return BS_OK;
  if ((num_slots > 0 && !state) || (!slots && num_slots < batch) || !aligned(state, 4) ||
      !aligned(slots, 4))
    return BS_ERR_INVALID_ARG;
  if (!apart({operand(ao, batch), block(state, num_slots * heads_v * dk * dv * 4)},
             {operand(aq, batch), operand(ak, batch), operand(av, batch), operand(ag, batch),
              operand(ab, batch), block(slots, batch * 4)}))
    return BS_ERR_INVALID_ARG;
  return done(with_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    return bsolve::launch_gdelta_step<T>(
        gdelta_rows<T>(heads_k, heads_v, dk, dv, batch, batch, nullptr, aq, ak, av, ag, ab, scale),
        state, num_slots, slots, static_cast<T*>(o), ldo, static_cast<cudaStream_t>(stream));
  }));
}

size_t bs_gdelta_workspace(int heads_v, int64_t batch, int64_t rows) {
  if (heads_v < 1 || heads_v > 65535 || batch < 0 || rows < 0 || !gdelta_counts(batch, heads_v, rows))
    return 0;
  return bsolve::gdelta_workspace(heads_v, batch, rows);
}

size_t bs_gdelta_tape(int heads_v, int dk, int dv, int64_t batch, int64_t rows) {
  if (!gdelta_ok(BS_FP32, 1, heads_v, dk, dv) || batch < 0 || rows < 0 ||
      !gdelta_counts(batch, heads_v, rows))
    return 0;
  return bsolve::gdelta_tape(heads_v, dk, dv, batch, rows);
}

size_t bs_gdelta_backward_workspace(int heads_v, int dk, int dv, int64_t batch, int64_t rows) {
  if (!gdelta_ok(BS_FP32, 1, heads_v, dk, dv) || batch < 0 || rows < 0 ||
      !gdelta_counts(batch, heads_v, rows))
    return 0;
  return bsolve::gdelta_backward_workspace(heads_v, dk, dv, batch, rows);
}

int bs_gdelta_supported(bs_dtype dtype, int heads_k, int heads_v, int dk, int dv) {
  return gdelta_ok(dtype, heads_k, heads_v, dk, dv) ? 1 : 0;
}

}  // extern "C"
