// Gated linear recurrence (bs_grec calls of bsolve.h): forward over sequences, backward, and
// one row from kept states.
//
// One thread per sequence and channel walks the rows, so that neighbouring threads take
// neighbouring channels of one row.
#include "grec_math.cuh"
#include "kernels.h"
#include "row_types.cuh"

namespace bsolve {
namespace {

template <typename T>
__global__ void __launch_bounds__(128)
grec_forward_kernel(GrecRows<T> p, const float* __restrict__ lam, float kappa,
                    const float* h0, T* __restrict__ h, int64_t ldh, float* hT,
                    float* __restrict__ tape) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.channels) return;
  const float rate = grec_rate(lam[c], kappa);
  for (int64_t s = blockIdx.y; s < p.batch; s += gridDim.y) {
    int64_t start, end;
    sequence_rows(p.offsets, s, p.length, p.rows, &start, &end);
    float state = h0 ? h0[s * p.channels + c] : 0.f;
    const int64_t tb = tape_base(start, s);
    for (int64_t j = start; j < end; ++j) {
      if (tape && (j - start) % kTapeRows == 0)
        tape[(tb + (j - start) / kTapeRows) * p.channels + c] = state;
      const Gates g = grec_gates(to_f32(p.r[j * p.ldr + c]), to_f32(p.i[j * p.ldi + c]), rate);
      state = fmaf(g.a, state, g.s * g.si * to_f32(p.x[j * p.ldx + c]));
      h[j * ldh + c] = from_f32<T>(state);
    }
    if (hT) hT[s * p.channels + c] = state;
  }
}

template <typename T>
__global__ void __launch_bounds__(128)
grec_backward_kernel(GrecRows<T> p, const float* __restrict__ lam, float kappa,
                     const float* __restrict__ tape, const T* __restrict__ dh, int64_t lddh,
                     const float* dhT, T* __restrict__ dx, int64_t lddx, T* __restrict__ dr,
                     int64_t lddr, T* __restrict__ di, int64_t lddi, float* dh0,
                     float* __restrict__ partial) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.channels) return;
  const float rate = grec_rate(lam[c], kappa);
  for (int64_t s = blockIdx.y; s < p.batch; s += gridDim.y) {
    int64_t start, end;
    sequence_rows(p.offsets, s, p.length, p.rows, &start, &end);
    float carry = dhT ? dhT[s * p.channels + c] : 0.f;  // a_{t+1} g_{t+1}
    float sum = 0.f;
    const int64_t tb = tape_base(start, s);
    const int64_t chunks = (end - start + kTapeRows - 1) / kTapeRows;
    for (int64_t k = chunks - 1; k >= 0; --k) {
      const int64_t from = start + k * kTapeRows;
      const int n = static_cast<int>(end - from < kTapeRows ? end - from : kTapeRows);
      float before[kTapeRows];
      float state = tape[(tb + k) * p.channels + c];
      for (int j = 0; j < n; ++j) {
        before[j] = state;
        const int64_t row = from + j;
        const Gates g =
            grec_gates(to_f32(p.r[row * p.ldr + c]), to_f32(p.i[row * p.ldi + c]), rate);
        state = fmaf(g.a, state, g.s * g.si * to_f32(p.x[row * p.ldx + c]));
      }
      for (int j = n - 1; j >= 0; --j) {
        const int64_t row = from + j;
        const float x = to_f32(p.x[row * p.ldx + c]);
        const Gates g =
            grec_gates(to_f32(p.r[row * p.ldr + c]), to_f32(p.i[row * p.ldi + c]), rate);
        const float gt = to_f32(dh[row * lddh + c]) + carry;
        const float y = g.si * x;
        const float d = gt * (g.l * g.a * before[j] - y * g.a * g.a * (g.l * g.rs));
        dx[row * lddx + c] = from_f32<T>(gt * g.s * g.si);
        di[row * lddi + c] = from_f32<T>(gt * g.s * y * (g.ei * g.si));
        dr[row * lddr + c] = from_f32<T>(d * (g.er * g.sr));
        sum += d;
        carry = g.a * gt;
      }
    }
    if (dh0) dh0[s * p.channels + c] = carry;
    partial[s * p.channels + c] = sum;
  }
}

// dlam[c] = slope(lam_c) * sum of the partial sums, in their order.
__global__ void __launch_bounds__(128)
grec_dlam_kernel(int channels, int64_t parts, const float* __restrict__ lam,
                 const float* __restrict__ partial, float* __restrict__ dlam) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= channels) return;
  float sum = 0.f;
  for (int64_t k = 0; k < parts; ++k) sum += partial[k * channels + c];
  dlam[c] = sum * grec_rate_slope(lam[c]);
}

template <typename T>
__global__ void __launch_bounds__(128)
grec_step_kernel(GrecRows<T> p, const float* __restrict__ lam, float kappa,
                 float* __restrict__ state, int64_t num_slots, const int32_t* __restrict__ slots,
                 T* __restrict__ y, int64_t ldy) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= p.channels) return;
  const float rate = grec_rate(lam[c], kappa);
  for (int64_t j = blockIdx.y; j < p.batch; j += gridDim.y) {
    const int64_t slot = slots ? slots[j] : j;
    float h = 0.f;
    if (slot >= 0 && slot < num_slots) {
      const Gates g = grec_gates(to_f32(p.r[j * p.ldr + c]), to_f32(p.i[j * p.ldi + c]), rate);
      float* at = state + slot * p.channels + c;
      h = fmaf(g.a, *at, g.s * g.si * to_f32(p.x[j * p.ldx + c]));
      *at = h;
    }
    y[j * ldy + c] = from_f32<T>(h);
  }
}

dim3 grid_of(int channels, int64_t batch) {
  return dim3((channels + 127) / 128, static_cast<unsigned>(batch < 65535 ? batch : 65535));
}

}  // namespace

size_t grec_backward_workspace(int channels, int64_t batch, int64_t) {
  return static_cast<size_t>(batch) * channels * sizeof(float);
}

template <typename T>
cudaError_t launch_grec(const GrecRows<T>& p, const float* lam, float kappa, const float* h0,
                        T* h, int64_t ldh, float* hT, float* tape, cudaStream_t stream) {
  grec_forward_kernel<T><<<grid_of(p.channels, p.batch), 128, 0, stream>>>(p, lam, kappa, h0, h,
                                                                          ldh, hT, tape);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_grec_backward(const GrecRows<T>& p, const float* lam, float kappa,
                                 const float* tape, const T* dh, int64_t lddh, const float* dhT,
                                 T* dx, int64_t lddx, T* dr, int64_t lddr, T* di, int64_t lddi,
                                 float* dlam, float* dh0, void* work, cudaStream_t stream) {
  float* partial = static_cast<float*>(work);
  if (p.batch > 0) {
    grec_backward_kernel<T><<<grid_of(p.channels, p.batch), 128, 0, stream>>>(
        p, lam, kappa, tape, dh, lddh, dhT, dx, lddx, dr, lddr, di, lddi, dh0, partial);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  grec_dlam_kernel<<<(p.channels + 127) / 128, 128, 0, stream>>>(p.channels, p.batch, lam, partial,
                                                                 dlam);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_grec_step(const GrecRows<T>& p, const float* lam, float kappa, float* state,
                             int64_t num_slots, const int32_t* slots, T* y, int64_t ldy,
                             cudaStream_t stream) {
  grec_step_kernel<T><<<grid_of(p.channels, p.batch), 128, 0, stream>>>(p, lam, kappa, state,
                                                                       num_slots, slots, y, ldy);
  return cudaGetLastError();
}

#define BSOLVE_GREC(T)                                                                          \
  template cudaError_t launch_grec<T>(const GrecRows<T>&, const float*, float, const float*,    \
                                      T*, int64_t, float*, float*, cudaStream_t);               \
  template cudaError_t launch_grec_backward<T>(                                                 \
      const GrecRows<T>&, const float*, float, const float*, const T*, int64_t, const float*,   \
      T*, int64_t, T*, int64_t, T*, int64_t, float*, float*, void*, cudaStream_t);              \
  template cudaError_t launch_grec_step<T>(const GrecRows<T>&, const float*, float, float*,     \
                                           int64_t, const int32_t*, T*, int64_t, cudaStream_t);
BSOLVE_GREC(float)
BSOLVE_GREC(__nv_bfloat16)
BSOLVE_GREC(__half)
#undef BSOLVE_GREC

}  // namespace bsolve
