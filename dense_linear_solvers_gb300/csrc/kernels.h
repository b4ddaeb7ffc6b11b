// Host-side launchers of the CUDA kernels (internal to libbsolve.so).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bsolve {

// LU + solve, rows in registers, 1 <= n <= 32, 0 <= nrhs <= 8 (0: factor only). The
// LU and Cholesky launchers below take nrhs = 0 the same way.
template <typename T>
cudaError_t launch_lu_reg(int layout, int n, int nrhs, int64_t batch, T* A, T* B,
                          int32_t* ipiv, int32_t* info, cudaStream_t stream);
// The same on the interleaved batched layout (element e of system s at
// (s / ilv) * ilv * size + e * ilv + s % ilv for A, B and ipiv), 1 <= nrhs <= 8.
template <typename T>
cudaError_t launch_lu_reg_il(int layout, int n, int nrhs, int64_t batch, int64_t ilv, T* A, T* B,
                             int32_t* ipiv, int32_t* info, cudaStream_t stream);

// LU + solve, one block of four warps per system in shared memory, 1 <= n <= 128, 0 <= nrhs <= 8.
template <typename T>
cudaError_t launch_lu_smem(int layout, int n, int nrhs, int64_t batch, T* A, T* B,
                           int32_t* ipiv, int32_t* info, cudaStream_t stream);

// The same with the options of the _ex calls: TDLS threshold tau in (0, 1], RUDA status
// contract (ruda != 0); any 1 <= n <= 128.
// LU + solve for FP32, 8 < n <= 16, nrhs <= 8 (0: factor only), two rows per lane and
// four systems per warp; ilv: the element stride of an interleaved batched layout (1: plain).
cudaError_t launch_lu_rows2(int layout, int n, int nrhs, int64_t batch, float* A, float* B,
                            int32_t* ipiv, int32_t* info, cudaStream_t stream, int64_t ilv = 1);

template <typename T>
cudaError_t launch_lu_smem_ex(int layout, int n, int nrhs, int64_t batch, T* A, T* B,
                              int32_t* ipiv, int32_t* info, double tau, int ruda,
                              cudaStream_t stream, int64_t ilv = 1, int scale = 0);

// Solve with a stored factor: getrs (L\U and the 1-based swap sequence of getrf) and
// potrs (Cholesky factor), 1 <= n <= 128.
// Any nrhs >= 1 (a register tier's worth at a time). zinfo (may be null): X = 0 where
// zinfo[s] != 0.
// ilv: the element stride of an interleaved batched layout (1: the plain layout; > 1:
// n <= 128, one warp per system).
template <typename T>
cudaError_t launch_getrs(int layout, int n, int nrhs, int64_t batch, const T* LU,
                         const int32_t* ipiv, T* B, const int32_t* zinfo, cudaStream_t stream,
                         int64_t ilv = 1);
template <typename T>
cudaError_t launch_potrs(int layout, int n, int nrhs, int64_t batch, const T* L, T* B,
                         const int32_t* zinfo, cudaStream_t stream, int64_t ilv = 1);
// potrs for FP64, 1 <= n <= 32, nrhs == 1: one system per lane, the factor streamed by
// columns through shared memory (layout bit 0: the factor's storage order).
cudaError_t launch_potrs_lane(int layout, int n, int nrhs, int64_t batch, const double* L,
                              double* B, const int32_t* zinfo, cudaStream_t stream);

// The mirror solve of the row-major reading (U^T z = b, L^T w = z, x = P^T w) with the LU
// factor of S, the stored array read column-major; layout packs S's order (bit 0) and B's.
template <typename T>
cudaError_t launch_getrs_mirror(int layout, int n, int nrhs, int64_t batch, const T* S,
                                const int32_t* ipiv, T* B, const int32_t* zinfo,
                                cudaStream_t stream, int64_t ilv = 1);

// The Cholesky launchers (chol_smem, chol_sys, potrs) take a packed storage-order code:
// bit 0 for A (or the factor), bit 1 for B; upper fill is passed as the lower fill of A in
// the other order.
// Lower Cholesky + solve, one warp per system in shared memory, 1 <= n <= 128.
template <typename T>
cudaError_t launch_chol_smem(int layout, int n, int nrhs, int64_t batch, T* A, T* B,
                             int32_t* info, cudaStream_t stream);

// The same under the RUDA status contract (ruda != 0): -1 non-finite input, -2 input
// not symmetric (the whole matrix is read), -3 non-finite result; failures zeroed.
template <typename T>
cudaError_t launch_chol_smem_ex(int layout, int n, int nrhs, int64_t batch, T* A, T* B,
                                int32_t* info, int ruda, cudaStream_t stream, int64_t ilv = 1);

// Lower Cholesky factor (potrf) for 128 < n <= 256 on a cluster of four CTAs, the tiles
// of one system spread over their shared memory; layout bit 0: A's storage order.
template <typename T>
cudaError_t launch_chol_cluster(int layout, int n, int64_t batch, T* A, int32_t* info,
                                cudaStream_t stream);
// potrs for 128 < n <= 256, any nrhs >= 1: one CTA per system (packed storage-order code).
template <typename T>
cudaError_t launch_potrs_big(int layout, int n, int nrhs, int64_t batch, const T* L, T* B,
                             const int32_t* zinfo, cudaStream_t stream);

// Lower Cholesky + solve, sixteen systems per block in lockstep, 1 <= n <= 32.
template <typename T>
cudaError_t launch_chol_sys(int layout, int n, int nrhs, int64_t batch, T* A, T* B,
                            int32_t* info, cudaStream_t stream, int64_t ilv = 1);

// Block-tridiagonal block-Cholesky sweep, one thread per system, 1 <= bs <= 8.
template <typename T>
cudaError_t launch_bdsv(int nbr, int bs, int64_t batch, T* strips, T* xpad, int32_t* info,
                        cudaStream_t stream);

// The factor sweep alone, and the substitutions alone on factored strips.
template <typename T>
cudaError_t launch_bdsv_factor(int nbr, int bs, int64_t batch, T* strips, int32_t* info,
                               cudaStream_t stream);
template <typename T>
cudaError_t launch_bdsv_solve(int nbr, int bs, int64_t batch, const T* strips, T* xpad,
                              cudaStream_t stream);

// Block-tridiagonal matrix-vector product on padded vectors, 1 <= bs <= 8; ypad2, when
// not null, receives the same product too.
template <typename T>
cudaError_t launch_bdmv(int nbr, int bs, int64_t batch, const T* strips, const T* xpad, T* ypad,
                        T* ypad2, cudaStream_t stream);

// Shared memory one system needs in the shared-memory kernels.
size_t lu_cta_bytes(int n, int nrhs, int elem_size);
size_t chol_smem_bytes(int n, int nrhs, int elem_size);
size_t chol_sys_bytes(int n, int nrhs, int elem_size);

// SMs of the GPU that the row operators' grids and thresholds are made for.
constexpr int kSms = 152;

// The row operators (bs_grec and bs_gnorm calls): operands of T (float, __nv_bfloat16 or
// __half) as rows of contiguous elements, row j at j * ld of its base.

// The inputs of a gated linear recurrence. offsets == nullptr: sequences of `length` rows.
template <typename T>
struct GrecRows {
  int channels;
  int64_t batch, rows, length;
  const int64_t* offsets;
  const T *x, *r, *i;
  int64_t ldx, ldr, ldi;
};

template <typename T>
cudaError_t launch_grec(const GrecRows<T>& p, const float* lam, float kappa, const float* h0,
                        T* h, int64_t ldh, float* hT, float* tape, cudaStream_t stream);
template <typename T>
cudaError_t launch_grec_backward(const GrecRows<T>& p, const float* lam, float kappa,
                                 const float* tape, const T* dh, int64_t lddh, const float* dhT,
                                 T* dx, int64_t lddx, T* dr, int64_t lddr, T* di, int64_t lddi,
                                 float* dlam, float* dh0, void* work, cudaStream_t stream);
size_t grec_backward_workspace(int channels, int64_t batch, int64_t rows);
template <typename T>
cudaError_t launch_grec_step(const GrecRows<T>& p, const float* lam, float kappa, float* state,
                             int64_t num_slots, const int32_t* slots, T* y, int64_t ldy,
                             cudaStream_t stream);

// The operands of the norms around a block; null: absent (see bsolve.h).
template <typename T>
struct GnormRows {
  int64_t rows;
  int width;
  const T *f, *z, *x;
  int64_t ldf, ldz, ldx;
  const float *w_post, *scale, *w_pre;
  float eps;
  int gate;
};

template <typename T>
struct GnormGrads {
  const T *dy, *du;
  int64_t lddy, lddu;
  T *df, *dz, *dx;
  int64_t lddf, lddz, lddx;
  float *dw_post, *dscale, *dw_pre;
};

template <typename T>
cudaError_t launch_gnorm(const GnormRows<T>& p, T* y, int64_t ldy, T* u, int64_t ldu,
                         cudaStream_t stream);
template <typename T>
cudaError_t launch_gnorm_backward(const GnormRows<T>& p, const GnormGrads<T>& g, void* work,
                                  cudaStream_t stream);
size_t gnorm_backward_workspace(int width, int64_t rows);

// Rows in e4m3 with one FP32 scale for each 128 elements.
struct Bytes8 {
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t lds;
};

template <typename T>
cudaError_t launch_gnorm_q8(const GnormRows<T>& p, T* y, int64_t ldy, const Bytes8& out,
                            cudaStream_t stream);

// y (m x n) from a (m x k) and w (n x k) in e4m3, a scale for each 128 of a row of a and for each
// 128 x 128 of w.
template <typename T>
struct GemmQ8 {
  int64_t m, n, k;
  const uint8_t* a;
  int64_t lda;
  const float* sa;
  int64_t ldsa;
  const uint8_t* w;
  int64_t ldw;
  const float* sw;
  int64_t ldsw;
  T* y;
  int64_t ldy;
};

template <typename T>
cudaError_t launch_gemm_q8(const GemmQ8<T>& g, cudaStream_t stream);

// The inputs of a gated delta rule: rows of heads_k heads of dk elements (q, k), heads_v of dv (v), and
// FP32 rows of heads_v (g, beta). offsets == nullptr: sequences of `length` rows.
template <typename T>
struct GdeltaRows {
  int heads_k, heads_v, dk, dv;
  int64_t batch, rows, length;
  const int64_t* offsets;
  const T *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const float *g, *beta;
  int64_t ldg, ldbeta;
  float scale;
};

// Whether every head of every row starts on a 16-byte boundary and ends on one.
template <typename T>
bool gdelta_aligned(const T* p, int64_t ld, int width) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * sizeof(T)) |
           static_cast<uintptr_t>(width * sizeof(T))) & 15) == 0;
}

template <typename T>
cudaError_t launch_gdelta(const GdeltaRows<T>& p, const float* h0, T* o, int64_t ldo, float* hT,
                          void* tape, void* work, cudaStream_t stream);
template <typename T>
cudaError_t launch_gdelta_backward(const GdeltaRows<T>& p, const void* tape, const T* dout,
                                   int64_t lddo, const float* dhT, T* dq, int64_t lddq, T* dk,
                                   int64_t lddk, T* dv, int64_t lddv, float* dg, int64_t lddg,
                                   float* dbeta, int64_t lddbeta, float* dh0, void* work,
                                   cudaStream_t stream);
// One row of it for each of p.batch sequences.
template <typename T>
cudaError_t launch_gdelta_step(const GdeltaRows<T>& p, float* state, int64_t num_slots,
                               const int32_t* slots, T* o, int64_t ldo, cudaStream_t stream);
size_t gdelta_workspace(int heads_v, int64_t batch, int64_t rows);
size_t gdelta_tape(int heads_v, int dk, int dv, int64_t batch, int64_t rows);
size_t gdelta_backward_workspace(int heads_v, int dk, int dv, int64_t batch, int64_t rows);

// Records a launch error as the one bs_last_cuda_error() returns.
void record_cuda_error(cudaError_t e);

}  // namespace bsolve
