// The gradients of q, k, g and beta from what both chains have left (bs_gdelta_backward_batched).
#pragma once

#include "gdelta_tile.cuh"

namespace bsolve {

template <typename T>
struct GdeltaGrads {
  const T* dout;
  int64_t lddo;
  T* dq;
  int64_t lddq;
  T* dk;
  int64_t lddk;
  float* dg;
  int64_t lddg;
  float* dbeta;
  int64_t lddbeta;
  const uint4* forward;   // states in front of the chunks, and M
  const uint4* backward;  // gradients of the states behind them, and dU
  const Prepared* prepared;
};

template <typename T>
cudaError_t launch_gdelta_grad(const GdeltaRows<T>& p, const GdeltaGrads<T>& g, cudaStream_t stream);

}  // namespace bsolve
