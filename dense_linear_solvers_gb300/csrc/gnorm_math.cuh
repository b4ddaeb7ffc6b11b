// The gate of the norms around a block (bs_gnorm calls).
#pragma once

#include <cuda_runtime.h>

namespace bsolve {

struct Gate {
  float act, slope;  // act(z) and its derivative
};

// kind: a bs_gate. sigma(z) = 1 / (1 + e^-z), 1 - sigma(z) = e^-z sigma(z).
__device__ __forceinline__ Gate gate_of(float z, int kind) {
  if (kind == 2) return {z, 1.f};
  const float e = __expf(-z);
  const float s = __frcp_rn(1.f + e);
  const float c = z < -80.f ? 1.f : e * s;
  if (kind == 1) return {s, s * c};
  return {z * s, fmaf(z * s, c, s)};
}

}  // namespace bsolve
