// The norms around a block on rows of float (bs_gnorm calls of bsolve.h).
#include "gnorm.cuh"

namespace bsolve {
BSOLVE_GNORM(float)
}  // namespace bsolve
