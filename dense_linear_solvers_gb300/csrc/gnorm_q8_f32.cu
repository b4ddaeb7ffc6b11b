// The norms around a block on rows of float (bs_gnorm calls of bsolve.h).
#include "gnorm.cuh"

namespace bsolve {
BSOLVE_GNORM_Q8(float)
}  // namespace bsolve
