// The norms around a block on rows of __half (bs_gnorm calls of bsolve.h).
#include "gnorm.cuh"

namespace bsolve {
BSOLVE_GNORM(__half)
}  // namespace bsolve
