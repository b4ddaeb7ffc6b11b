// The norms around a block on rows of __nv_bfloat16 (bs_gnorm calls of bsolve.h).
#include "gnorm.cuh"

namespace bsolve {
BSOLVE_GNORM(__nv_bfloat16)
}  // namespace bsolve
