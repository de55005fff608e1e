// The residual operator's backward for one storage type (a file each, to build them in parallel).
#include "residual_bwd.h"

namespace moe {

hipError_t launch_residual_bwd_bf16(const ResidualBwdArgs& a, hipStream_t s) {
  return launch_bwd<bf16_t>(a, s);
}

}  // namespace moe
