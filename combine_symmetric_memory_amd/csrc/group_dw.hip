// group_dw.hip -- dW_g = sum over a group's rows of dy[r]^T x[r] (see
// group_kernels.h).
#include "group_kernels.h"

namespace cco {

hipError_t launch_group_dw(bool f16, bool out_f32, bool aligned, const GroupArgs &a,
                           hipStream_t st) {
  return launch_op<kGroupDw>(f16, out_f32, aligned, a, st);
}

}  // namespace cco
