// group_dx.hip -- dx[r] = dy[r] W_g over rows grouped by expert (see
// group_kernels.h).
#include "group_kernels.h"

namespace cco {

hipError_t launch_group_dx(bool f16, bool aligned, const GroupArgs &a, hipStream_t st) {
  return launch_op<kGroupDx>(f16, false, aligned, a, st);
}

}  // namespace cco
