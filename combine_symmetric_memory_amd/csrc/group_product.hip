// group_product.hip -- y[r] = x[r] W_g^T over rows grouped by expert, and the
// choice between the three directions (see group_kernels.h).
#include "group_kernels.h"

namespace cco {

hipError_t launch_group_product(bool f16, bool aligned, const GroupArgs &a, hipStream_t st) {
  return launch_op<kGroupProduct>(f16, false, aligned, a, st);
}

int group_parts(GroupOp op, int32_t groups, int32_t rows, int32_t n, int32_t k) {
  if (rows == 0) return 1;
  const int64_t tiles = even_tiles(op, 128, groups, rows, n, k);
  const int64_t kdim = op == kGroupProduct ? k : (op == kGroupDx ? n : rows / groups);
  const int64_t steps = kdim / 64;
  if (tiles > kPartTiles || steps < kSplitSteps) return 1;
  return (int)std::min<int64_t>(std::min<int64_t>(steps / kPartSteps, 2 * kNumCus / tiles),
                                kMaxParts);
}

hipError_t launch_group(GroupOp op, bool f16, bool out_f32, bool aligned, const GroupArgs &a,
                        hipStream_t st) {
  switch (op) {
    case kGroupProduct: return launch_group_product(f16, aligned, a, st);
    case kGroupDx: return launch_group_dx(f16, aligned, a, st);
    default: return launch_group_dw(f16, out_f32, aligned, a, st);
  }
}

}  // namespace cco
