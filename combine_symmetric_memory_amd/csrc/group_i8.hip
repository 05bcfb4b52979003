// group_i8.hip -- y[r] = xs[r] ws_g (x[r] W_g^T) over rows grouped by expert,
// 8-bit integers with a scale per row and per column (include/cco_ops.h).
//
// The tiles are those of the 16-bit products (group_tile.h): a 32x32x32 MFMA
// of 8-bit values takes the same 16 bytes a lane as the 32x32x16 one of 16-bit
// values, in the same time, so rows of k 8-bit values are fed as rows of k / 2
// 16-bit ones and a step of 128 bytes is twice the work.  The sums are exact
// (int32, at most 2^14 k); a result is its sum, rounded to fp32, times the two
// scales, so it carries three roundings and the output's.
#include "group_kernels.h"

namespace cco {

hipError_t launch_group_i8(int out_dtype, bool aligned, const GroupArgs &a, hipStream_t st) {
  switch (out_dtype) {
    case CCO_BF16: return launch_either<kGroupProduct, kElemI8, false, false>(aligned, a, st);
    case CCO_F16: return launch_either<kGroupProduct, kElemI8, true, false>(aligned, a, st);
    default: return launch_either<kGroupProduct, kElemI8, false, true>(aligned, a, st);
  }
}

}  // namespace cco
