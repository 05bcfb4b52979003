// ops_internal.h -- descriptors and launchers of the operators in
// include/cco_ops.h, shared by their host side (ops_api.cpp) and kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/cco_ops.h"
#include "cco_internal.h"

namespace cco {

constexpr int kNumCus = 256;          // compute units of one MI355X
constexpr int kMaxGroups = 1024;      // groups of a grouped product
constexpr int kMaxRouteGroups = 64;   // groups of experts in the router
constexpr int kMaxNormHidden = 16384; // a row stays in one workgroup's registers

// ------------------------------------------------------------- the router
struct RouteArgs {
  const void *logits;
  int64_t ld;
  int32_t dtype;
  int32_t E, K, T;
  int32_t score, renorm;
  float scale;
  int32_t groups, kept;
  const float *bias;
  int32_t *idx;       // choice: out; gradient: in
  float *w;           // choice: out
  const float *dw;    // gradient
  void *dlogits;
  int64_t lddl;
};
hipError_t launch_route(const RouteArgs &a, hipStream_t st);
hipError_t launch_route_grad(const RouteArgs &a, hipStream_t st);

// ----------------------------------------------------- products by group
// C (+)= A op B per group; which operand is which depends on the direction:
//   product  A = x [rows][k], B = w [g][n][k], C = y [rows][n]
//   dx       A = dy [rows][n], B = w [g][n][k], C = dx [rows][k]
//   dw       A = dy [rows][n], B = x [rows][k], C = dw [g][n][k]
struct GroupArgs {
  int32_t groups, rows;
  const int32_t *first, *count;
  const char *a, *b;
  char *c;
  int64_t lda, ldb, ldc;  // elements
  int32_t n, k;
  int32_t accumulate;     // dw: add to C
  int32_t parts;          // parts of the reduction, whose sums go to ws: 1 unsplit
  float *ws;              // [parts][rows of C][columns of C]
};
enum GroupOp { kGroupProduct = 0, kGroupDx = 1, kGroupDw = 2 };
// Parts a product of whole 16-byte rows is split into when it has workspace.
int group_parts(GroupOp op, int32_t groups, int32_t rows, int32_t n, int32_t k);
hipError_t launch_group_product(bool f16, bool aligned, const GroupArgs &a, hipStream_t st);
hipError_t launch_group_dx(bool f16, bool aligned, const GroupArgs &a, hipStream_t st);
hipError_t launch_group_dw(bool f16, bool out_f32, bool aligned, const GroupArgs &a,
                           hipStream_t st);
hipError_t launch_group(GroupOp op, bool f16, bool out_f32, bool aligned, const GroupArgs &a,
                        hipStream_t st);

// -------------------------------------------------------------- the norms
struct NormArgs {
  int32_t H, T;
  int32_t w_f32;       // post, pre and a channel gate are fp32, or the rows' type:
  int32_t w_f16;       // ... fp16 (else bf16)
  int32_t gate_kind;
  float scale, eps;
  const void *post, *gate, *pre;
  const void *x, *y, *dout, *du;
  void *out, *u;       // forward
  void *dx, *dy;       // gradient
  float *dpost, *dgate, *dpre, *partial;
};
// Workgroups of the gradient's row pass, and the column sums each leaves.
int norm_grad_workgroups(int32_t H, int32_t T);
hipError_t launch_block_norm(int dtype, const NormArgs &a, hipStream_t st);
hipError_t launch_block_norm_grad(int dtype, const NormArgs &a, hipStream_t st);
// The combine's view of one layer for the fused form.
struct CombineView {
  MoeArgs moe;
  uint64_t win;
  const float *w;
  void *y_out;
};
hipError_t launch_combine_norm(const CombineView &c, const NormArgs &a, hipStream_t st);

// What the fused form needs of a layer (defined in api.cpp, where the layer
// is): checks, then `fn` launched on `st` as the layer's combine.
int moe_combine_view(::cco_moe *m, int32_t T, CombineView *out, int *device, int32_t *hidden);
int moe_timed_combine(::cco_moe *m, hipStream_t st, hipError_t (*fn)(void *), void *ctx);

}  // namespace cco
