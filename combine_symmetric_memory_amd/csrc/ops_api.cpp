// ops_api.cpp -- the C ABI of include/cco_ops.h: argument checks and
// launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/cco_ops.h"
#include "ops_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool is_dtype(int32_t d) { return d == CCO_BF16 || d == CCO_F16 || d == CCO_F32; }
uintptr_t size_of(int32_t d) { return d == CCO_F32 ? 4 : 2; }
int status(hipError_t e) { return e == hipSuccess ? CCO_OK : CCO_ERR_HIP; }

bool route_ok(const cco_route_desc *d, int32_t dtype, int64_t ld, int32_t T) {
  if (!d || !is_dtype(dtype) || T < 0) return false;
  if (d->num_experts < 1 || d->num_experts > cco::kMaxExperts) return false;
  if (d->topk < 1 || d->topk > cco::kMaxTopk || d->topk > d->num_experts) return false;
  if (d->score != CCO_SCORE_SOFTMAX && d->score != CCO_SCORE_SIGMOID) return false;
  return ld >= d->num_experts;
}

cco::RouteArgs route_args(const cco_route_desc *d, const void *logits, int32_t dtype, int64_t ld,
                          int32_t T) {
  cco::RouteArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.dtype = dtype;
  a.E = d->num_experts;
  a.K = d->topk;
  a.T = T;
  a.score = d->score;
  a.renorm = d->renorm != 0;
  a.scale = d->scale;
  return a;
}

// row distances and widths the kernels address with 31-bit byte offsets
// inside a tile of up to 512 rows
bool width_ok(int64_t v) { return v >= 1 && v < (1 << 21); }

int group_call(cco::GroupOp op, const cco_groups *g, int32_t dtype, const void *a, int64_t lda,
               int32_t acols, const void *b, int64_t ldb, int32_t bcols, int32_t n, int32_t k,
               void *c, int64_t ldc, int32_t ccols, int32_t out_dtype, int32_t accumulate,
               void *workspace, uint64_t workspace_bytes, void *stream) {
  if (!g || g->groups < 1 || g->groups > cco::kMaxGroups || g->rows < 0) return CCO_ERR_INVALID_ARG;
  if (dtype != CCO_BF16 && dtype != CCO_F16) return CCO_ERR_INVALID_ARG;
  if (!width_ok(n) || !width_ok(k) || !width_ok(lda) || !width_ok(ldb) || !width_ok(ldc))
    return CCO_ERR_INVALID_ARG;
  if (lda < acols || ldb < bcols || ldc < ccols) return CCO_ERR_INVALID_ARG;
  if (out_dtype != dtype && !(op == cco::kGroupDw && out_dtype == CCO_F32))
    return CCO_ERR_INVALID_ARG;
  if (!g->first || !g->count || !aligned(g->first, 4) || !aligned(g->count, 4))
    return CCO_ERR_INVALID_ARG;
  // without rows the row operands may be NULL; only dw has work then (zeros)
  const bool rows = g->rows > 0, dw = op == cco::kGroupDw;
  if (!rows && (!dw || accumulate)) return CCO_OK;
  if (rows && (!a || !b || !c)) return CCO_ERR_INVALID_ARG;
  if (!c || !aligned(a, 2) || !aligned(b, 2) || !aligned(c, size_of(out_dtype)))
    return CCO_ERR_INVALID_ARG;
  if (workspace && (!aligned(workspace, 16) ||
                    workspace_bytes < cco_group_product_workspace(op, g, n, k)))
    return CCO_ERR_INVALID_ARG;
  cco::GroupArgs ga{};
  ga.groups = g->groups;
  ga.rows = g->rows;
  ga.first = g->first;
  ga.count = g->count;
  ga.a = (const char *)a;
  ga.b = (const char *)b;
  ga.c = (char *)c;
  ga.lda = lda;
  ga.ldb = ldb;
  ga.ldc = ldc;
  ga.n = n;
  ga.k = k;
  ga.accumulate = accumulate != 0;
  const bool vec = n % 8 == 0 && k % 8 == 0 && lda % 8 == 0 && ldb % 8 == 0 && ldc % 8 == 0 &&
                   aligned(a, 16) && aligned(b, 16) && aligned(c, 16);
  ga.parts = vec && workspace ? cco::group_parts(op, g->groups, g->rows, n, k) : 1;
  ga.ws = (float *)workspace;
  return status(cco::launch_group(op, dtype == CCO_F16, out_dtype == CCO_F32, vec, ga,
                                  (hipStream_t)stream));
}

bool norm_ok(const cco_block_norm_desc *d, int32_t T) {
  if (T < 0 || !d || d->hidden < 1 || d->hidden > cco::kMaxNormHidden || !is_dtype(d->dtype))
    return false;
  if (d->wdtype != CCO_F32 && d->wdtype != d->dtype) return false;
  if (!(d->eps >= 0.0f)) return false;
  if (d->gate_kind != CCO_GATE_NONE && d->gate_kind != CCO_GATE_CHANNEL &&
      d->gate_kind != CCO_GATE_TOKEN)
    return false;
  // a gate per token of no tokens may be NULL
  if (d->gate ? d->gate_kind == CCO_GATE_NONE
              : d->gate_kind == CCO_GATE_CHANNEL || (d->gate_kind == CCO_GATE_TOKEN && T > 0))
    return false;
  const uintptr_t ws = size_of(d->wdtype);
  return aligned(d->post, ws) && aligned(d->pre, ws) &&
         aligned(d->gate, d->gate_kind == CCO_GATE_TOKEN ? 4 : ws);
}

cco::NormArgs norm_args(const cco_block_norm_desc *d, const void *x, const void *y, int32_t T) {
  cco::NormArgs a{};
  a.H = d->hidden;
  a.T = T;
  a.w_f32 = d->wdtype == CCO_F32;
  a.w_f16 = d->wdtype == CCO_F16;
  a.gate_kind = d->gate_kind;
  a.scale = d->scale;
  a.eps = d->eps;
  a.post = d->post;
  a.gate = d->gate;
  a.pre = d->pre;
  a.x = x;
  a.y = y;
  return a;
}

struct DeviceGuard {
  int prev = -1;
  bool ok = false;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) return;
    ok = (prev == dev) || hipSetDevice(dev) == hipSuccess;
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

struct CombineNormCall {
  cco::CombineView view;
  cco::NormArgs args;
  hipStream_t st;
};

}  // namespace

extern "C" {

int cco_route(const cco_route_desc *d, const void *logits, int32_t dtype, int64_t ld,
              const float *bias, int32_t T, int32_t *idx, float *w, void *stream) {
  if (!route_ok(d, dtype, ld, T)) return CCO_ERR_INVALID_ARG;
  if (d->groups < 1 || d->groups > cco::kMaxRouteGroups || d->num_experts % d->groups != 0 ||
      d->kept < 1 || d->kept > d->groups || d->topk > d->kept * (d->num_experts / d->groups))
    return CCO_ERR_INVALID_ARG;
  if (!aligned(bias, 4)) return CCO_ERR_INVALID_ARG;
  if (T == 0) return CCO_OK;
  if (!logits || !idx || !w || !aligned(logits, size_of(dtype)) || !aligned(idx, 4) ||
      !aligned(w, 4))
    return CCO_ERR_INVALID_ARG;
  cco::RouteArgs a = route_args(d, logits, dtype, ld, T);
  a.groups = d->groups;
  a.kept = d->kept;
  a.bias = bias;
  a.idx = idx;
  a.w = w;
  return status(cco::launch_route(a, (hipStream_t)stream));
}

int cco_route_grad(const cco_route_desc *d, const void *logits, int32_t dtype, int64_t ld,
                   const int32_t *idx, const float *dw, int32_t T, void *dlogits, int64_t lddl,
                   void *stream) {
  if (!route_ok(d, dtype, ld, T) || lddl < d->num_experts) return CCO_ERR_INVALID_ARG;
  if (T == 0) return CCO_OK;
  if (!logits || !idx || !dw || !dlogits || !aligned(logits, size_of(dtype)) ||
      !aligned(dlogits, size_of(dtype)) || !aligned(idx, 4) || !aligned(dw, 4))
    return CCO_ERR_INVALID_ARG;
  cco::RouteArgs a = route_args(d, logits, dtype, ld, T);
  a.idx = const_cast<int32_t *>(idx);
  a.dw = dw;
  a.dlogits = dlogits;
  a.lddl = lddl;
  return status(cco::launch_route_grad(a, (hipStream_t)stream));
}

uint64_t cco_group_product_workspace(int32_t op, const cco_groups *g, int32_t n, int32_t k) {
  if (!g || g->groups < 1 || g->groups > cco::kMaxGroups || g->rows < 0 || !width_ok(n) ||
      !width_ok(k) || op < CCO_GROUP_PRODUCT || op > CCO_GROUP_DW || n % 8 != 0 || k % 8 != 0)
    return 0;
  const uint64_t parts = (uint64_t)cco::group_parts((cco::GroupOp)op, g->groups, g->rows, n, k);
  if (parts <= 1) return 0;
  const uint64_t out = op == CCO_GROUP_DW
                           ? (uint64_t)g->groups * (uint64_t)n * (uint64_t)k
                           : (uint64_t)g->rows * (uint64_t)(op == CCO_GROUP_PRODUCT ? n : k);
  return parts * out * sizeof(float);
}

int cco_group_product(const cco_groups *g, int32_t dtype, const void *x, int64_t ldx,
                      const void *w, int32_t n, int32_t k, void *y, int64_t ldy, void *workspace,
                      uint64_t workspace_bytes, void *stream) {
  return group_call(cco::kGroupProduct, g, dtype, x, ldx, k, w, k, k, n, k, y, ldy, n, dtype, 0,
                    workspace, workspace_bytes, stream);
}

int cco_group_product_dx(const cco_groups *g, int32_t dtype, const void *dy, int64_t lddy,
                         const void *w, int32_t n, int32_t k, void *dx, int64_t lddx,
                         void *workspace, uint64_t workspace_bytes, void *stream) {
  return group_call(cco::kGroupDx, g, dtype, dy, lddy, n, w, k, k, n, k, dx, lddx, k, dtype, 0,
                    workspace, workspace_bytes, stream);
}

int cco_group_product_dw(const cco_groups *g, int32_t dtype, const void *dy, int64_t lddy,
                         const void *x, int64_t ldx, int32_t n, int32_t k, void *dw,
                         int32_t out_dtype, int32_t accumulate, void *workspace,
                         uint64_t workspace_bytes, void *stream) {
  return group_call(cco::kGroupDw, g, dtype, dy, lddy, n, x, ldx, k, n, k, dw, k, k, out_dtype,
                    accumulate, workspace, workspace_bytes, stream);
}

int cco_block_norm(const cco_block_norm_desc *d, const void *x, const void *y, int32_t T,
                   void *out, void *u, void *stream) {
  if (!norm_ok(d, T)) return CCO_ERR_INVALID_ARG;
  const uintptr_t es = size_of(d->dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(out, es) || !aligned(u, es))
    return CCO_ERR_INVALID_ARG;
  if (T == 0) return CCO_OK;
  if (!x || (d->pre != nullptr) != (u != nullptr) || (!out && !u)) return CCO_ERR_INVALID_ARG;
  if (!y && (out || d->post || d->gate)) return CCO_ERR_INVALID_ARG;
  cco::NormArgs a = norm_args(d, x, y, T);
  a.out = out;
  a.u = u;
  return status(cco::launch_block_norm(d->dtype, a, (hipStream_t)stream));
}

uint64_t cco_block_norm_grad_workspace(const cco_block_norm_desc *d, int32_t T) {
  if (!norm_ok(d, T)) return 0;
  const uint64_t sums = (d->post || d->gate_kind == CCO_GATE_CHANNEL) + (d->pre != nullptr);
  return sums * (uint64_t)cco::norm_grad_workgroups(d->hidden, T) * (uint64_t)d->hidden *
         sizeof(float);
}

int cco_block_norm_grad(const cco_block_norm_desc *d, const void *x, const void *y,
                        const void *dout, const void *du, int32_t T, void *dx, void *dy,
                        float *dpost, float *dgate, float *dpre, void *workspace,
                        uint64_t workspace_bytes, void *stream) {
  if (!norm_ok(d, T)) return CCO_ERR_INVALID_ARG;
  const uintptr_t es = size_of(d->dtype);
  if (!aligned(x, es) || !aligned(y, es) || !aligned(dout, es) || !aligned(du, es) ||
      !aligned(dx, es) || !aligned(dy, es) || !aligned(dpost, 4) || !aligned(dgate, 4) ||
      !aligned(dpre, 4) || !aligned(workspace, 16))
    return CCO_ERR_INVALID_ARG;
  if ((d->post != nullptr) != (dpost != nullptr) || (d->pre != nullptr) != (dpre != nullptr))
    return CCO_ERR_INVALID_ARG;
  if ((d->gate_kind != CCO_GATE_NONE) != (dgate != nullptr) &&
      !(T == 0 && d->gate_kind == CCO_GATE_TOKEN))
    return CCO_ERR_INVALID_ARG;
  if (T > 0) {
    if (!x || !dx || (y != nullptr) != (dy != nullptr) || (!dout && !du) ||
        (d->pre != nullptr) != (du != nullptr))
      return CCO_ERR_INVALID_ARG;
    if (!y && (d->post || d->gate)) return CCO_ERR_INVALID_ARG;
  }
  const uint64_t need = cco_block_norm_grad_workspace(d, T);
  if (need > 0 && (!workspace || workspace_bytes < need)) return CCO_ERR_INVALID_ARG;
  cco::NormArgs a = norm_args(d, x, y, T);
  a.dout = dout;
  a.du = du;
  a.dx = dx;
  a.dy = dy;
  a.dpost = dpost;
  a.dgate = dgate;
  a.dpre = dpre;
  a.partial = (float *)workspace;
  return status(cco::launch_block_norm_grad(d->dtype, a, (hipStream_t)stream));
}

int cco_moe_combine_norm(cco_moe *m, const float *weights, const cco_block_norm_desc *d,
                         const void *x, int32_t T, void *y_out, void *out, void *u,
                         void *stream) {
  CombineNormCall call{};
  int device = 0;
  int32_t hidden = 0;
  if (!m || !norm_ok(d, T) || d->dtype != CCO_BF16) return CCO_ERR_INVALID_ARG;
  const int rc = cco::moe_combine_view(m, T, &call.view, &device, &hidden);
  if (rc != CCO_OK) return rc;
  if (d->hidden != hidden) return CCO_ERR_INVALID_ARG;
  if (T == 0) return CCO_OK;
  if (!weights || !x || (d->pre != nullptr) != (u != nullptr) || (!out && !u))
    return CCO_ERR_INVALID_ARG;
  if (!aligned(weights, 4) || !aligned(x, 16) || !aligned(y_out, 16) || !aligned(out, 16) ||
      !aligned(u, 16))
    return CCO_ERR_INVALID_ARG;
  DeviceGuard dg(device);
  if (!dg.ok) return CCO_ERR_HIP;
  call.view.w = weights;
  call.view.y_out = y_out;
  call.args = norm_args(d, x, nullptr, T);
  call.args.out = out;
  call.args.u = u;
  call.st = (hipStream_t)stream;
  return cco::moe_timed_combine(
      m, call.st,
      [](void *p) {
        CombineNormCall *c = (CombineNormCall *)p;
        return cco::launch_combine_norm(c->view, c->args, c->st);
      },
      &call);
}

}  // extern "C"
