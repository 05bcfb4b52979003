// serve_api.cpp -- the C ABI of include/cco_ops.h, the operators in 8 bits and
// the layer for a few tokens: argument checks and launches.
#include <hip/hip_runtime.h>

#include "../../include/cco_ops.h"
#include "ops_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool is_dtype(int32_t d) { return d == CCO_BF16 || d == CCO_F16 || d == CCO_F32; }
uintptr_t size_of(int32_t d) { return d == CCO_F32 ? 4 : 2; }
int status(hipError_t e) { return e == hipSuccess ? CCO_OK : CCO_ERR_HIP; }

// widths and row distances, which the kernels address with 32-bit offsets
// inside a tile
bool width_ok(int64_t v) { return v >= 1 && v < (1 << 21); }
// |sum| <= 2^14 k stays inside an int32
constexpr int32_t kMaxI8Sum = (1 << 17) - 1;

bool groups_ok(const cco_groups *g) {
  return g && g->groups >= 1 && g->groups <= cco::kMaxGroups && g->rows >= 0;
}
bool few_ok(const cco_few_desc *d, int32_t T) {
  if (!d || T < 0 || d->hidden < 1 || d->inter < 1 || d->hidden > (1 << 20) ||
      d->inter > (1 << 19))
    return false;
  if (d->num_experts < 1 || d->num_experts > cco::kMaxExperts) return false;
  if (d->topk < 1 || d->topk > cco::kMaxTopk) return false;
  if (d->dtype != CCO_BF16 && d->dtype != CCO_F16) return false;
  return d->wdtype == d->dtype || d->wdtype == CCO_I8;
}
// The workspace: h and the parts' sums.
struct FewSpace {
  int32_t pitch, parts;
  uint64_t partial, bytes;  // where the sums begin, and the whole
};
FewSpace few_space(const cco_few_desc *d, int32_t T) {
  FewSpace s{};
  s.pitch = (d->inter + 255) / 256 * 256;  // whole chunks of the down product
  s.parts = cco::few_parts(d->wdtype == CCO_I8, T, d->topk, d->num_experts, d->hidden, d->inter);
  s.partial = (uint64_t)T * d->topk * 2 * s.pitch * sizeof(uint16_t);
  s.bytes = s.partial +
            (s.parts > 1 ? (uint64_t)s.parts * T * (uint64_t)d->hidden * sizeof(float) : 0);
  return s;
}

}  // namespace

extern "C" {

int cco_quant_rows(const void *x, int32_t dtype, int64_t ldx, int32_t rows, int32_t cols,
                   int32_t swiglu, int8_t *q, int64_t ldq, float *s, int64_t lds, void *stream) {
  if (!is_dtype(dtype) || rows < 0 || !width_ok(cols) || !width_ok(ldx) || !width_ok(ldq) ||
      lds < 1 || lds >= (1ll << 40))
    return CCO_ERR_INVALID_ARG;
  if (ldx < (swiglu ? 2 : 1) * (int64_t)cols || ldq < cols) return CCO_ERR_INVALID_ARG;
  if (!aligned(x, size_of(dtype)) || !aligned(s, 4)) return CCO_ERR_INVALID_ARG;
  if (rows == 0) return CCO_OK;
  if (!x || !q || !s) return CCO_ERR_INVALID_ARG;
  cco::QuantArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  a.q = q;
  a.ldq = ldq;
  a.s = s;
  a.lds = lds;
  return status(cco::launch_quant(dtype, swiglu != 0, a, (hipStream_t)stream));
}

uint64_t cco_group_product_i8_workspace(const cco_groups *g, int32_t n, int32_t k) {
  if (!groups_ok(g) || !width_ok(n) || k < 1 || k > kMaxI8Sum || n % 8 != 0 || k % 16 != 0)
    return 0;
  const uint64_t parts =
      (uint64_t)cco::group_parts(cco::kGroupProduct, g->groups, g->rows, n, k / 2);
  return parts <= 1 ? 0 : parts * (uint64_t)g->rows * (uint64_t)n * sizeof(int32_t);
}

int cco_group_product_i8(const cco_groups *g, const int8_t *x, int64_t ldx, const float *xs,
                         int64_t ldxs, const int8_t *w, const float *ws, int32_t n, int32_t k,
                         void *y, int32_t out_dtype, int64_t ldy, void *workspace,
                         uint64_t workspace_bytes, void *stream) {
  if (!groups_ok(g) || !is_dtype(out_dtype)) return CCO_ERR_INVALID_ARG;
  if (!width_ok(n) || k < 1 || k > kMaxI8Sum || !width_ok(ldx) || !width_ok(ldy) || ldx < k ||
      ldy < n || ldxs < 1 || ldxs >= (1ll << 40))
    return CCO_ERR_INVALID_ARG;
  if (!g->first || !g->count || !aligned(g->first, 4) || !aligned(g->count, 4))
    return CCO_ERR_INVALID_ARG;
  if (!aligned(xs, 4) || !aligned(ws, 4) || !aligned(y, size_of(out_dtype)))
    return CCO_ERR_INVALID_ARG;
  if (workspace && (!aligned(workspace, 16) ||
                    workspace_bytes < cco_group_product_i8_workspace(g, n, k)))
    return CCO_ERR_INVALID_ARG;
  if (g->rows == 0) return CCO_OK;
  if (!x || !xs || !w || !ws || !y) return CCO_ERR_INVALID_ARG;
  const bool vec = n % 8 == 0 && k % 16 == 0 && ldx % 16 == 0 && ldy % 8 == 0 && aligned(x, 16) &&
                   aligned(w, 16) && aligned(ws, 16) && aligned(y, 16);
  const int32_t pair = vec ? 2 : 1;
  cco::GroupArgs a{};
  a.groups = g->groups;
  a.rows = g->rows;
  a.first = g->first;
  a.count = g->count;
  a.a = (const char *)x;
  a.b = (const char *)w;
  a.c = (char *)y;
  a.lda = ldx / pair;
  a.ldb = k / pair;
  a.ldc = ldy;
  a.n = n;
  a.k = k / pair;
  a.parts = vec && workspace
                ? cco::group_parts(cco::kGroupProduct, g->groups, g->rows, n, k / pair)
                : 1;
  a.ws = (float *)workspace;
  a.rs = xs;
  a.ldrs = ldxs;
  a.cs = ws;
  return status(cco::launch_group_i8(out_dtype, vec, a, (hipStream_t)stream));
}

uint64_t cco_moe_few_workspace(const cco_few_desc *d, int32_t T) {
  if (!few_ok(d, T) || T > cco::kFewMaxTokens) return 0;
  return T == 0 ? 0 : few_space(d, T).bytes;
}

int cco_moe_few(const cco_few_desc *d, const void *x, const int32_t *idx, const float *w,
                int32_t T, void *out, void *workspace, uint64_t workspace_bytes, void *stream) {
  if (!few_ok(d, T)) return CCO_ERR_INVALID_ARG;
  const uintptr_t ws = d->wdtype == CCO_I8 ? 1 : 2;
  if (!aligned(x, 2) || !aligned(out, 2) || !aligned(idx, 4) || !aligned(w, 4) ||
      !aligned(d->w13, ws) || !aligned(d->w2, ws) || !aligned(d->s13, 4) || !aligned(d->s2, 4) ||
      !aligned(workspace, 16))
    return CCO_ERR_INVALID_ARG;
  if ((d->wdtype == CCO_I8) != (d->s13 != nullptr) || (d->wdtype == CCO_I8) != (d->s2 != nullptr))
    return CCO_ERR_INVALID_ARG;
  if (T > cco::kFewMaxTokens) return CCO_ERR_TOO_LARGE;
  if (T == 0) return CCO_OK;
  if (!x || !idx || !w || !out || !d->w13 || !d->w2 || !workspace ||
      workspace_bytes < cco_moe_few_workspace(d, T))
    return CCO_ERR_INVALID_ARG;
  cco::FewArgs a{};
  a.T = T;
  a.K = d->topk;
  a.E = d->num_experts;
  a.H = d->hidden;
  a.I = d->inter;
  const FewSpace space = few_space(d, T);
  a.Ipad = space.pitch;
  a.parts = space.parts;
  a.partial = (float *)((char *)workspace + space.partial);
  a.idx = idx;
  a.w = w;
  a.x = (const char *)x;
  a.w13 = (const char *)d->w13;
  a.w2 = (const char *)d->w2;
  a.s13 = d->s13;
  a.s2 = d->s2;
  a.h = (uint16_t *)workspace;
  a.out = out;
  return status(
      cco::launch_moe_few(d->dtype == CCO_F16, d->wdtype == CCO_I8, a, (hipStream_t)stream));
}

}  // extern "C"
