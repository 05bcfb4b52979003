// Calls the operators' C entry points (csrc/ops_api.cpp) with good, bad and
// extreme arguments; built with AddressSanitizer and UBSan, the launchers
// are stubs that count.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "../combine_symmetric_memory_amd/csrc/ops_internal.h"

static int launches = 0;
namespace cco {
hipError_t launch_route(const RouteArgs &, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_route_grad(const RouteArgs &, hipStream_t) { ++launches; return hipSuccess; }
int group_parts(GroupOp, int32_t, int32_t rows, int32_t, int32_t k) {
  return rows > 0 && k >= 4096 ? 4 : 1;
}
hipError_t launch_group(GroupOp, bool, bool, bool, const GroupArgs &, hipStream_t) {
  ++launches;
  return hipSuccess;
}
int norm_grad_workgroups(int32_t, int32_t T) { return T < 256 ? T : 256; }
hipError_t launch_block_norm(int, const NormArgs &, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_block_norm_grad(int, const NormArgs &, hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t launch_combine_norm(const CombineView &, const NormArgs &, hipStream_t) {
  ++launches;
  return hipSuccess;
}
int moe_combine_view(::cco_moe *, int32_t, CombineView *, int *, int32_t *) {
  return CCO_ERR_INVALID_ARG;
}
int moe_timed_combine(::cco_moe *, hipStream_t, hipError_t (*fn)(void *), void *ctx) {
  return fn(ctx) == hipSuccess ? CCO_OK : CCO_ERR_HIP;
}
}  // namespace cco

#define CHECK(c)                                                  \
  do {                                                            \
    if (!(c)) {                                                   \
      std::printf("line %d: %s\n", __LINE__, #c);                 \
      std::exit(1);                                               \
    }                                                             \
  } while (0)

int main() {
  char *p = (char *)(uintptr_t)(1 << 20);
  float *f = (float *)p;
  int32_t *i = (int32_t *)p;
  const int32_t ext[] = {INT_MIN, -1, 0, 1, 2, 64, 65, 1024, 1025, INT_MAX};
  for (int32_t E : ext)
    for (int32_t K : ext)
      for (int32_t G : ext)
        for (int32_t kept : ext) {
          cco_route_desc d{E, K, 0, 0, 1.0f, G, kept};
          const int rc = cco_route(&d, p, CCO_F32, E > 0 ? E : 1, nullptr, 4, i, f, nullptr);
          const bool ok = E >= 1 && E <= 1024 && K >= 1 && K <= 32 && K <= E && G >= 1 && G <= 64 &&
                          E % G == 0 && kept >= 1 && kept <= G && K <= (int64_t)kept * (E / G);
          CHECK(rc == (ok ? CCO_OK : CCO_ERR_INVALID_ARG));
        }
  for (int32_t n : ext)
    for (int32_t k : ext)
      for (int32_t rows : ext)
        for (int32_t groups : ext) {
          cco_groups g{groups, rows, i, i};
          const int rc = cco_group_product(&g, CCO_BF16, p, k, p, n, k, p, n, nullptr, 0, nullptr);
          const bool ok = n >= 1 && n < (1 << 21) && k >= 1 && k < (1 << 21) && rows >= 0 &&
                          groups >= 1 && groups <= 1024;
          CHECK(rc == (ok ? CCO_OK : CCO_ERR_INVALID_ARG));
          (void)cco_group_product_workspace(CCO_GROUP_DW, &g, n, k);
        }
  // sizes past 32 bits
  cco_groups big{1024, INT_MAX, i, i};
  CHECK(cco_group_product_workspace(CCO_GROUP_DX, &big, 8, (1 << 21) - 8) ==
        4ull * INT_MAX * ((1u << 21) - 8) * 4);
  for (int32_t h : ext)
    for (int32_t T : ext) {
      cco_block_norm_desc d{h, CCO_BF16, CCO_F32, CCO_GATE_CHANNEL, 1.0f, 1e-6f, p, p, p};
      const uint64_t ws = cco_block_norm_grad_workspace(&d, T);
      const bool ok = h >= 1 && h <= 16384 && T >= 0;
      CHECK(ok || ws == 0);
      CHECK(cco_block_norm(&d, p, p, T, p, p, nullptr) == (ok ? CCO_OK : CCO_ERR_INVALID_ARG));
      CHECK(cco_block_norm_grad(&d, p, p, p, p, T, p, p, f, f, f, p, ws, nullptr) ==
            (ok ? CCO_OK : CCO_ERR_INVALID_ARG));
      if (ws > 0)
        CHECK(cco_block_norm_grad(&d, p, p, p, p, T, p, p, f, f, f, p, ws - 1, nullptr) ==
              CCO_ERR_INVALID_ARG);
    }
  cco_block_norm_desc nan{64, CCO_BF16, CCO_F32, CCO_GATE_NONE, 1.0f, NAN, nullptr, nullptr, p};
  CHECK(cco_block_norm(&nan, p, p, 1, p, p, nullptr) == CCO_ERR_INVALID_ARG);
  CHECK(cco_moe_combine_norm(nullptr, f, &nan, p, 1, p, p, p, nullptr) == CCO_ERR_INVALID_ARG);
  CHECK(launches > 0);
  std::printf("operators' host driver ok\n");
  return 0;
}
