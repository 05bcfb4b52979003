// Calls the C entry points of csrc/serve_api.cpp with good, bad and extreme
// arguments; built with AddressSanitizer and UBSan, the launchers are stubs
// that count.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "../combine_symmetric_memory_amd/csrc/ops_internal.h"

static int launches = 0;
namespace cco {
int group_parts(GroupOp, int32_t, int32_t rows, int32_t, int32_t k) {
  return rows > 0 && k >= 4096 ? 16 : 1;
}
hipError_t launch_group_i8(int, bool, const GroupArgs &, hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t launch_quant(int, bool, const QuantArgs &, hipStream_t) { ++launches; return hipSuccess; }
int few_parts(bool, int32_t, int32_t, int32_t, int32_t H, int32_t) { return H > 16 ? 32 : 0; }
hipError_t launch_moe_few(bool, bool, const FewArgs &, hipStream_t) {
  ++launches;
  return hipSuccess;
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
  int8_t *q = (int8_t *)p;
  const int32_t ext[] = {INT_MIN, -1, 0, 1, 2, 16, 64, 65, 1024, 1 << 17, 1 << 20, 1 << 21, INT_MAX};
  const int64_t lds[] = {INT64_MIN, -1, 0, 1, 64, (1 << 21) - 1, 1 << 21, INT64_MAX};
  for (int32_t rows : ext)
    for (int32_t cols : ext)
      for (int64_t ld : lds)
        for (int sw = 0; sw < 2; ++sw) {
          const int was = launches;
          const int rc = cco_quant_rows(p, CCO_F32, ld, rows, cols, sw, q, ld, f, 1, nullptr);
          const bool ok = rows >= 0 && cols >= 1 && ld < (1 << 21) && ld >= (1 + sw) * (int64_t)cols;
          CHECK((rc == CCO_OK) == ok);
          CHECK(launches - was == (ok && rows > 0));
        }
  for (int32_t n : ext)
    for (int32_t k : ext)
      for (int32_t rows : ext) {
        cco_groups g{1, rows, i, i};
        const uint64_t ws = cco_group_product_i8_workspace(&g, n, k);
        const bool ok = rows >= 0 && n >= 1 && n < (1 << 21) && k >= 1 && k < (1 << 17);
        if (!ok) CHECK(ws == 0);
        const int was = launches;
        const int rc = cco_group_product_i8(&g, q, k, f, 1, q, f, n, k, p, CCO_F32, n,
                                            ws ? p : nullptr, ws, nullptr);
        CHECK((rc == CCO_OK) == ok);
        CHECK(launches - was == (ok && rows > 0));
      }
  for (int32_t H : ext)
    for (int32_t I : ext)
      for (int32_t K : ext)
        for (int32_t T : ext) {
          cco_few_desc d{H, I, 8, K, CCO_BF16, CCO_I8, p, p, f, f};
          const uint64_t ws = cco_moe_few_workspace(&d, T);
          const int rc = cco_moe_few(&d, p, i, f, T, p, p, ws, nullptr);
          const bool ok = H >= 1 && H <= (1 << 20) && I >= 1 && I <= (1 << 19) && K >= 1 &&
                          K <= 32 && T >= 0;
          CHECK(rc == (!ok ? CCO_ERR_INVALID_ARG : T > 64 ? CCO_ERR_TOO_LARGE : CCO_OK));
          CHECK((ws > 0) == (ok && T > 0 && T <= 64));
        }
  std::printf("driver ok\n");
  return 0;
}
