// Host-side checks of the row operators' entry points (include/qmoe.h) built
// with AddressSanitizer and UndefinedBehaviorSanitizer on their boundary code:
// argument validation at the ends of the integer ranges.  No call reaches the
// device.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "qmoe.h"

static int failures = 0;
#define EXPECT(call, want)                                                             \
  do {                                                                                 \
    const moe_status got_ = (call);                                                    \
    if (got_ != (want)) {                                                              \
      std::fprintf(stderr, "line %d: %s -> %d, expected %d\n", __LINE__, #call, (int)got_, (int)(want)); \
      ++failures;                                                                      \
    }                                                                                  \
  } while (0)
// an error of the arguments, not of HIP
#define REFUSED(call)                                                                  \
  do {                                                                                 \
    const moe_status got_ = (call);                                                    \
    if (got_ != MOE_ERR_INVALID_ARG && got_ != MOE_ERR_UNSUPPORTED) {                  \
      std::fprintf(stderr, "line %d: %s -> %d\n", __LINE__, #call, (int)got_);         \
      ++failures;                                                                      \
    }                                                                                  \
  } while (0)

int main() {
  void* p = reinterpret_cast<void*>(uintptr_t(0x100000));   // aligned, never dereferenced
  uint8_t* u = static_cast<uint8_t*>(p);
  int32_t* i = static_cast<int32_t*>(p);
  float* f = static_cast<float*>(p);
  const int64_t lds[] = {INT64_MIN, -1, 0, INT64_MAX};

  for (int32_t rows : {INT_MIN, -1, 4, 16 * MOE_MAX_TOKENS, INT_MAX})
    for (int32_t cols : {INT_MIN, 0, 1, 65536, 65537, INT_MAX})
      for (int64_t ld : lds) {
        moe_rmsnorm_config n{rows, cols, 0, 1, 0, 1, MOE_DT_E4M3, 1e-6f, ld, ld, ld, ld};
        REFUSED(moe_rmsnorm(&n, p, p, p, p, p, u, p, nullptr));
        moe_rmsnorm_grad_config g{rows, cols, 0, 0, 1, 1, 1e-6f, ld, ld, ld, ld};
        REFUSED(moe_rmsnorm_grad(&g, p, p, p, p, p, f, p, SIZE_MAX, nullptr));
        moe_swiglu_config s{rows, cols, 3, 1, 1, ld, ld};
        REFUSED(moe_swiglu(&s, p, i, p, nullptr, nullptr));
        REFUSED(moe_swiglu_grad(&s, p, p, i, p, nullptr));
        moe_rows_config r{rows, cols, 2, rows, 1, 1, 1, ld, ld, ld};
        REFUSED(moe_dispatch(&r, p, nullptr, i, p, nullptr, nullptr));
        REFUSED(moe_collect(&r, p, i, f, p, p, nullptr));
        REFUSED(moe_collect_grad(&r, p, p, i, f, p, f, nullptr));
      }
  for (int32_t d : {INT_MIN, -1, 2, 5, INT_MAX}) {
    moe_rmsnorm_config n{4, 64, d, 0, 0, 0, 4, 1e-6f, 64, 64, 64, 64};
    EXPECT(moe_rmsnorm(&n, p, p, p, p, p, u, p, nullptr), MOE_ERR_INVALID_ARG);
    n.x_dtype = 0, n.q_dtype = d == 2 ? 0 : d;
    EXPECT(moe_rmsnorm(&n, p, p, p, p, p, u, p, nullptr), MOE_ERR_INVALID_ARG);
    moe_rows_config r{4, 64, 2, 8, d, 1, 1, 64, 64, 64};
    EXPECT(moe_dispatch(&r, p, p, i, p, p, nullptr), MOE_ERR_INVALID_ARG);
    moe_swiglu_config s{4, 64, 3, 1, d, 128, 64};
    EXPECT(moe_swiglu(&s, p, i, p, nullptr, nullptr), MOE_ERR_INVALID_ARG);
  }
  for (float eps : {0.0f, -0.0f, -1e-6f, NAN, INFINITY, -INFINITY}) {
    moe_rmsnorm_config n{4, 64, 0, 0, 0, 0, 4, eps, 64, 64, 64, 64};
    EXPECT(moe_rmsnorm(&n, p, p, p, p, p, u, p, nullptr), MOE_ERR_INVALID_ARG);
    moe_rmsnorm_grad_config g{4, 64, 0, 0, 0, 0, eps, 64, 64, 64, 64};
    EXPECT(moe_rmsnorm_grad(&g, p, p, p, p, p, f, p, SIZE_MAX, nullptr), MOE_ERR_INVALID_ARG);
  }
  for (int32_t v : {INT_MIN, -1, INT_MAX})
    for (int field = 0; field < 3; ++field) {
      moe_rows_config r{4, 64, 2, 8, 1, 1, 1, 64, 64, 64};
      (field == 0 ? r.tokens : field == 1 ? r.top_k : r.slots) = v;
      EXPECT(moe_collect(&r, p, i, f, p, p, nullptr), v < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
    }
  for (int32_t e : {INT_MIN, -1, 0}) {
    moe_swiglu_config s{4, 64, e, 1, 1, 128, 64};
    EXPECT(moe_swiglu(&s, p, i, p, nullptr, nullptr), MOE_ERR_INVALID_ARG);
  }
  size_t bytes = 0;
  for (int32_t rows : {0, 1, 512, 16 * MOE_MAX_TOKENS})
    for (int32_t cols : {1, 6144, 65536}) {
      EXPECT(moe_rmsnorm_workspace_size(rows, cols, &bytes), MOE_OK);
      if (bytes == 0 || bytes % 256 != 0 || bytes < (size_t)cols * 4) ++failures;
      moe_rmsnorm_grad_config g{rows, cols, 0, 0, 0, 0, 1e-6f, 65536, 65536, 65536, 65536};
      EXPECT(moe_rmsnorm_grad(&g, p, p, p, p, p, f, p, bytes - 1, nullptr), MOE_ERR_WORKSPACE_TOO_SMALL);
    }
  for (int32_t v : {INT_MIN, -1, INT_MAX}) {
    EXPECT(moe_rmsnorm_workspace_size(v, 64, &bytes), v < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
    EXPECT(moe_rmsnorm_workspace_size(64, v, &bytes), v < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
  }
  std::printf("%d failure(s)\n", failures);
  return failures ? 1 : 0;
}
