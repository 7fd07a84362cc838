// Host-side checks of the MXFP4 and router-balance entry points
// (include/qmoe.h) built with AddressSanitizer and UndefinedBehaviorSanitizer
// on their boundary code: argument validation at the ends of the integer
// ranges and the workspace sizing.  No call reaches the device.
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

int main() {
  void* p = reinterpret_cast<void*>(uintptr_t(0x100000));   // aligned, never dereferenced
  uint8_t* u = static_cast<uint8_t*>(p);
  int32_t* i = static_cast<int32_t*>(p);
  float* f = static_cast<float*>(p);
  for (int64_t rows : {INT64_MIN, (int64_t)-1, (int64_t)INT32_MAX + 1, INT64_MAX})
    for (int64_t cols : {INT64_MIN, (int64_t)0, (int64_t)1, (int64_t)(1 << 24) + 1, INT64_MAX})
      for (int64_t ld : {INT64_MIN, (int64_t)0, INT64_MAX}) {
        const bool bad = rows < 0 || cols < 1 || ld < cols;
        EXPECT(moe_mxfp4_quantize(p, 1, rows, cols, ld, u, u, nullptr), bad ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
        EXPECT(moe_mxfp4_dequantize(u, u, rows, cols, p, 1, ld, nullptr), bad ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
      }
  EXPECT(moe_mxfp4_quantize(p, 0, 4, 64, INT64_MAX, u, u, nullptr), MOE_ERR_UNSUPPORTED);
  for (int32_t d : {INT_MIN, -1, 3, INT_MAX}) EXPECT(moe_mxfp4_quantize(p, d, 4, 64, 64, u, u, nullptr), MOE_ERR_INVALID_ARG);

  for (int32_t rows : {INT_MIN, -1, 0, 4, INT_MAX})
    for (int32_t n : {INT_MIN, 0, 32, 65536, INT_MAX})
      for (int32_t k : {INT_MIN, 0, 32, 65536, INT_MAX - 31})
        for (int32_t e : {INT_MIN, 0, 1, 256, INT_MAX})
          for (int64_t ld : {INT64_MIN, (int64_t)0, (int64_t)65536, INT64_MAX - 7}) {
            moe_matmul_config c{rows, n, k, e, rows, MOE_DT_BF16, MOE_DT_F32, ld, ld};
            // no valid call here: rows beyond the limit, or a null output
            const moe_status a = moe_mxfp4_matmul(&c, p, nullptr, u, u, i, nullptr, nullptr, nullptr);
            const moe_status b = moe_mxfp4_matmul_dx(&c, p, u, u, i, nullptr, nullptr);
            if (rows != 0 && (a == MOE_OK || b == MOE_OK)) ++failures;
            if (a == MOE_ERR_HIP || b == MOE_ERR_HIP) ++failures;
          }
  moe_matmul_config mx{4, 64, 96, 2, 4, MOE_DT_MXFP4, MOE_DT_BF16, 96, 64};
  EXPECT(moe_mxfp4_matmul(&mx, p, nullptr, u, u, i, nullptr, p, nullptr), MOE_ERR_INVALID_ARG);
  mx.a_rows = INT_MAX;
  EXPECT(moe_mxfp4_matmul(&mx, p, u, u, u, i, i, p, nullptr), MOE_ERR_UNSUPPORTED);

  size_t bytes = 0;
  for (int32_t t : {0, 1, 31, 128, 129, 4096, MOE_MAX_TOKENS})
    for (int32_t e : {1, 7, 32, 33, 256})
      for (int32_t s : {1, 2, 300, 65536}) {
        moe_balance_config c{t, e, 1, s, MOE_SCORE_SIGMOID, MOE_DT_F32, 0.5f};
        EXPECT(moe_balance_workspace_size(&c, &bytes), MOE_OK);
        if (bytes == 0 || bytes % 256 != 0) ++failures;
        EXPECT(moe_balance_loss(&c, p, i, i, i, i, f, p, bytes - 1, nullptr), MOE_ERR_WORKSPACE_TOO_SMALL);
        EXPECT(moe_balance_loss(&c, p, i, i, i, i, nullptr, p, bytes, nullptr), MOE_ERR_INVALID_ARG);
      }
  for (float coef : {NAN, INFINITY, -INFINITY}) {
    moe_balance_config c{8, 4, 2, 1, MOE_SCORE_SOFTMAX, MOE_DT_BF16, coef};
    EXPECT(moe_balance_workspace_size(&c, &bytes), MOE_ERR_INVALID_ARG);
    EXPECT(moe_balance_loss_grad(&c, p, i, i, i, i, nullptr, p, nullptr), MOE_ERR_INVALID_ARG);
  }
  for (int32_t v : {INT_MIN, -1, INT_MAX}) {
    for (int field = 0; field < 4; ++field) {
      moe_balance_config c{8, 4, 2, 1, MOE_SCORE_SOFTMAX, MOE_DT_BF16, 1.0f};
      (field == 0 ? c.tokens : field == 1 ? c.n_experts : field == 2 ? c.top_k : c.n_seq) = v;
      EXPECT(moe_balance_workspace_size(&c, &bytes), v < 0 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED);
    }
  }
  std::printf("%d failure(s)\n", failures);
  return failures ? 1 : 0;
}
