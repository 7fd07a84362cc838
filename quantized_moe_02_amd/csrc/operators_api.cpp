// C-ABI entry points of the MXFP4 and router-balance operators (declared in
// include/qmoe.h): argument validation, workspace layout and dispatch.  Every
// check runs before the first HIP call.
#include <cmath>
#include <cstdint>

#include "operators_internal.h"

namespace qmoe {
namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = (int64_t)16 * MOE_MAX_TOKENS;

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool float_dtype(int32_t d) { return d == MOE_DT_F32 || d == MOE_DT_BF16 || d == MOE_DT_F16; }

moe_status check_mx_rows(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                         const uint8_t* codes, const uint8_t* scale) {
  if (!float_dtype(dtype) || rows < 0 || cols < 1 || ld < cols) return MOE_ERR_INVALID_ARG;
  if (cols > (1 << 24) || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  if (ld > INT64_MAX / 4 / (rows > 0 ? rows : 1)) return MOE_ERR_UNSUPPORTED;   // byte offsets pass int64
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scale) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, dtype == MOE_DT_F32 ? 4 : 2) || !aligned(codes, 16)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Checks shared by the product and its gradient.  in_cols / out_cols: columns
// of the input and the output matrix.
moe_status check_matmul(const moe_matmul_config* c, int in_cols, int out_cols, const void* a,
                        const uint8_t* w_codes, const uint8_t* w_scale, const int32_t* offsets,
                        const void* out) {
  if (c->out_dtype != MOE_DT_F32 && c->out_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
  if (c->lda < in_cols || c->ldo < out_cols) return MOE_ERR_INVALID_ARG;
  if (c->a_dtype == MOE_DT_BF16 && c->lda % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (c->a_dtype == MOE_DT_MXFP4 && c->lda != in_cols) return MOE_ERR_INVALID_ARG;
  if (c->n_experts > kMatmulMaxExperts || c->n > 65536 || c->k > 65536) return MOE_ERR_UNSUPPORTED;
  if (c->rows > kMaxRows || c->a_rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (c->lda > INT64_MAX / 4 / kMaxRows || c->ldo > INT64_MAX / 4 / kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (c->rows == 0) return MOE_OK;
  if (!a || !w_codes || !w_scale || !out) return MOE_ERR_INVALID_ARG;
  if (!offsets && c->n_experts != 1) return MOE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(w_codes, 16) || !aligned(w_scale, 4) || !aligned(out, 16))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_matmul_geom(const moe_matmul_config* c) {
  if (!c || c->rows < 0 || c->a_rows < 0 || c->n < 1 || c->k < 1 || c->n_experts < 1)
    return MOE_ERR_INVALID_ARG;
  return c->k % kMxBlock == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
}

MatmulArgs matmul_args(const moe_matmul_config& c, const void* a, const uint8_t* a_scale,
                       const uint8_t* w_codes, const uint8_t* w_scale, const int32_t* offsets,
                       const int32_t* index, void* out) {
  return MatmulArgs{a, a_scale, w_codes, w_scale, offsets, index, out, c.rows, c.n, c.k,
                    c.n_experts, c.a_rows, c.lda, c.ldo, c.out_dtype == MOE_DT_BF16};
}

moe_status check_balance(const moe_balance_config* c) {
  if (!c || c->tokens < 0 || c->n_experts < 1 || c->top_k < 1 || c->n_seq < 1) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SIGMOID && c->score != MOE_SCORE_SOFTMAX) return MOE_ERR_INVALID_ARG;
  if (c->logits_dtype != MOE_DT_F32 && c->logits_dtype != MOE_DT_BF16) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->coef)) return MOE_ERR_INVALID_ARG;
  if (c->tokens > MOE_MAX_TOKENS || c->n_experts > 256 || c->top_k > 16 || c->n_seq > 65536)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

BalanceArgs balance_args(const moe_balance_config& c, const void* logits, const int32_t* ids,
                         const int32_t* seq) {
  BalanceArgs a{};
  a.logits = logits;
  a.ids = ids;
  a.seq = seq;
  a.T = c.tokens;
  a.E = c.n_experts;
  a.K = c.top_k;
  a.S = c.n_seq;
  a.sigmoid = c.score == MOE_SCORE_SIGMOID;
  a.bf16 = c.logits_dtype == MOE_DT_BF16;
  a.coef = c.coef;
  return a;
}

// Lays the workspace out from `base` (nullptr: only sizes it).
size_t carve_balance(const moe_balance_config& c, void* base, BalanceArgs* a) {
  const size_t slots = (size_t)balance_max_chunks(c.tokens, c.n_seq) + (size_t)c.n_seq;
  const size_t E = (size_t)c.n_experts;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = round_up(off + bytes, kAlign);
    return o;
  };
  const size_t parts = (size_t)c.n_seq * balance_slices(c.n_experts);
  const size_t o_loss = take(parts * sizeof(double));
  const size_t o_p = take(slots * E * sizeof(float));
  const size_t o_c = take(slots * E * sizeof(int32_t));
  const size_t o_n = take(slots * sizeof(int32_t));
  const size_t o_k = take(slots * sizeof(int32_t));
  if (a) {
    char* b = static_cast<char*>(base);
    a->seq_loss = reinterpret_cast<double*>(b + o_loss);
    a->part_p = reinterpret_cast<float*>(b + o_p);
    a->part_c = reinterpret_cast<int32_t*>(b + o_c);
    a->part_n = reinterpret_cast<int32_t*>(b + o_n);
    a->part_k = reinterpret_cast<int32_t*>(b + o_k);
  }
  return off;
}

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" {

moe_status moe_mxfp4_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols,
                              int64_t ld, uint8_t* codes, uint8_t* scale, hipStream_t stream) {
  const moe_status s = check_mx_rows(src, dtype, rows, cols, ld, codes, scale);
  if (s != MOE_OK || rows == 0) return s;
  return hip_status(launch_mx_quantize(
      MxQuantArgs{const_cast<void*>(src), codes, scale, rows, cols, ld, dtype}, stream));
}

moe_status moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scale, int64_t rows,
                                int64_t cols, void* dst, int32_t dtype, int64_t ld,
                                hipStream_t stream) {
  const moe_status s = check_mx_rows(dst, dtype, rows, cols, ld, codes, scale);
  if (s != MOE_OK || rows == 0) return s;
  return hip_status(launch_mx_dequantize(
      MxQuantArgs{dst, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scale), rows, cols, ld, dtype},
      stream));
}

moe_status moe_mxfp4_matmul(const moe_matmul_config* cfg, const void* a, const uint8_t* a_scale,
                            const uint8_t* w_codes, const uint8_t* w_scale,
                            const int32_t* expert_offsets, const int32_t* row_index, void* out,
                            hipStream_t stream) {
  moe_status s;
  if ((s = check_matmul_geom(cfg)) != MOE_OK) return s;
  if (cfg->a_dtype != MOE_DT_BF16 && cfg->a_dtype != MOE_DT_MXFP4) return MOE_ERR_INVALID_ARG;
  if ((s = check_matmul(cfg, cfg->k, cfg->n, a, w_codes, w_scale, expert_offsets, out)) != MOE_OK)
    return s;
  const bool mx = cfg->a_dtype == MOE_DT_MXFP4;
  if (!row_index && cfg->a_rows != cfg->rows) return MOE_ERR_INVALID_ARG;
  if (cfg->rows == 0) return MOE_OK;
  if (mx ? !a_scale || !aligned(a_scale, 4) : a_scale != nullptr) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_mx_matmul(
      matmul_args(*cfg, a, a_scale, w_codes, w_scale, expert_offsets, row_index, out), mx, stream));
}

moe_status moe_mxfp4_matmul_dx(const moe_matmul_config* cfg, const void* dy,
                               const uint8_t* w_codes, const uint8_t* w_scale,
                               const int32_t* expert_offsets, void* dx, hipStream_t stream) {
  moe_status s;
  if ((s = check_matmul_geom(cfg)) != MOE_OK) return s;
  if (cfg->a_dtype != MOE_DT_BF16 || cfg->a_rows != cfg->rows || cfg->n % kMxBlock != 0)
    return MOE_ERR_INVALID_ARG;
  if ((s = check_matmul(cfg, cfg->n, cfg->k, dy, w_codes, w_scale, expert_offsets, dx)) != MOE_OK)
    return s;
  if (cfg->rows == 0) return MOE_OK;
  return hip_status(launch_mx_matmul_dx(
      matmul_args(*cfg, dy, nullptr, w_codes, w_scale, expert_offsets, nullptr, dx), stream));
}

moe_status moe_balance_workspace_size(const moe_balance_config* cfg, size_t* bytes) {
  const moe_status s = check_balance(cfg);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = carve_balance(*cfg, nullptr, nullptr);
  return MOE_OK;
}

moe_status moe_balance_loss(const moe_balance_config* cfg, const void* logits,
                            const int32_t* topk_ids, const int32_t* seq_offsets, int32_t* counts,
                            int32_t* tokens, float* loss, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
  const moe_status s = check_balance(cfg);
  if (s != MOE_OK) return s;
  if (cfg->tokens > 0 && (!logits || !topk_ids || !aligned(logits, 16))) return MOE_ERR_INVALID_ARG;
  if (!counts || !tokens || !loss || !ws || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
  if (!seq_offsets && cfg->n_seq != 1) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < carve_balance(*cfg, nullptr, nullptr)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  BalanceArgs a = balance_args(*cfg, logits, topk_ids, seq_offsets);
  a.counts = counts;
  a.tokens = tokens;
  a.loss = loss;
  carve_balance(*cfg, ws, &a);
  return hip_status(launch_balance(a, stream));
}

moe_status moe_balance_loss_grad(const moe_balance_config* cfg, const void* logits,
                                 const int32_t* topk_ids, const int32_t* seq_offsets,
                                 const int32_t* counts, const int32_t* tokens, const float* dloss,
                                 void* dlogits, hipStream_t stream) {
  const moe_status s = check_balance(cfg);
  if (s != MOE_OK) return s;
  if (!seq_offsets && cfg->n_seq != 1) return MOE_ERR_INVALID_ARG;
  if (cfg->tokens == 0) return MOE_OK;
  if (!logits || !topk_ids || !counts || !tokens || !dlogits) return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(dlogits, 16)) return MOE_ERR_INVALID_ARG;
  BalanceArgs a = balance_args(*cfg, logits, topk_ids, seq_offsets);
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.dloss = dloss;
  a.dlogits = dlogits;
  return hip_status(launch_balance_grad(a, stream));
}

}  // extern "C"
