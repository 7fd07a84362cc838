// C-ABI entry points of the row operators (declared in include/qmoe.h):
// argument validation and dispatch.  Every check runs before the first HIP call.
#include <cmath>
#include <cstdint>

#include "rows_internal.h"

namespace qmoe {
namespace {

constexpr size_t kAlign = 256;

bool plain_dtype(int32_t d) { return d == MOE_DT_F32 || d == MOE_DT_BF16; }
bool coded_dtype(int32_t d) { return d == MOE_DT_E4M3 || d == MOE_DT_MXFP4; }
bool element_aligned(const void* p, int32_t d) { return aligned(p, element(d)); }

// Limits of a matrix's size; columns before rows.
moe_status check_size(int32_t rows, int32_t cols) {
  if (rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  return rows > kRowMaxRows || cols > kRowMaxCols ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// A stride holds a row, and byte offsets stay in 63 bits.
moe_status check_stride(int64_t ld, int64_t cols) {
  if (ld < cols) return MOE_ERR_INVALID_ARG;
  return ld > INT64_MAX / 4 / kRowMaxRows ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// First of several results that is none of MOE_OK, the errors of arguments first.
moe_status first_of(std::initializer_list<moe_status> all) {
  moe_status worst = MOE_OK;
  for (moe_status s : all) {
    if (s == MOE_ERR_INVALID_ARG) return s;
    if (worst == MOE_OK) worst = s;
  }
  return worst;
}

moe_status invalid_unless(bool ok) { return ok ? MOE_OK : MOE_ERR_INVALID_ARG; }

moe_status check_codes(int32_t dtype, const void* codes, const void* scale) {
  return invalid_unless(codes && scale && aligned(codes, dtype == MOE_DT_MXFP4 ? 16 : 8) &&
                        (dtype == MOE_DT_MXFP4 || aligned(scale, 4)));
}

RowMat mat(const void* p, int64_t ld, int dtype) { return RowMat{const_cast<void*>(p), ld, dtype}; }

int scale_bytes(int dtype, int cols) {
  return dtype == MOE_DT_E4M3 ? 4 : dtype == MOE_DT_MXFP4 ? (cols + kMxBlock - 1) / kMxBlock : 0;
}

// Ascends in both sizes, and is not 0 for no rows.
size_t norm_workspace(int rows, int cols) {
  return (norm_grad_part_bytes(rows, cols) + kAlign - 1) / kAlign * kAlign;
}

moe_status check_rows(const moe_rows_config* c) {
  if (!c || c->tokens < 0 || c->slots < 0 || c->cols < 1 || c->top_k < 1) return MOE_ERR_INVALID_ARG;
  if (c->tokens > MOE_MAX_TOKENS || c->slots > kRowMaxRows || c->top_k > 16 || c->cols > kRowMaxCols)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_swiglu(const moe_swiglu_config* c) {
  if (!c || c->n_experts < 1 || !plain_dtype(c->gu_dtype)) return MOE_ERR_INVALID_ARG;
  return check_size(c->rows, c->cols);
}

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" {

moe_status moe_rmsnorm(const moe_rmsnorm_config* cfg, const void* x, const void* residual,
                       const void* weight, void* h, void* y, uint8_t* q, void* q_scale,
                       hipStream_t stream) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  const moe_rmsnorm_config& c = *cfg;
  if (!plain_dtype(c.x_dtype) || !plain_dtype(c.weight_dtype) || !(c.eps > 0.0f) || !std::isfinite(c.eps))
    return MOE_ERR_INVALID_ARG;
  if ((residual && !plain_dtype(c.residual_dtype)) || (y && !plain_dtype(c.y_dtype)) || (q && !coded_dtype(c.q_dtype)))
    return MOE_ERR_INVALID_ARG;
  if ((h && !residual) || (!q && q_scale)) return MOE_ERR_INVALID_ARG;
  const moe_status s =
      first_of({check_size(c.rows, c.cols), check_stride(c.ldx, c.cols), residual ? check_stride(c.ldr, c.cols) : MOE_OK,
                h ? check_stride(c.ldh, c.cols) : MOE_OK, y ? check_stride(c.ldy, c.cols) : MOE_OK});
  if (s != MOE_OK || c.rows == 0) return s;
  if (!h && !y && !q) return MOE_ERR_INVALID_ARG;
  if (!x || !weight || !element_aligned(x, c.x_dtype) || !element_aligned(weight, c.weight_dtype)) return MOE_ERR_INVALID_ARG;
  if (!element_aligned(residual, residual ? c.residual_dtype : MOE_DT_F32) ||
      !element_aligned(h, h ? c.residual_dtype : MOE_DT_F32) || !element_aligned(y, y ? c.y_dtype : MOE_DT_F32))
    return MOE_ERR_INVALID_ARG;
  if (q && check_codes(c.q_dtype, q, q_scale) != MOE_OK) return MOE_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = mat(x, c.ldx, c.x_dtype);
  a.res = mat(residual, c.ldr, c.residual_dtype);
  a.h = mat(h, c.ldh, c.residual_dtype);
  a.y = mat(y, c.ldy, c.y_dtype);
  a.w = weight;
  a.w_dtype = c.weight_dtype;
  a.q = q;
  a.q_scale = q_scale;
  a.q_dtype = c.q_dtype;
  a.rows = c.rows;
  a.cols = c.cols;
  a.eps = c.eps;
  return hip_status(launch_rmsnorm(a, stream));
}

moe_status moe_rmsnorm_workspace_size(int32_t rows, int32_t cols, size_t* bytes) {
  const moe_status s = check_size(rows, cols);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = norm_workspace(rows, cols);
  return MOE_OK;
}

moe_status moe_rmsnorm_grad(const moe_rmsnorm_grad_config* cfg, const void* dy, const void* h,
                            const void* weight, const void* dh, void* dx, float* dweight,
                            void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!cfg) return MOE_ERR_INVALID_ARG;
  const moe_rmsnorm_grad_config& c = *cfg;
  if (!plain_dtype(c.h_dtype) || !plain_dtype(c.weight_dtype) || !plain_dtype(c.dy_dtype) || !plain_dtype(c.dx_dtype))
    return MOE_ERR_INVALID_ARG;
  if (!(c.eps > 0.0f) || !std::isfinite(c.eps)) return MOE_ERR_INVALID_ARG;
  const moe_status s =
      first_of({check_size(c.rows, c.cols), check_stride(c.ldh, c.cols), check_stride(c.lddy, c.cols),
                dh ? check_stride(c.lddh, c.cols) : MOE_OK, check_stride(c.lddx, c.cols)});
  if (s != MOE_OK) return s;
  if (!aligned(dweight, 4)) return MOE_ERR_INVALID_ARG;
  if (c.rows == 0 && !dweight) return MOE_OK;
  if (c.rows > 0 && (!dy || !h || !weight || !dx || !element_aligned(dy, c.dy_dtype) || !element_aligned(h, c.h_dtype) ||
                     !element_aligned(weight, c.weight_dtype) || !element_aligned(dx, c.dx_dtype) ||
                     !element_aligned(dh, c.dx_dtype)))
    return MOE_ERR_INVALID_ARG;
  if (dweight) {
    if (!ws || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < norm_workspace(c.rows, c.cols)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  NormGradArgs a{};
  a.h = mat(h, c.ldh, c.h_dtype);
  a.dy = mat(dy, c.lddy, c.dy_dtype);
  a.dh = mat(dh, c.lddh, c.dx_dtype);
  a.dx = mat(dx, c.lddx, c.dx_dtype);
  a.w = weight;
  a.w_dtype = c.weight_dtype;
  a.dw = dweight;
  a.part = ws;
  a.rows = c.rows;
  a.cols = c.cols;
  a.eps = c.eps;
  return hip_status(launch_rmsnorm_grad(a, stream));
}

moe_status moe_dispatch(const moe_rows_config* cfg, const void* x, const void* x_scale,
                        const int32_t* inv_perm, void* rows, void* row_scale, hipStream_t stream) {
  moe_status s = check_rows(cfg);
  if (s != MOE_OK) return s;
  const moe_rows_config& c = *cfg;
  const bool coded = coded_dtype(c.token_dtype);
  if (coded ? c.row_dtype != c.token_dtype : !plain_dtype(c.token_dtype) || !plain_dtype(c.row_dtype))
    return MOE_ERR_INVALID_ARG;
  if (coded ? c.ldt != c.cols || c.ldr != c.cols : x_scale || row_scale) return MOE_ERR_INVALID_ARG;
  if ((s = first_of({check_stride(c.ldt, c.cols), check_stride(c.ldr, c.cols)})) != MOE_OK) return s;
  if (c.tokens == 0 || c.slots == 0) return MOE_OK;
  if (!x || !rows || !inv_perm || !aligned(inv_perm, 4)) return MOE_ERR_INVALID_ARG;
  if (coded) {
    if ((s = first_of({check_codes(c.token_dtype, x, x_scale), check_codes(c.row_dtype, rows, row_scale)})) != MOE_OK) return s;
  } else if (!element_aligned(x, c.token_dtype) || !element_aligned(rows, c.row_dtype)) {
    return MOE_ERR_INVALID_ARG;
  }
  DispatchArgs a{};
  a.x = mat(x, c.ldt, c.token_dtype);
  a.rows = mat(rows, c.ldr, c.row_dtype);
  a.x_scale = static_cast<const uint8_t*>(x_scale);
  a.row_scale = static_cast<uint8_t*>(row_scale);
  a.scale_bytes = scale_bytes(c.row_dtype, c.cols);
  a.inv = inv_perm;
  a.T = c.tokens;
  a.K = c.top_k;
  a.slots = c.slots;
  a.cols = c.cols;
  return hip_status(launch_dispatch(a, stream));
}

moe_status moe_collect(const moe_rows_config* cfg, const void* rows, const int32_t* inv_perm,
                       const float* weights, const void* addend, void* y, hipStream_t stream) {
  moe_status s = check_rows(cfg);
  if (s != MOE_OK) return s;
  const moe_rows_config& c = *cfg;
  if (!plain_dtype(c.token_dtype) || !plain_dtype(c.row_dtype) || (addend && !plain_dtype(c.addend_dtype)))
    return MOE_ERR_INVALID_ARG;
  s = first_of({check_stride(c.ldt, c.cols), check_stride(c.ldr, c.cols), addend ? check_stride(c.lda, c.cols) : MOE_OK});
  if (s != MOE_OK || c.tokens == 0) return s;
  if (!y || !inv_perm || !aligned(inv_perm, 4) || !aligned(weights, 4) || !element_aligned(y, c.token_dtype))
    return MOE_ERR_INVALID_ARG;
  if (c.slots > 0 && (!rows || !element_aligned(rows, c.row_dtype))) return MOE_ERR_INVALID_ARG;
  if (addend && !element_aligned(addend, c.addend_dtype)) return MOE_ERR_INVALID_ARG;
  CollectArgs a{};
  a.rows = mat(rows, c.ldr, c.row_dtype);
  a.add = mat(addend, c.lda, c.addend_dtype);
  a.y = mat(y, c.ldt, c.token_dtype);
  a.inv = inv_perm;
  a.w = weights;
  a.T = c.tokens;
  a.K = c.top_k;
  a.slots = c.slots;
  a.cols = c.cols;
  return hip_status(launch_collect(a, stream));
}

moe_status moe_collect_grad(const moe_rows_config* cfg, const void* dy, const void* rows,
                            const int32_t* inv_perm, const float* weights, void* drows,
                            float* dweights, hipStream_t stream) {
  moe_status s = check_rows(cfg);
  if (s != MOE_OK) return s;
  const moe_rows_config& c = *cfg;
  if (!plain_dtype(c.token_dtype) || !plain_dtype(c.row_dtype)) return MOE_ERR_INVALID_ARG;
  s = first_of({check_stride(c.ldt, c.cols), check_stride(c.ldr, c.cols)});
  if (s != MOE_OK || c.tokens == 0) return s;
  if (!drows && !dweights) return invalid_unless(c.slots == 0);
  if (!dy || !inv_perm || !aligned(inv_perm, 4) || !aligned(weights, 4) || !aligned(dweights, 4)) return MOE_ERR_INVALID_ARG;
  if (!element_aligned(dy, c.token_dtype) || !element_aligned(rows, c.row_dtype) || !element_aligned(drows, c.row_dtype))
    return MOE_ERR_INVALID_ARG;
  if (dweights && c.slots > 0 && !rows) return MOE_ERR_INVALID_ARG;
  CollectGradArgs a{};
  a.dy = mat(dy, c.ldt, c.token_dtype);
  a.rows = mat(rows, c.ldr, c.row_dtype);
  a.drows = mat(drows, c.ldr, c.row_dtype);
  a.inv = inv_perm;
  a.w = weights;
  a.dw = dweights;
  a.T = c.tokens;
  a.K = c.top_k;
  a.slots = c.slots;
  a.cols = c.cols;
  return hip_status(launch_collect_grad(a, stream));
}

moe_status moe_swiglu(const moe_swiglu_config* cfg, const void* gu, const int32_t* expert_offsets,
                      void* out, void* out_scale, hipStream_t stream) {
  moe_status s = check_swiglu(cfg);
  if (s == MOE_ERR_INVALID_ARG) return s;
  const moe_swiglu_config& c = *cfg;
  const bool coded = coded_dtype(c.out_dtype);
  if (!coded && !plain_dtype(c.out_dtype)) return MOE_ERR_INVALID_ARG;
  if (coded ? c.ldo != c.cols : out_scale != nullptr) return MOE_ERR_INVALID_ARG;
  s = first_of({s, check_stride(c.ldg, (int64_t)2 * c.cols), check_stride(c.ldo, c.cols)});
  if (s != MOE_OK || c.rows == 0) return s;
  if (!gu || !out || !element_aligned(gu, c.gu_dtype) || !aligned(expert_offsets, 4)) return MOE_ERR_INVALID_ARG;
  if (coded ? check_codes(c.out_dtype, out, out_scale) != MOE_OK : !element_aligned(out, c.out_dtype)) return MOE_ERR_INVALID_ARG;
  SwigluArgs a{};
  a.gu = mat(gu, c.ldg, c.gu_dtype);
  a.out = mat(out, c.ldo, c.out_dtype);
  a.out_scale = out_scale;
  a.end = expert_offsets ? expert_offsets + c.n_experts : nullptr;
  a.rows = c.rows;
  a.cols = c.cols;
  return hip_status(launch_swiglu(a, stream));
}

moe_status moe_swiglu_grad(const moe_swiglu_config* cfg, const void* gu, const void* dh,
                           const int32_t* expert_offsets, void* dgu, hipStream_t stream) {
  moe_status s = check_swiglu(cfg);
  if (s == MOE_ERR_INVALID_ARG) return s;
  const moe_swiglu_config& c = *cfg;
  if (!plain_dtype(c.out_dtype)) return MOE_ERR_INVALID_ARG;
  s = first_of({s, check_stride(c.ldg, (int64_t)2 * c.cols), check_stride(c.ldo, c.cols)});
  if (s != MOE_OK || c.rows == 0) return s;
  if (!gu || !dh || !dgu || !element_aligned(gu, c.gu_dtype) || !element_aligned(dgu, c.gu_dtype) ||
      !element_aligned(dh, c.out_dtype) || !aligned(expert_offsets, 4))
    return MOE_ERR_INVALID_ARG;
  SwigluArgs a{};
  a.gu = mat(gu, c.ldg, c.gu_dtype);
  a.dgu = mat(dgu, c.ldg, c.gu_dtype);
  a.out = mat(dh, c.ldo, c.out_dtype);
  a.end = expert_offsets ? expert_offsets + c.n_experts : nullptr;
  a.rows = c.rows;
  a.cols = c.cols;
  return hip_status(launch_swiglu_grad(a, stream));
}

}  // extern "C"
