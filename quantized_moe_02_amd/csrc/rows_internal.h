// Internal interfaces of the row operators (norm, dispatch and collect,
// SwiGLU), between their C-ABI layer (rows_api.cpp) and the kernel launchers.
#pragma once

#include "operators_internal.h"

namespace qmoe {

constexpr int kRowMaxCols = 65536;
constexpr int kRowMaxRows = 16 * MOE_MAX_TOKENS;

// Bytes of a value of MOE_DT_F32 or MOE_DT_BF16.
inline int element(int dtype) { return dtype == MOE_DT_F32 ? 4 : 2; }

// A matrix in device memory; ld in elements.
struct RowMat {
  void* p;
  int64_t ld;
  int dtype;
};

struct NormArgs {
  RowMat x, res, h, y;     // res.p, h.p, y.p nullable
  const void* w;
  int w_dtype;
  void* q;                 // nullable: E4M3 codes or MXFP4 codes
  void* q_scale;
  int q_dtype;
  int rows, cols;
  float eps;
  // set by the launcher: row of a launch's first workgroup; whether results go past
  // the caches
  int first;
  bool past_cache;
};
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  RowMat h, dy, dh, dx;    // dh.p nullable
  const void* w;
  int w_dtype;
  float* dw;               // nullable
  void* part;              // [workgroups][cols]: the workgroups' sums for dw (norm_grad_part_bytes)
  int rows, cols;
  float eps;
  bool past_cache;         // as above
};
// Columns up to which the gradient holds a row in registers; past it parts may be float64.
constexpr int kNormGradCols = 16384;
// Bytes of `part` that are enough for the gradient of no more rows and columns.
size_t norm_grad_part_bytes(int rows, int cols);
hipError_t launch_rmsnorm_grad(const NormGradArgs& a, hipStream_t s);

struct DispatchArgs {
  RowMat x, rows;
  const uint8_t* x_scale;  // E4M3, MXFP4: scale_bytes of them a row
  uint8_t* row_scale;
  int scale_bytes;
  const int32_t* inv;
  int T, K, slots, cols;
};
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s);

struct CollectArgs {
  RowMat rows, add, y;     // add.p nullable
  const int32_t* inv;
  const float* w;          // nullable
  int T, K, slots, cols;
};
hipError_t launch_collect(const CollectArgs& a, hipStream_t s);

struct CollectGradArgs {
  RowMat dy, rows, drows;  // rows.p, drows.p nullable
  const int32_t* inv;
  const float* w;          // nullable
  float* dw;               // nullable
  int T, K, slots, cols;
};
hipError_t launch_collect_grad(const CollectGradArgs& a, hipStream_t s);

struct SwigluArgs {
  RowMat gu, out;          // out: of the gradient, dh
  RowMat dgu;              // of the gradient
  void* out_scale;
  const int32_t* end;      // nullable: the row behind the last that counts
  int rows, cols;
  int first;               // as above
};
hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s);
hipError_t launch_swiglu_grad(const SwigluArgs& a, hipStream_t s);

// How the rows of a matrix lie over workgroups where each lane takes one chunk of
// a row: rows of over 32 chunks take `parts` workgroups of `threads` lanes, shorter
// ones 2^bits lanes (bits = -1 for the former).
struct RowMap {
  int parts, threads, bits;
  int first;                // row of the launch's first workgroup
  bool in_order;            // block_number
};

}  // namespace qmoe
