// Internal interfaces of the MXFP4 and router-balance operators, between
// their C-ABI layer (operators_api.cpp) and the kernel launchers.
#pragma once

#include "qmoe_internal.h"

namespace qmoe {

constexpr int kMxBlock = 32;          // inputs per MXFP4 block
constexpr int kMatmulMaxExperts = 256;

struct MxQuantArgs {
  void* x;         // quantise: source; dequantise: destination
  uint8_t* codes;  // [rows][16 nb]
  uint8_t* scale;  // [rows][nb]
  int64_t rows, cols, ld;
  int dtype;
};
hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t s);
hipError_t launch_mx_dequantize(const MxQuantArgs& a, hipStream_t s);

struct MatmulArgs {
  const void* a;            // bf16 rows, MXFP4 codes, or (dx) bf16 dy
  const uint8_t* a_scale;   // MXFP4 rows only
  const uint8_t* w_codes;
  const uint8_t* w_scale;
  const int32_t* offsets;   // nullable: one expert
  const int32_t* index;     // nullable
  void* out;
  int R, N, K, E, a_rows;
  int64_t lda, ldo;
  bool out_bf16;
};
hipError_t launch_mx_matmul(const MatmulArgs& a, bool a_mxfp4, hipStream_t s);
hipError_t launch_mx_matmul_large(const MatmulArgs& a, hipStream_t s);
hipError_t launch_mx_matmul_mid(const MatmulArgs& a, hipStream_t s);
hipError_t launch_mx_matmul4_large(const MatmulArgs& a, hipStream_t s);
hipError_t launch_mx_matmul_dx_mid(const MatmulArgs& a, hipStream_t s);
hipError_t launch_mx_matmul_dx_large(const MatmulArgs& a, hipStream_t s);
hipError_t launch_mx_matmul_dx(const MatmulArgs& a, hipStream_t s);

struct BalanceArgs {
  const void* logits;
  const int32_t* ids;
  const int32_t* seq;       // nullable: one sequence
  int32_t* counts;
  int32_t* tokens;
  float* loss;              // forward
  const float* dloss;       // gradient, nullable
  void* dlogits;            // gradient
  int T, E, K, S;
  bool sigmoid, bf16;
  float coef;
  // workspace of the forward pass
  double* seq_loss;         // [S][slices]
  float* part_p;            // [slots][E]
  int32_t* part_c;          // [slots][E]
  int32_t* part_n;          // [slots] routed tokens
  int32_t* part_k;          // [slots] picks
};
// Token chunks of the forward pass: one partial sum per (chunk, sequence)
// pair that share a token, at slot chunk + sequence.
int balance_chunk(int T, int S);
// Chunks of any T tokens or fewer, at most: what the workspace holds.
int balance_max_chunks(int T, int S);
// Workgroups per sequence of its second launch.
int balance_slices(int E);
hipError_t launch_balance(const BalanceArgs& a, hipStream_t s);
hipError_t launch_balance_grad(const BalanceArgs& a, hipStream_t s);

}  // namespace qmoe
