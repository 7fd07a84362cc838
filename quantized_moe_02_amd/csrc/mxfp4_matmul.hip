// Grouped products over MXFP4 expert weights for few rows, and the choice of
// the kernel.
//
// A block of 32 inputs is one lane's share: 16 bytes of codes and one scale
// byte.  Rows in bf16: the codes become bf16 with their scale (exact: E2M1
// times a power of two) in four 16x16x32 steps.  Rows in MXFP4: the codes go
// into one 16x16x128 scaled step as they are.
#include <algorithm>

#include "mxfp4_tile.h"

namespace qmoe {
namespace {

// At most this many units for R rows of E experts.
long max_units(const MatmulArgs& g, int BM) {
  return (long)g.R / BM + (g.offsets ? (long)min(g.E, g.R) : 1);
}

// One wave: 16 outputs x 16 rows.
template <bool MX>
__global__ void __launch_bounds__(256) mx_matmul_kernel(MatmulArgs g, int nt) {
  const int ub = blockIdx.x / nt, tile = blockIdx.x - ub * nt;
  const RowUnit u = find_unit(g.offsets, g.E, g.R, 16, ub);
  if (u.M <= 0) return;
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4, wv = threadIdx.x >> 6;
  const int n0 = tile * 64 + wv * 16;
  if (n0 >= g.N) return;
  const int nb = g.K / kMxBlock;
  const int64_t wrow = (int64_t)u.e * g.N + n0 + lr;
  const bool wok = n0 + lr < g.N;
  const int64_t arow = lr < u.M ? source_row(g, u.r0 + lr) : -1;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int b0 = 0; b0 < nb; b0 += 4) {
    const int b = b0 + lq;
    uint4 w = make_uint4(0, 0, 0, 0);
    uint32_t sb = 0;
    if (wok && b < nb) {
      w = reinterpret_cast<const uint4*>(g.w_codes)[wrow * nb + b];
      sb = g.w_scale[wrow * nb + b];
    }
    if constexpr (MX) {
      uint4 x = make_uint4(0, 0, 0, 0);
      uint32_t xb = 0;
      if (arow >= 0 && b < nb) {
        x = static_cast<const uint4*>(g.a)[arow * nb + b];
        xb = g.a_scale[arow * nb + b];
      }
      const i32x8 A = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
      const i32x8 B = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc, 4, 4, 0, (int)sb, 0, (int)xb);
    } else {
      const float s = __uint_as_float(sb << 23);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (arow >= 0 && b < nb)
          x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g.a) + arow * g.lda + b * kMxBlock + 8 * i);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_of(ww[i], s), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
      }
    }
  }
  if (lr >= u.M) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + 4 * lq + i < g.N) store_out(g, u.r0 + lr, n0 + 4 * lq + i, acc[i]);
}

// One thread: two neighbouring inputs of one row.
__global__ void __launch_bounds__(256) mx_matmul_dx_kernel(MatmulArgs g, int nt) {
  const int ub = blockIdx.x / nt, tile = blockIdx.x - ub * nt;
  const RowUnit u = find_unit(g.offsets, g.E, g.R, 1, ub);
  const int k = (tile * 256 + threadIdx.x) * 2;
  if (u.M <= 0 || k >= g.K) return;
  const int nb = g.K / kMxBlock;
  const uint16_t* dy = static_cast<const uint16_t*>(g.a) + u.r0 * g.lda;
  float a0 = 0.f, a1 = 0.f;
  for (int j = 0; j < g.N; ++j) {
    const int64_t wrow = (int64_t)u.e * g.N + j;
    const float d = __uint_as_float((uint32_t)dy[j] << 16);
    const uint32_t w = g.w_codes[wrow * (g.K / 2) + k / 2];
    const float s = __uint_as_float((uint32_t)g.w_scale[wrow * nb + k / kMxBlock] << 23);
    const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
    a0 = fmaf(d, v[0], a0);
    a1 = fmaf(d, v[1], a1);
  }
  store_out(g, u.r0, k, a0);
  store_out(g, u.r0, k + 1, a1);
}

}  // namespace

hipError_t launch_mx_matmul(const MatmulArgs& g, bool a_mxfp4, hipStream_t s) {
  // few rows per expert, or too few outputs to give a quarter of the CUs an
  // item: the small kernel; sources past 32-bit offsets too
  const int64_t ldb = a_mxfp4 ? g.K / 2 : g.lda * 2;
  const int64_t span = (g.index ? (int64_t)g.a_rows : kFatRows) * ldb;
  if (g.R >= 8 * (int64_t)g.E && (int64_t)g.R * g.N >= 64 * 256 * 256 && span < (int64_t)kOutside)
    return a_mxfp4 ? launch_mx_matmul4_large(g, s) : launch_mx_matmul_large(g, s);
  const int nt = (g.N + 63) / 64;
  const dim3 grid((unsigned)(max_units(g, 16) * nt));
  if (a_mxfp4) hipLaunchKernelGGL(mx_matmul_kernel<true>, grid, dim3(256), 0, s, g, nt);
  else hipLaunchKernelGGL(mx_matmul_kernel<false>, grid, dim3(256), 0, s, g, nt);
  return hipGetLastError();
}

hipError_t launch_mx_matmul_dx(const MatmulArgs& g, hipStream_t s) {
  if (g.R >= 8 * (int64_t)g.E && (int64_t)g.R * g.K >= 64 * 256 * 256 && kFatRows * g.lda * 2 < (int64_t)kOutside)
    return launch_mx_matmul_dx_large(g, s);
  const int nt = (g.K + 511) / 512;
  hipLaunchKernelGGL(mx_matmul_dx_kernel, dim3((unsigned)(max_units(g, 1) * nt)), dim3(256), 0, s, g, nt);
  return hipGetLastError();
}

}  // namespace qmoe
