// Grouped products over MXFP4 expert weights, and their gradient with respect
// to the rows.
//
// MFMA operands (a wave of 64, lane = 16 lq + lr): of a 16 x 16 tile, lane
// (lr, lq) feeds row lr of A and column lr of B with the same inputs, any
// assignment of inputs to (step, lq, element) being valid as long as A and B
// share it, and holds rows 4 lq .. 4 lq + 3 of column lr of the result.  Here
// A is the weights (rows: output features) and B the activations (columns:
// rows of `a`), so a lane ends up with four consecutive outputs of one row.
//
// A block of 32 inputs is one lane's share: 16 bytes of codes and one scale
// byte.  Rows in bf16: the codes become bf16 with their scale (exact: E2M1
// times a power of two) in four 16x16x32 steps.  Rows in MXFP4: the codes go
// into one 16x16x128 scaled step as they are.
#include "operators_internal.h"
#include "qmoe_device.h"

namespace qmoe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct RowUnit {
  int e, r0, M;   // expert, first row, rows (0: no such unit)
};

// Unit `b` of the rows cut into runs of at most BM rows of one expert: thread
// i counts the units of expert i, a scan over the 256 threads finds the expert
// that holds unit b.  Called by all 256 threads; offsets are clamped to
// ascending values in [0, R], so no row outside the output is ever touched.
__device__ __forceinline__ RowUnit find_unit(const int32_t* offsets, int E, int R, int BM, int b) {
  if (!offsets) {
    const int r0 = b * BM;
    return RowUnit{0, r0, max(0, min(BM, R - r0))};
  }
  __shared__ int wave_sum[4], hit[3];
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  int lo = 0, cnt = 0;
  if (t < E) {
    lo = min(max(offsets[t], 0), R);
    cnt = min(max(offsets[t + 1], lo), R) - lo;
  }
  const int u = (cnt + BM - 1) / BM;
  int inc = u;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(inc, d, 64);
    if (lane >= d) inc += v;
  }
  if (lane == 63) wave_sum[wv] = inc;
  if (t == 0) hit[2] = 0;
  __syncthreads();
  for (int i = 0; i < wv; ++i) inc += wave_sum[i];
  if (b >= inc - u && b < inc) {
    const int k = b - (inc - u);
    hit[0] = t;
    hit[1] = lo + k * BM;
    hit[2] = min(BM, cnt - k * BM);
  }
  __syncthreads();
  return RowUnit{__builtin_amdgcn_readfirstlane(hit[0]), __builtin_amdgcn_readfirstlane(hit[1]),
                 __builtin_amdgcn_readfirstlane(hit[2])};
}

// At most this many units for R rows of E experts.
long max_units(const MatmulArgs& g, int BM) {
  return (long)g.R / BM + (g.offsets ? (long)min(g.E, g.R) : 1);
}

__device__ __forceinline__ void store_out(const MatmulArgs& g, int row, int col, float v) {
  const int64_t i = (int64_t)row * g.ldo + col;
  if (g.out_bf16) static_cast<__bf16*>(g.out)[i] = (__bf16)v;
  else static_cast<float*>(g.out)[i] = v;
}

// Row of `a` behind output row r, or -1 where the index points outside.
__device__ __forceinline__ int64_t source_row(const MatmulArgs& g, int r) {
  if (!g.index) return r;
  const int t = g.index[r];
  return t >= 0 && t < g.a_rows ? t : -1;
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
        union {
          bf16x2 p[4];
          bf16x8 v;
        } A;
        A.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ww[i], s, 0);
        A.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ww[i], s, 1);
        A.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ww[i], s, 2);
        A.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ww[i], s, 3);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A.v, __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
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
  const int nt = (g.N + 63) / 64;
  const dim3 grid((unsigned)(max_units(g, 16) * nt));
  if (a_mxfp4) hipLaunchKernelGGL(mx_matmul_kernel<true>, grid, dim3(256), 0, s, g, nt);
  else hipLaunchKernelGGL(mx_matmul_kernel<false>, grid, dim3(256), 0, s, g, nt);
  return hipGetLastError();
}

hipError_t launch_mx_matmul_dx(const MatmulArgs& g, hipStream_t s) {
  const int nt = (g.K + 511) / 512;
  hipLaunchKernelGGL(mx_matmul_dx_kernel, dim3((unsigned)(max_units(g, 1) * nt)), dim3(256), 0, s, g, nt);
  return hipGetLastError();
}

}  // namespace qmoe
