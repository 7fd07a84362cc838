// Root-mean-square norm with the residual's addition, and its gradient.
//
// A row lies in the registers of the G lanes that share it, U units of eight
// values a lane, so that it is read once for its sum of squares and its result
// alike: a wave takes a row of up to 512 columns, a workgroup of 256 one of up to
// 8192.  Longer rows are read again from L2 for each pass over them.
#include <algorithm>

#include "rows_device.h"

namespace qmoe {
namespace {

constexpr int kBlock = 256;
constexpr int kWide = 1024;      // lanes for rows past kBlock * 4 units

// What is done with eight values of y.
template <int G>
__device__ __forceinline__ void put_y(const NormArgs& a, int row, int c, const float (&v)[kUnit]) {
  const int n = a.cols - c;
  if (a.y.p && n > 0) store_unit(a.y.p, a.y.dtype, (int64_t)row * a.y.ld + c, n, v);
}

// MXFP4 of a unit; all lanes of a quad take part, also those past the row's end.
__device__ __forceinline__ void put_mxfp4(const NormArgs& a, int row, int c, const float (&v)[kUnit]) {
  uint32_t byte;
  const uint32_t q = mxfp4_codes(v, byte);
  const int nb = (a.cols + kMxBlock - 1) / kMxBlock;
  if (c < nb * kMxBlock) {
    static_cast<uint32_t*>(a.q)[(int64_t)row * nb * 4 + c / kUnit] = q;
    if (c % kMxBlock == 0) static_cast<uint8_t*>(a.q_scale)[(int64_t)row * nb + c / kMxBlock] = (uint8_t)byte;
  }
}

// h of a unit (rounded to the stream's type), 0 past the row's end.
template <int DT>
__device__ __forceinline__ void add_residual(const NormArgs& a, const Unit<DT>& x, const Unit<DT>& r, float (&h)[kUnit]) {
  unit_floats(x, a.x.dtype, h);
  if (a.res.p) {
    float v[kUnit];
    unit_floats(r, a.res.dtype, v);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) h[i] += v[i];
    round_to(a.res.dtype, h);
  }
}

__device__ __forceinline__ float inverse_rms(double sum, int cols, float eps) {
  return (float)(1.0 / sqrt(sum / cols + (double)eps));
}

template <int DT, int G, int U>
__global__ void __launch_bounds__(kBlock) rmsnorm_kernel(NormArgs a) {
  __shared__ double sums[kBlock / kWave];
  __shared__ uint32_t tops[kBlock / kWave];
  const int lane = threadIdx.x % G;
  const int row = blockIdx.x * (kBlock / G) + __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  if (row >= a.rows) return;
  Unit<DT> x[U], r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * G + lane) * kUnit;
    load_unit(x[u], a.x.p, a.x.dtype, (int64_t)row * a.x.ld + c, a.cols - c);
    if (a.res.p) load_unit(r[u], a.res.p, a.res.dtype, (int64_t)row * a.res.ld + c, a.cols - c);
  }
  float h[U][kUnit];
  double sum = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * G + lane) * kUnit, n = a.cols - c;
    add_residual(a, x[u], r[u], h[u]);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) sum += (double)h[u][i] * h[u][i];
    if (a.h.p && n > 0) store_unit(a.h.p, a.h.dtype, (int64_t)row * a.h.ld + c, n, h[u]);
  }
  if (!a.y.p && !a.q) return;
  const float m = inverse_rms(group_sum<G>(sum, sums), a.cols, a.eps);
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * G + lane) * kUnit;
    Unit<kAnyDtype> w;
    float wv[kUnit];
    load_unit(w, a.w, a.w_dtype, c, a.cols - c);
    unit_floats(w, a.w_dtype, wv);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) h[u][i] = c + i < a.cols ? h[u][i] * m * wv[i] : 0.0f;
    put_y<G>(a, row, c, h[u]);
    if (a.q && a.q_dtype == MOE_DT_MXFP4) put_mxfp4(a, row, c, h[u]);
    top = max(top, top_bits(h[u]));
  }
  if (a.q && a.q_dtype == MOE_DT_E4M3) {
    const float scale = e4m3_scale(group_max<G>(top, tops));
    const float inv = scale == scale ? 1.0f / scale : 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (u * G + lane) * kUnit, n = a.cols - c;
      if (n > 0) store_bytes(static_cast<uint8_t*>(a.q) + (int64_t)row * a.cols + c, n, e4m3_codes(h[u], inv));
    }
    if (lane == 0) static_cast<float*>(a.q_scale)[row] = scale;
  }
}

// Rows of any length, a workgroup each, read again for each pass over them.  h,
// which may be the residual itself, is written with the last reading.
__global__ void __launch_bounds__(kWide) rmsnorm_wide_kernel(NormArgs a) {
  __shared__ double sums[kWide / kWave];
  __shared__ uint32_t tops[kWide / kWave];
  const int row = blockIdx.x;
  const int span = (a.cols + kMxBlock - 1) / kMxBlock * kMxBlock;     // whole quads of lanes
  auto read = [&](int c, float (&h)[kUnit]) {
    Unit<kAnyDtype> x, r;
    load_unit(x, a.x.p, a.x.dtype, (int64_t)row * a.x.ld + c, a.cols - c);
    if (a.res.p) load_unit(r, a.res.p, a.res.dtype, (int64_t)row * a.res.ld + c, a.cols - c);
    add_residual(a, x, r, h);
  };
  auto normed = [&](int c, float m, float (&h)[kUnit]) {
    Unit<kAnyDtype> w;
    float wv[kUnit];
    load_unit(w, a.w, a.w_dtype, c, a.cols - c);
    unit_floats(w, a.w_dtype, wv);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) h[i] = c + i < a.cols ? h[i] * m * wv[i] : 0.0f;
  };
  double sum = 0;
  float h[kUnit];
  for (int c = threadIdx.x * kUnit; c < span; c += kWide * kUnit) {
    read(c, h);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) sum += (double)h[i] * h[i];
  }
  const float m = inverse_rms(group_sum<kWide>(sum, sums), a.cols, a.eps);
  float scale = 0.0f, inv = 0.0f;
  if (a.q && a.q_dtype == MOE_DT_E4M3) {
    uint32_t top = 0;
    for (int c = threadIdx.x * kUnit; c < span; c += kWide * kUnit) {
      read(c, h);
      normed(c, m, h);
      top = max(top, top_bits(h));
    }
    scale = e4m3_scale(group_max<kWide>(top, tops));
    inv = scale == scale ? 1.0f / scale : 0.0f;
    if (threadIdx.x == 0) static_cast<float*>(a.q_scale)[row] = scale;
  }
  for (int c = threadIdx.x * kUnit; c < span; c += kWide * kUnit) {
    const int n = a.cols - c;
    read(c, h);
    if (a.h.p && n > 0) store_unit(a.h.p, a.h.dtype, (int64_t)row * a.h.ld + c, n, h);
    normed(c, m, h);
    put_y<kWide>(a, row, c, h);
    if (!a.q) continue;
    if (a.q_dtype == MOE_DT_MXFP4) put_mxfp4(a, row, c, h);
    else if (n > 0) store_bytes(static_cast<uint8_t*>(a.q) + (int64_t)row * a.cols + c, n, e4m3_codes(h, inv));
  }
}

// Sums over a row that the gradient needs.
struct RowSums {
  double squares, product;     // of h; of g * h
};

// m and m^2 * mean(g * h) of a row.
__device__ __forceinline__ void row_factors(RowSums s, int cols, float eps, float& m, float& k) {
  const double r = 1.0 / sqrt(s.squares / cols + (double)eps);
  m = (float)r;
  k = (float)(s.product / cols * r * r);
}

template <int DT, int G, int U>
__global__ void __launch_bounds__(kBlock) rmsnorm_grad_kernel(NormGradArgs a) {
  constexpr int kRows = kBlock / G;
  __shared__ double lds[2][2][kBlock / kWave];
  const int lane = threadIdx.x % G;
  const int first = blockIdx.x * kRows + __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  float acc[U][kUnit] = {};
  int turn = 0;
  for (int row = first; row < a.rows; row += gridDim.x * kRows, turn ^= 1) {
    Unit<DT> hr[U], yr[U], dr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (u * G + lane) * kUnit, n = a.cols - c;
      load_unit(hr[u], a.h.p, a.h.dtype, (int64_t)row * a.h.ld + c, n);
      load_unit(yr[u], a.dy.p, a.dy.dtype, (int64_t)row * a.dy.ld + c, n);
      if (a.dh.p) load_unit(dr[u], a.dh.p, a.dh.dtype, (int64_t)row * a.dh.ld + c, n);
    }
    RowSums s{0, 0};
    float h[U][kUnit], dy[U][kUnit], w[U][kUnit];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (u * G + lane) * kUnit, n = a.cols - c;
      Unit<kAnyDtype> wr;
      load_unit(wr, a.w, a.w_dtype, c, n);
      unit_floats(wr, a.w_dtype, w[u]);
      unit_floats(hr[u], a.h.dtype, h[u]);
      unit_floats(yr[u], a.dy.dtype, dy[u]);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        s.squares += (double)h[u][i] * h[u][i];
        s.product += (double)(dy[u][i] * w[u][i]) * h[u][i];
      }
    }
    s.squares = group_sum<G>(s.squares, lds[turn][0]);
    s.product = group_sum<G>(s.product, lds[turn][1]);
    float m, k;
    row_factors(s, a.cols, a.eps, m, k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (u * G + lane) * kUnit, n = a.cols - c;
      float dx[kUnit];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        dx[i] = m * (dy[u][i] * w[u][i] - h[u][i] * k);
        acc[u][i] += dy[u][i] * (h[u][i] * m);
      }
      if (a.dh.p) {
        float d[kUnit];
        unit_floats(dr[u], a.dh.dtype, d);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) dx[i] += d[i];
      }
      if (n > 0) store_unit(a.dx.p, a.dx.dtype, (int64_t)row * a.dx.ld + c, n, dx);
    }
  }
  if (!a.dw) return;
  float* part = gridDim.x == 1 ? a.dw : a.part + (int64_t)blockIdx.x * a.cols;
  if constexpr (kRows > 1) {       // the waves' sums, in order
    __shared__ float waves[kRows][G * U * kUnit];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) waves[threadIdx.x / G][(u * G + lane) * kUnit + i] = acc[u][i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kBlock) {
      float v = waves[0][c];
#pragma unroll
      for (int i = 1; i < kRows; ++i) v += waves[i][c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (u * G + lane) * kUnit;
      if (c < a.cols) store_unit(part, MOE_DT_F32, c, a.cols - c, acc[u]);
    }
  }
}

// Rows past kBlock * 4 units: read twice, dweight's sums in registers.
template <int U>
__global__ void __launch_bounds__(kWide) rmsnorm_grad_wide_kernel(NormGradArgs a) {
  __shared__ double lds[2][2][kWide / kWave];
  float acc[U][kUnit] = {};
  int turn = 0;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    auto read = [&](int c, float (&h)[kUnit], float (&dy)[kUnit], float (&g)[kUnit]) {
      Unit<kAnyDtype> v;
      const int n = a.cols - c;
      load_unit(v, a.h.p, a.h.dtype, (int64_t)row * a.h.ld + c, n);
      unit_floats(v, a.h.dtype, h);
      load_unit(v, a.dy.p, a.dy.dtype, (int64_t)row * a.dy.ld + c, n);
      unit_floats(v, a.dy.dtype, dy);
      load_unit(v, a.w, a.w_dtype, c, n);
      unit_floats(v, a.w_dtype, g);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) g[i] *= dy[i];
    };
    RowSums s{0, 0};
    float h[kUnit], dy[kUnit], g[kUnit];
    for (int c = threadIdx.x * kUnit; c < a.cols; c += kWide * kUnit) {
      read(c, h, dy, g);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        s.squares += (double)h[i] * h[i];
        s.product += (double)g[i] * h[i];
      }
    }
    s.squares = group_sum<kWide>(s.squares, lds[turn][0]);
    s.product = group_sum<kWide>(s.product, lds[turn][1]);
    float m, k;
    row_factors(s, a.cols, a.eps, m, k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (u * kWide + threadIdx.x) * kUnit, n = a.cols - c;
      if (n <= 0) continue;
      read(c, h, dy, g);
      float dx[kUnit];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        dx[i] = m * (g[i] - h[i] * k);
        acc[u][i] += dy[i] * (h[i] * m);
      }
      if (a.dh.p) {
        Unit<kAnyDtype> v;
        load_unit(v, a.dh.p, a.dh.dtype, (int64_t)row * a.dh.ld + c, n);
        unit_floats(v, a.dh.dtype, h);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) dx[i] += h[i];
      }
      store_unit(a.dx.p, a.dx.dtype, (int64_t)row * a.dx.ld + c, n, dx);
    }
  }
  if (!a.dw) return;
  float* part = gridDim.x == 1 ? a.dw : a.part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * kWide + threadIdx.x) * kUnit;
    if (c < a.cols) store_unit(part, MOE_DT_F32, c, a.cols - c, acc[u]);
  }
}

// dw[c] = sum of the workgroups' parts: 64 columns a workgroup, a share of the
// parts each wave, joined in order.
__global__ void __launch_bounds__(kWide) rmsnorm_dw_kernel(const float* part, int parts, int cols, float* dw) {
  __shared__ double lds[kWide / kWave][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * kWave + lane;
  double v = 0;
  if (c < cols) {
#pragma unroll 8
    for (int p = wave; p < parts; p += kWide / kWave) v += part[(int64_t)p * cols + c];
  }
  lds[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && c < cols) {
    for (int i = 1; i < kWide / kWave; ++i) v += lds[i][lane];
    dw[c] = (float)v;
  }
}

__global__ void __launch_bounds__(kBlock) fill_zero_kernel(float* p, int n) {
  const int i = blockIdx.x * kBlock + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

constexpr int kGradBlocks = 1024;

// Calls f(dtype, lanes, units) as integral constants for rows of up to 8192
// columns, g() for longer ones.
template <class F, class G>
void by_shape(bool all_bf16, bool all_f32, int cols, F&& f, G&& g) {
  using std::integral_constant;
  const int units = (cols + kUnit - 1) / kUnit;
  auto shape = [&](auto D) {
    if (units <= 64) f(D, integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (units <= 256) f(D, integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (units <= 512) f(D, integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (units <= 768) f(D, integral_constant<int, 256>{}, integral_constant<int, 3>{});
    else f(D, integral_constant<int, 256>{}, integral_constant<int, 4>{});
  };
  if (units > 1024) g();
  else if (all_bf16) shape(integral_constant<int, MOE_DT_BF16>{});
  else if (all_f32) shape(integral_constant<int, MOE_DT_F32>{});
  else shape(integral_constant<int, kAnyDtype>{});
}

bool all_of(int dtype, std::initializer_list<const RowMat*> all) {
  return std::all_of(all.begin(), all.end(), [&](const RowMat* m) { return !m->p || m->dtype == dtype; });
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s) {
  by_shape(all_of(MOE_DT_BF16, {&a.x, &a.res}), all_of(MOE_DT_F32, {&a.x, &a.res}), a.cols,
           [&](auto D, auto G, auto U) {
             constexpr int g = decltype(G)::value, rows = kBlock / g;
             hipLaunchKernelGGL((rmsnorm_kernel<decltype(D)::value, g, decltype(U)::value>),
                                dim3((a.rows + rows - 1) / rows), dim3(kBlock), 0, s, a);
           },
           [&] { hipLaunchKernelGGL(rmsnorm_wide_kernel, dim3(a.rows), dim3(kWide), 0, s, a); });
  return hipGetLastError();
}

int norm_grad_most_blocks(int rows) { return std::min(std::max(rows, 1), kGradBlocks); }

hipError_t launch_rmsnorm_grad(const NormGradArgs& a, hipStream_t s) {
  if (a.rows == 0) {
    hipLaunchKernelGGL(fill_zero_kernel, dim3((a.cols + kBlock - 1) / kBlock), dim3(kBlock), 0, s, a.dw, a.cols);
    return hipGetLastError();
  }
  const int per = a.cols <= 64 * kUnit ? kBlock / 64 : 1;     // rows a workgroup takes at a time
  const int blocks = std::min((a.rows + per - 1) / per, kGradBlocks);
  by_shape(all_of(MOE_DT_BF16, {&a.h, &a.dy, &a.dh}), all_of(MOE_DT_F32, {&a.h, &a.dy, &a.dh}), a.cols,
           [&](auto D, auto G, auto U) {
             hipLaunchKernelGGL((rmsnorm_grad_kernel<decltype(D)::value, decltype(G)::value, decltype(U)::value>),
                                dim3(blocks), dim3(kBlock), 0, s, a);
           },
           [&] {
             if (a.cols <= 2 * kWide * kUnit) hipLaunchKernelGGL((rmsnorm_grad_wide_kernel<2>), dim3(blocks), dim3(kWide), 0, s, a);
             else if (a.cols <= 4 * kWide * kUnit) hipLaunchKernelGGL((rmsnorm_grad_wide_kernel<4>), dim3(blocks), dim3(kWide), 0, s, a);
             else hipLaunchKernelGGL((rmsnorm_grad_wide_kernel<8>), dim3(blocks), dim3(kWide), 0, s, a);
           });
  if (a.dw && blocks > 1)
    hipLaunchKernelGGL(rmsnorm_dw_kernel, dim3((a.cols + kWave - 1) / kWave), dim3(kWide), 0, s, a.part, blocks, a.cols, a.dw);
  return hipGetLastError();
}

}  // namespace qmoe
