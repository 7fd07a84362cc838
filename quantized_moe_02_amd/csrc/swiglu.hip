// SwiGLU over rows [gate | up] in expert order, and its gradient.
//
//   out = g s up with s = 1 / (1 + e^-g);  dgate = dh up s (1 + g (1 - s)),  dup = dh g s
//
// Both move bytes and are bound by HBM: a lane takes eight values of gate, up (and dh)
// at once, rows behind the last expert's are left out by their number alone.  E4M3 needs
// a row's largest value first, so there the row stays in the registers of 8 to 1024
// lanes.  s is off by up to 6 2^-24 of itself at any g, 1 - s by 7 (sigmoids), and s is 0
// where it lies below 2^-126.
//
// Measured, averages: 32768 x 2048 bf16 66 us, its gradient 122 (403 and 671 MB, 6.1 and
// 5.5 TB/s); to E4M3 20000 x 2048 34.5 us (5.9 TB/s); 777 x 1001 fp32 4.0 and 5.0 us; 8 x
// 2048 to E4M3 2.8 us.
#include <algorithm>

#include "rows_device.h"

namespace qmoe {
namespace {

// s = 1 / (1 + e^-g) and 1 - s = e^-g s, without overflow and without cancellation.  The
// hardware's power of two takes t = g log2(e) as rounded; c, what t says less than g, comes in
// behind it, e^-c being 1 - c.  Without c, whose three operations do not show beside the bytes
// (32768 x 2048 bf16 67.8 us against 66.9, fp32 the same), s is off by 1.5 |g| 2^-24 more.
// Between the two ends e^-g is finite; at the lower one the reciprocal, which has no subnormal
// results, gives s = 0.  NaN comes back with the products by g.
__device__ __forceinline__ void sigmoids(float gate, float& s, float& rest) {
  constexpr double kLn2 = 0.693147180559945309417;
  constexpr float kHigh = (float)kLn2, kLow = (float)(kLn2 - kHigh);
  const float g = __builtin_amdgcn_fmed3f(gate, -88.5f, 200.0f), t = g * (float)(1 / kLn2);
  const float p = __builtin_amdgcn_exp2f(-t);
  const float c = fmaf(-t, kLow, fmaf(-t, kHigh, g));
  const float x = fmaf(p, -c, p);
  s = __builtin_amdgcn_rcpf(1.0f + x);
  rest = x * s;
}

__device__ __forceinline__ int rows_that_count(const SwigluArgs& a) {
  return a.end ? min(max(*a.end, 0), a.rows) : a.rows;
}

template <bool TAIL, int DT>
__device__ __forceinline__ void load_gate_up(const SwigluArgs& a, int64_t row, const Span<TAIL>& p, Unit<DT>& g, Unit<DT>& u) {
  load_unit<TAIL>(g, a.gu.p, kPlain<DT>, row * a.gu.ld + p.c, p.n);
  load_unit<TAIL>(u, a.gu.p, kPlain<DT>, row * a.gu.ld + a.cols + p.c, p.n);
}

template <int DT>
__device__ __forceinline__ void swiglu_unit(const Unit<DT>& gr, const Unit<DT>& ur, float (&v)[kUnit]) {
  float g[kUnit], up[kUnit];
  unit_floats(gr, kPlain<DT>, g);
  unit_floats(ur, kPlain<DT>, up);
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    float s, t;
    sigmoids(g[i], s, t);
    v[i] = g[i] * s * up[i];
  }
}

// fp32, bf16 and MXFP4: a unit a lane.  A row's units come in whole quads, which
// share a block of MXFP4.
template <int DT, bool LONG, bool TAIL>
__global__ void __launch_bounds__(kMapBlock) swiglu_kernel(SwigluArgs a, RowMap m) {
  int row, unit;
  locate<LONG>(m, row, unit);
  const int nb = (a.cols + kMxBlock - 1) / kMxBlock;
  if (row >= rows_that_count(a) || unit >= nb * 4) return;
  const Span<TAIL> p(unit, a.cols);
  Unit<DT> g, u;
  float v[kUnit];
  load_gate_up(a, row, p, g, u);
  swiglu_unit(g, u, v);
  if (a.out.dtype == MOE_DT_MXFP4) {
    uint32_t byte;
    own_first(v, p.skip);
    const uint32_t q = mxfp4_codes(v, byte);
    static_cast<uint32_t*>(a.out.p)[(int64_t)row * nb * 4 + unit] = q;
    if (unit % 4 == 0) static_cast<uint8_t*>(a.out_scale)[(int64_t)row * nb + unit / 4] = (uint8_t)byte;
  } else if (p.n > 0) {
    store_unit<TAIL>(a.out.p, a.out.dtype, row * a.out.ld + p.c, p.n, v);
  }
}

// E4M3: G lanes a row, which lies in their registers until its scale is known.
template <int DT, int G, int U, bool TAIL>
__global__ void __launch_bounds__(G > 256 ? G : 256) swiglu_e4m3_kernel(SwigluArgs a) {
  constexpr int kBlock = G > 256 ? G : 256;
  __shared__ uint32_t tops[kBlock / kWave];
  const int lane = threadIdx.x % G;
  int64_t row = a.first + (int64_t)blockIdx.x * (kBlock / G);
  if constexpr (G < kWave) row += threadIdx.x / G;
  else if constexpr (G == kWave) row += __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  if (row >= rows_that_count(a)) return;
  Unit<DT> g[U], u[U];
#pragma unroll
  for (int i = 0; i < U; ++i) load_gate_up(a, row, Span<TAIL>(i * G + lane, a.cols), g[i], u[i]);
  float v[U][kUnit];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    swiglu_unit(g[i], u[i], v[i]);
    top = max(top, top_bits(v[i]));
  }
  const float scale = e4m3_scale(group_max<G>(top, tops));
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const Span<TAIL> p(i * G + lane, a.cols);
    if (p.n > 0) store_bytes<TAIL>(static_cast<uint8_t*>(a.out.p) + row * a.cols + p.c, p.n, e4m3_codes(v[i], scale));
  }
  if (lane == 0) static_cast<float*>(a.out_scale)[row] = scale;
}

// Rows past 16384 columns, read again once their scale is known.
template <int DT>
__global__ void __launch_bounds__(1024) swiglu_e4m3_wide_kernel(SwigluArgs a) {
  __shared__ uint32_t tops[16];
  const int64_t row = a.first + (int64_t)blockIdx.x;
  if (row >= rows_that_count(a)) return;
  Unit<DT> g, u;
  float v[kUnit];
  uint32_t top = 0;
  for (int i = threadIdx.x; i * kUnit < a.cols; i += 1024) {
    load_gate_up(a, row, Span<false>(i, a.cols), g, u);
    swiglu_unit(g, u, v);
    top = max(top, top_bits(v));
  }
  const float scale = e4m3_scale(group_max<1024>(top, tops));
  for (int i = threadIdx.x; i * kUnit < a.cols; i += 1024) {
    const Span<false> p(i, a.cols);
    load_gate_up(a, row, p, g, u);
    swiglu_unit(g, u, v);
    store_bytes<false>(static_cast<uint8_t*>(a.out.p) + row * a.cols + p.c, p.n, e4m3_codes(v, scale));
  }
  if (threadIdx.x == 0) static_cast<float*>(a.out_scale)[row] = scale;
}

template <int DT, bool LONG, bool TAIL>
__global__ void __launch_bounds__(kMapBlock) swiglu_grad_kernel(SwigluArgs a, RowMap m) {
  int row, unit;
  locate<LONG>(m, row, unit);
  const Span<TAIL> p(unit, a.cols);
  if (row >= rows_that_count(a) || p.n <= 0) return;
  Unit<DT> gr, ur;
  Unit<kAnyDtype> dr;
  load_gate_up(a, row, p, gr, ur);
  load_unit<TAIL>(dr, a.out.p, a.out.dtype, row * a.out.ld + p.c, p.n);
  float g[kUnit], up[kUnit], dh[kUnit];
  unit_floats(gr, kPlain<DT>, g);
  unit_floats(ur, kPlain<DT>, up);
  unit_floats(dr, a.out.dtype, dh);
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    float s, t;
    sigmoids(g[i], s, t);
    const float d = dh[i] * s;
    const float dg = d * up[i] * fmaf(g[i], t, 1.0f);
    up[i] = d * g[i];
    g[i] = dg;
  }
  store_unit<TAIL>(a.dgu.p, kPlain<DT>, row * a.dgu.ld + p.c, p.n, g);
  store_unit<TAIL>(a.dgu.p, kPlain<DT>, row * a.dgu.ld + a.cols + p.c, p.n, up);
}

template <int DT>
hipError_t launch_e4m3(SwigluArgs a, hipStream_t s) {
  using std::integral_constant;
  const int units = (a.cols + kUnit - 1) / kUnit;
  // lanes that a row fills to two thirds and more (bf16 20000 x 1500 30 us against 32 with
  // half of 256 idle, 8000 x 6144 36 against 38, 4000 x 9000 36 against 40)
  auto with = [&](auto G, auto U, auto T) {
    constexpr int g = decltype(G)::value, block = g > 256 ? g : 256;
    return by_runs(a.rows, block, block / g, [&](int first, dim3 grid) {
      a.first = first;
      hipLaunchKernelGGL((swiglu_e4m3_kernel<DT, g, decltype(U)::value, decltype(T)::value>), grid, dim3(block), 0, s, a);
    });
  };
  auto at = [&](auto G, auto U) { return with(G, U, std::false_type{}); };
  if constexpr (DT != kBf16Once) {
    if (a.cols < kUnit) return with(integral_constant<int, 8>{}, integral_constant<int, 1>{}, std::true_type{});
  }
  if (units <= 8) return at(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (units <= 16) return at(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (units <= 32) return at(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (units <= 64) return at(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (units <= 128) return at(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if (units <= 192) return at(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  if (units <= 256) return at(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (units <= 512) return at(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (units <= 768) return at(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  if (units <= 1024) return at(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  if (units <= 1536) return at(integral_constant<int, 512>{}, integral_constant<int, 3>{});
  if (units <= 2048) return at(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  return by_runs(a.rows, 1024, 1, [&](int first, dim3 grid) {
    a.first = first;
    hipLaunchKernelGGL((swiglu_e4m3_wide_kernel<kPlain<DT>>), grid, dim3(1024), 0, s, a);
  });
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s) {
  const bool once = a.cols >= kUnit && read_once(a.gu, a.rows, (int64_t)2 * a.cols);
  if (a.out.dtype == MOE_DT_E4M3)
    return a.gu.dtype == MOE_DT_F32 ? launch_e4m3<MOE_DT_F32>(a, s) : once ? launch_e4m3<kBf16Once>(a, s) : launch_e4m3<MOE_DT_BF16>(a, s);
  const int nb = (a.cols + kMxBlock - 1) / kMxBlock;
  return by_rows<false>(row_map(nb * (kMxBlock / kUnit), a.out.dtype != MOE_DT_MXFP4 && ragged_lines(a.out.p, a.out.ld * element(a.out.dtype))), a.rows, a.cols < kUnit,
                 [&](auto L, auto T, dim3 grid, dim3 block, const RowMap& m) {
    constexpr bool l = decltype(L)::value, t = decltype(T)::value;
    if constexpr (!t) {
      if (once) {
        hipLaunchKernelGGL((swiglu_kernel<kBf16Once, l, t>), grid, block, 0, s, a, m);
        return;
      }
    }
    if (a.gu.dtype == MOE_DT_F32) hipLaunchKernelGGL((swiglu_kernel<MOE_DT_F32, l, t>), grid, block, 0, s, a, m);
    else hipLaunchKernelGGL((swiglu_kernel<MOE_DT_BF16, l, t>), grid, block, 0, s, a, m);
  });
}

hipError_t launch_swiglu_grad(const SwigluArgs& a, hipStream_t s) {
  const bool tail = a.cols < kUnit || (a.dgu.p == a.gu.p && a.cols % kUnit != 0);
  const bool once = !tail && a.dgu.p != a.gu.p && read_once(a.gu, a.rows, (int64_t)2 * a.cols);
  return by_rows<true>(row_map((a.cols + kUnit - 1) / kUnit, ragged_lines(a.dgu.p, a.dgu.ld * element(a.dgu.dtype))), a.rows, tail,
                 [&](auto L, auto T, dim3 grid, dim3 block, const RowMap& m) {
    constexpr bool l = decltype(L)::value, t = decltype(T)::value;
    if constexpr (!t) {
      if (once) {
        hipLaunchKernelGGL((swiglu_grad_kernel<kBf16Once, l, t>), grid, block, 0, s, a, m);
        return;
      }
    }
    if (a.gu.dtype == MOE_DT_F32) hipLaunchKernelGGL((swiglu_grad_kernel<MOE_DT_F32, l, t>), grid, block, 0, s, a, m);
    else hipLaunchKernelGGL((swiglu_grad_kernel<MOE_DT_BF16, l, t>), grid, block, 0, s, a, m);
  });
}

}  // namespace qmoe
