// SwiGLU over rows [gate | up] in expert order, and its gradient.
#include <algorithm>

#include "rows_device.h"

namespace qmoe {
namespace {

constexpr int kBlock = 256;

// s = 1 / (1 + e^-g) and 1 - s, without overflow and without cancellation.
__device__ __forceinline__ void sigmoids(float g, float& s, float& t) {
  const float x = __expf(-fabsf(g));
  const float r = __builtin_amdgcn_rcpf(1.0f + x);
  const float q = x * r;
  s = g < 0.0f ? q : r;
  t = g < 0.0f ? r : q;
}

__device__ __forceinline__ int rows_that_count(const SwigluArgs& a) {
  return a.end ? min(max(*a.end, 0), a.rows) : a.rows;
}

template <int DT>
__device__ __forceinline__ void swiglu_unit(const SwigluArgs& a, int64_t row, int c, float (&v)[kUnit]) {
  const int n = a.cols - c;
  Unit<DT> gr, ur;
  load_unit(gr, a.gu.p, DT, row * a.gu.ld + c, n);
  load_unit(ur, a.gu.p, DT, row * a.gu.ld + a.cols + c, n);
  float g[kUnit], up[kUnit];
  unit_floats(gr, DT, g);
  unit_floats(ur, DT, up);
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    float s, t;
    sigmoids(g[i], s, t);
    v[i] = g[i] * s * up[i];
  }
}

// A wave a row, `lanes` of it for MXFP4 a multiple of four.
template <int DT>
__global__ void __launch_bounds__(kBlock) swiglu_kernel(SwigluArgs a) {
  const int lane = threadIdx.x & 63;
  const int rows = rows_that_count(a);
  for (int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.x * 4) {
    const int nb = (a.cols + kMxBlock - 1) / kMxBlock;
    if (a.out.dtype == MOE_DT_E4M3) {
      uint32_t top = 0;
      float v[kUnit];
      for (int c = lane * kUnit; c < a.cols; c += kWave * kUnit) {
        swiglu_unit<DT>(a, row, c, v);
        top = max(top, top_bits(v));
      }
      const float scale = e4m3_scale(wave_max(top));
      const float inv = scale == scale ? 1.0f / scale : 0.0f;
      for (int c = lane * kUnit; c < a.cols; c += kWave * kUnit) {
        swiglu_unit<DT>(a, row, c, v);
        store_bytes(static_cast<uint8_t*>(a.out.p) + row * a.cols + c, a.cols - c, e4m3_codes(v, inv));
      }
      if (lane == 0) static_cast<float*>(a.out_scale)[row] = scale;
    } else {
      for (int c = lane * kUnit; c < nb * kMxBlock; c += kWave * kUnit) {
        float v[kUnit];
        swiglu_unit<DT>(a, row, c, v);
        if (a.out.dtype == MOE_DT_MXFP4) {
          uint32_t byte;
          const uint32_t q = mxfp4_codes(v, byte);
          static_cast<uint32_t*>(a.out.p)[row * nb * 4 + c / kUnit] = q;
          if (c % kMxBlock == 0) static_cast<uint8_t*>(a.out_scale)[row * nb + c / kMxBlock] = (uint8_t)byte;
        } else if (c < a.cols) {
          store_unit(a.out.p, a.out.dtype, row * a.out.ld + c, a.cols - c, v);
        }
      }
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(kBlock) swiglu_grad_kernel(SwigluArgs a) {
  const int lane = threadIdx.x & 63;
  const int rows = rows_that_count(a);
  for (int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.x * 4) {
    for (int c = lane * kUnit; c < a.cols; c += kWave * kUnit) {
      const int n = a.cols - c;
      Unit<DT> gr, ur;
      Unit<kAnyDtype> dr;
      load_unit(gr, a.gu.p, DT, row * a.gu.ld + c, n);
      load_unit(ur, a.gu.p, DT, row * a.gu.ld + a.cols + c, n);
      load_unit(dr, a.out.p, a.out.dtype, row * a.out.ld + c, n);
      float g[kUnit], up[kUnit], dh[kUnit];
      unit_floats(gr, DT, g);
      unit_floats(ur, DT, up);
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
      store_unit(a.dgu.p, DT, row * a.dgu.ld + c, n, g);
      store_unit(a.dgu.p, DT, row * a.dgu.ld + a.cols + c, n, up);
    }
  }
}

unsigned blocks_of(int rows) { return (unsigned)std::min((rows + 3) / 4, 1 << 16); }

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t s) {
  if (a.gu.dtype == MOE_DT_F32) hipLaunchKernelGGL((swiglu_kernel<MOE_DT_F32>), dim3(blocks_of(a.rows)), dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL((swiglu_kernel<MOE_DT_BF16>), dim3(blocks_of(a.rows)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_swiglu_grad(const SwigluArgs& a, hipStream_t s) {
  if (a.gu.dtype == MOE_DT_F32) hipLaunchKernelGGL((swiglu_grad_kernel<MOE_DT_F32>), dim3(blocks_of(a.rows)), dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL((swiglu_grad_kernel<MOE_DT_BF16>), dim3(blocks_of(a.rows)), dim3(kBlock), 0, s, a);
  return hipGetLastError();
}

}  // namespace qmoe
