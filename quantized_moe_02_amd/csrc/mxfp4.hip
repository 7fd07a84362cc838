// Rows to MXFP4 and back: E2M1 codes with one power-of-two scale (E8M0) per
// 32 inputs.
//
// With E the biased fp32 exponent of a block's largest magnitude, the scale's
// byte is max(E - 2, 0): 2^(floor(log2 amax) - 2), which brings the largest
// magnitude into [4, 8), E2M1's top binade and its overflow.  The conversion
// instructions take the scale as an fp32 of which they use the exponent field
// alone, 0 standing for 2^-127, so the byte shifted by 23 is their operand;
// they round to nearest even and saturate at 6.
#include "operators_internal.h"
#include "qmoe_device.h"

namespace qmoe {
namespace {

template <int DT>
__device__ __forceinline__ float mx_load(const void* p, int64_t i) {
  if constexpr (DT == MOE_DT_F32) return static_cast<const float*>(p)[i];
  if constexpr (DT == MOE_DT_BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  return (float)static_cast<const _Float16*>(p)[i];
}

template <int DT>
__device__ __forceinline__ void mx_store(void* p, int64_t i, float v) {
  if constexpr (DT == MOE_DT_F32) static_cast<float*>(p)[i] = v;
  else if constexpr (DT == MOE_DT_BF16) static_cast<__bf16*>(p)[i] = (__bf16)v;
  else static_cast<_Float16*>(p)[i] = (_Float16)v;
}

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`;
// 255 if that is an infinity or a NaN (whose bits compare above all others).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const int e = (int)(amax >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}

// One thread per block of 32 inputs.
template <int DT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(MxQuantArgs a, int nb) {
  const int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (b >= a.rows * nb) return;
  const int64_t row = b / nb, c0 = (b - row * nb) * kMxBlock;
  float v[kMxBlock];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < kMxBlock; ++i) {
    v[i] = c0 + i < a.cols ? mx_load<DT>(a.x, row * a.ld + c0 + i) : 0.0f;
    amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  }
  const uint32_t sb = mx_scale_byte(amax);
  const float s = __uint_as_float(sb << 23);
  uint32_t w[4] = {0, 0, 0, 0};
  if (sb != 255) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], v[8 * i], v[8 * i + 1], s, 0);
      w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], v[8 * i + 2], v[8 * i + 3], s, 1);
      w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], v[8 * i + 4], v[8 * i + 5], s, 2);
      w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], v[8 * i + 6], v[8 * i + 7], s, 3);
    }
  }
  reinterpret_cast<uint4*>(a.codes)[b] = make_uint4(w[0], w[1], w[2], w[3]);
  a.scale[b] = (uint8_t)sb;
}

template <int DT>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(MxQuantArgs a, int nb) {
  const int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (b >= a.rows * nb) return;
  const int64_t row = b / nb, c0 = (b - row * nb) * kMxBlock;
  const uint4 q = reinterpret_cast<const uint4*>(a.codes)[b];
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  const float s = __uint_as_float((uint32_t)a.scale[b] << 23);
  typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f32x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], s, 3);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c0 + 8 * i + j < a.cols) mx_store<DT>(a.x, row * a.ld + c0 + 8 * i + j, v[j >> 1][j & 1]);
  }
}

template <class F>
hipError_t by_dtype(int dtype, F&& f) {
  if (dtype == MOE_DT_F32) f(std::integral_constant<int, MOE_DT_F32>{});
  else if (dtype == MOE_DT_BF16) f(std::integral_constant<int, MOE_DT_BF16>{});
  else f(std::integral_constant<int, MOE_DT_F16>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t s) {
  const int nb = (int)((a.cols + kMxBlock - 1) / kMxBlock);
  const int64_t grid = (a.rows * nb + 255) / 256;
  return by_dtype(a.dtype, [&](auto D) {
    hipLaunchKernelGGL(mx_quantize_kernel<decltype(D)::value>, dim3((unsigned)grid), dim3(256), 0, s, a, nb);
  });
}

hipError_t launch_mx_dequantize(const MxQuantArgs& a, hipStream_t s) {
  const int nb = (int)((a.cols + kMxBlock - 1) / kMxBlock);
  const int64_t grid = (a.rows * nb + 255) / 256;
  return by_dtype(a.dtype, [&](auto D) {
    hipLaunchKernelGGL(mx_dequantize_kernel<decltype(D)::value>, dim3((unsigned)grid), dim3(256), 0, s, a, nb);
  });
}

}  // namespace qmoe
