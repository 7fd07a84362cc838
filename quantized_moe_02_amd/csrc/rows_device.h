// Device code shared by the row operators: eight neighbouring values of a row
// (a "unit") are what a lane holds, 16 bytes of bf16 or 32 of fp32.
#pragma once

#include "qmoe_device.h"
#include "rows_internal.h"

namespace qmoe {

constexpr int kUnit = 8;
// dtype of a matrix known at compile time, or only at run time
constexpr int kAnyDtype = -1;

template <int DT>
struct Unit {
  uint32_t w[DT == MOE_DT_BF16 ? 4 : 8];
};

template <int DT>
__device__ __forceinline__ bool is_bf16(int dtype) {
  if constexpr (DT == kAnyDtype) return dtype == MOE_DT_BF16;
  return DT == MOE_DT_BF16;
}

// Values [at, at + 8) of a matrix in memory, those past the first n as zeros
// (n <= 0: none is read).
template <int DT>
__device__ __forceinline__ void load_unit(Unit<DT>& u, const void* base, int dtype, int64_t at, int n) {
  constexpr int kWords = DT == MOE_DT_BF16 ? 4 : 8;
#pragma unroll
  for (int i = 0; i < kWords; ++i) u.w[i] = 0;
  if (is_bf16<DT>(dtype)) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (n >= kUnit) {
      __builtin_memcpy(u.w, p, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (i < n) u.w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    }
  } else if constexpr (kWords == 8) {
    const uint32_t* p = static_cast<const uint32_t*>(base) + at;
    if (n >= kUnit) {
      __builtin_memcpy(u.w, p, 32);
    } else {
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (i < n) u.w[i] = p[i];
    }
  }
}

template <int DT>
__device__ __forceinline__ void unit_floats(const Unit<DT>& u, int dtype, float (&v)[kUnit]) {
  if (is_bf16<DT>(dtype)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(u.w[i]);
      v[2 * i + 1] = bf16_hi(u.w[i]);
    }
  } else if constexpr (DT != MOE_DT_BF16) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = __uint_as_float(u.w[i]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// Rounds eight values to a dtype and back.
__device__ __forceinline__ void round_to(int dtype, float (&v)[kUnit]) {
  if (dtype != MOE_DT_BF16) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = pack_bf16(v[2 * i], v[2 * i + 1]);
    v[2 * i] = bf16_lo(w);
    v[2 * i + 1] = bf16_hi(w);
  }
}

// The first n of eight values to [at, at + n) of a matrix.
__device__ __forceinline__ void store_unit(void* base, int dtype, int64_t at, int n, const float (&v)[kUnit]) {
  if (dtype == MOE_DT_BF16) {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if (n >= kUnit) {
      __builtin_memcpy(p, w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (i < n) p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  } else {
    float* p = static_cast<float*>(base) + at;
    if (n >= kUnit) {
      __builtin_memcpy(p, v, 32);
    } else {
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (i < n) p[i] = v[i];
    }
  }
}

// Largest magnitude of eight values as fp32 bits, which order like the values,
// infinities and NaN last.
__device__ __forceinline__ uint32_t top_bits(const float (&v)[kUnit]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
  m = max(m, dpp<kDppXor1>(m));
  m = max(m, dpp<kDppXor2>(m));
  m = max(m, dpp<kDppHalfMirror>(m));
  m = max(m, dpp<kDppMirror>(m));
  auto r = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  m = max(r[0], r[1]);
  r = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  return max(r[0], r[1]);
}

// Scale of an E4M3 row from its largest magnitude.  Below 2^-126 a scale would
// lose bits, and its reciprocal could overflow.
__device__ __forceinline__ float e4m3_scale(uint32_t top) {
  if (top >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(top) / 448.0f, 0x1p-126f);
}

// E4M3 codes of eight values times 1 / scale (0: all codes 0).  The product with
// the rounded reciprocal may pass 448 by a unit in the last place of fp32; E4M3
// rounds everything below 464 to 448.
__device__ __forceinline__ uint2 e4m3_codes(const float (&v)[kUnit], float inv) {
  if (inv == 0.0f) return make_uint2(0u, 0u);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
    q = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, q, true);
    w[i] = (uint32_t)q;
  }
  return make_uint2(w[0], w[1]);
}

// The first n of eight code bytes.
__device__ __forceinline__ void store_bytes(uint8_t* p, int n, uint2 q) {
  if (n >= kUnit) {
    __builtin_memcpy(p, &q, 8);
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
      if (i < n) p[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

// MXFP4 of a block of 32 that four neighbouring lanes hold, eight values each
// (values past the row's end zeros): this lane's codes and the block's scale
// byte, as moe_mxfp4_quantize makes them.
__device__ __forceinline__ uint32_t mxfp4_codes(const float (&v)[kUnit], uint32_t& byte) {
  uint32_t m = top_bits(v);
  m = max(m, dpp<kDppXor1>(m));
  m = max(m, dpp<kDppXor2>(m));
  const uint32_t e = m >> 23;
  byte = e == 255u ? 255u : (uint32_t)max((int)e - 2, 0);
  if (e == 255u) return 0;
  const float s = __uint_as_float(byte << 23);   // the conversion uses the exponent alone, 0 for 2^-127
  uint32_t q = 0;
  static_for<4>([&](auto I) {
    constexpr int i = decltype(I)::value;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2 * i], v[2 * i + 1], s, i);
  });
  return q;
}

// Sum (maximum) over the G lanes that share a row: a wave, or the whole
// workgroup through `lds`, which holds one value a wave and is free again after
// the next barrier.
template <int G>
__device__ __forceinline__ double group_sum(double v, double* lds) {
  v = wave_sum(v);
  if constexpr (G > kWave) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < G / kWave; ++i) v += lds[i];
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t* lds) {
  v = wave_max(v);
  if constexpr (G > kWave) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < G / kWave; ++i) v = max(v, lds[i]);
  }
  return v;
}

}  // namespace qmoe
