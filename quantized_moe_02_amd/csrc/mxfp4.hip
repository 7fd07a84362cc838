// Rows to MXFP4 and back: E2M1 codes with one power-of-two scale (E8M0) per
// 32 inputs.
//
// With E the biased fp32 exponent of a block's largest magnitude, the scale's
// byte is max(E - 2, 0): 2^(floor(log2 amax) - 2), which brings the largest
// magnitude into [4, 8), E2M1's top binade and its overflow.  The conversion
// instructions take the scale as an fp32 of which they use the exponent field
// alone, 0 standing for 2^-127, so the byte shifted by 23 is their operand;
// they round to nearest even and saturate at 6.
//
// Both directions move bytes and are bound by HBM (small calls: by the
// launch: a row of 6144 takes 1.8 us each way).  A lane takes a chunk of eight inputs, four lanes a block, so a
// wave reads (16-bit types) and writes whole lines; the four meet in two
// cross-lane maxima.  Magnitudes compare as integers, two 16-bit ones per
// instruction.  Rows may start at any element: the loads are declared
// unaligned, which costs nothing where they are aligned.
#include <algorithm>

#include "operators_internal.h"
#include "qmoe_device.h"

namespace qmoe {
namespace {

constexpr int kChunk = 8;     // inputs per lane

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Chunks are numbered along the rows, `cpr` a row.  Exact for every chunk of a
// workgroup: below 8192 (cpr <= 4096) or at most one row further.
struct ChunkMap {
  uint64_t magic64;   // floor(2^64 / cpr) + 1
  uint32_t magic32;   // floor(2^32 / cpr) + 1
  uint32_t cpr;
};

template <int DT>
struct Elem {
  static constexpr int kBytes = DT == MOE_DT_F32 ? 4 : 2;
  static constexpr int kWords = kChunk * kBytes / 4;
};

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// The fp32 exponent field of the largest magnitude of eight inputs (255: an
// infinity or a NaN among them).
template <int DT>
__device__ __forceinline__ uint32_t top_exponent(const uint32_t* w) {
  uint32_t m;
  if constexpr (DT == MOE_DT_F32) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
    m = max(m, dpp<kDppXor1>(m));
    m = max(m, dpp<kDppXor2>(m));
    return m >> 23;
  } else {
    m = pk_max_u16(pk_max_u16(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), pk_max_u16(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    m = pk_max_u16(m, dpp<kDppXor1>(m));
    m = pk_max_u16(m, dpp<kDppXor2>(m));
    m = max(m & 0xffffu, m >> 16);
    if constexpr (DT == MOE_DT_BF16) return m >> 7;
    return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)m)) >> 23;
  }
}

template <int DT>
__device__ __forceinline__ uint32_t encode(const uint32_t* w, float s) {
  uint32_t q = 0;
  static_for<4>([&](auto I) {
    constexpr int i = decltype(I)::value;
    if constexpr (DT == MOE_DT_F32)
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]), s, i);
    else if constexpr (DT == MOE_DT_BF16)
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, w[i]), s, i);
    else
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, w[i]), s, i);
  });
  return q;
}

// Row and column chunk of chunk `first + local` of a workgroup that starts at
// (row0, c0).
__device__ __forceinline__ void locate(const ChunkMap& m, uint32_t x, uint32_t& row, uint32_t& c) {
  row = m.cpr > 4096u ? (x >= m.cpr ? 1u : 0u) : m.cpr > 1u ? __umulhi(x, m.magic32) : x;
  c = x - row * m.cpr;
}

template <int DT, int U>
__global__ void __launch_bounds__(256) mx_quantize_kernel(MxQuantArgs a, ChunkMap m, uint64_t chunks) {
  using L = Elem<DT>;
  const uint64_t first = (uint64_t)blockIdx.x * (256 * U);
  const uint64_t row0 = m.cpr > 1u ? __umul64hi(first, m.magic64) : first;
  const uint32_t c0 = (uint32_t)(first - row0 * m.cpr);
  uint32_t w[U][L::kWords];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t r, c;
    locate(m, c0 + u * 256 + threadIdx.x, r, c);
#pragma unroll
    for (int i = 0; i < L::kWords; ++i) w[u][i] = 0;
    if (first + u * 256 + threadIdx.x < chunks) {
      const int64_t col = (int64_t)c * kChunk;
      const uint8_t* p = static_cast<const uint8_t*>(a.x) + ((int64_t)(row0 + r) * a.ld + col) * L::kBytes;
      if (col + kChunk <= a.cols) {
        __builtin_memcpy(w[u], p, kChunk * L::kBytes);
      } else {   // the row's last inputs, then zeros
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          if (col + i < a.cols) {
            if constexpr (DT == MOE_DT_F32) w[u][i] = reinterpret_cast<const uint32_t*>(p)[i];
            else w[u][i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
          }
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t e = top_exponent<DT>(w[u]);
    const uint32_t sb = e == 255u ? 255u : (uint32_t)max((int)e - 2, 0);
    const uint32_t q = e == 255u ? 0u : encode<DT>(w[u], __uint_as_float(sb << 23));
    const uint64_t at = first + u * 256 + threadIdx.x;
    if (at < chunks) {
      reinterpret_cast<uint32_t*>(a.codes)[at] = q;
      if ((threadIdx.x & 3) == 0) a.scale[at >> 2] = (uint8_t)sb;
    }
  }
}

template <int DT, int U>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(MxQuantArgs a, ChunkMap m, uint64_t chunks) {
  using L = Elem<DT>;
  const uint64_t first = (uint64_t)blockIdx.x * (256 * U);
  const uint64_t row0 = m.cpr > 1u ? __umul64hi(first, m.magic64) : first;
  const uint32_t c0 = (uint32_t)(first - row0 * m.cpr);
  uint32_t q[U], sb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t at = min(first + u * 256 + threadIdx.x, chunks - 1);
    q[u] = reinterpret_cast<const uint32_t*>(a.codes)[at];
    sb[u] = a.scale[at >> 2];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t r, c;
    locate(m, c0 + u * 256 + threadIdx.x, r, c);
    const float s = __uint_as_float(sb[u] << 23);
    uint32_t w[L::kWords];
    static_for<4>([&](auto I) {
      constexpr int i = decltype(I)::value;
      if constexpr (DT == MOE_DT_BF16) {
        w[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[u], s, i));
      } else {
        const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], s, i);
        if constexpr (DT == MOE_DT_F32) {
          w[2 * i] = __float_as_uint(v[0]);
          w[2 * i + 1] = __float_as_uint(v[1]);
        } else {
          const f16x2 h = {(_Float16)v[0], (_Float16)v[1]};
          w[i] = __builtin_bit_cast(uint32_t, h);
        }
      }
    });
    if (first + u * 256 + threadIdx.x < chunks) {
      const int64_t col = (int64_t)c * kChunk;
      uint8_t* p = static_cast<uint8_t*>(a.x) + ((int64_t)(row0 + r) * a.ld + col) * L::kBytes;
      if (col + kChunk <= a.cols) {
        __builtin_memcpy(p, w, kChunk * L::kBytes);
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          if (col + i < a.cols) {
            if constexpr (DT == MOE_DT_F32) reinterpret_cast<uint32_t*>(p)[i] = w[i];
            else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
          }
        }
      }
    }
  }
}

// Calls f(dtype, chunks per lane) as integral constants.  One chunk per lane:
// small workgroups in order suit HBM (fp32, 98304 x 2048: 191 us to codes and 173
// back, 4.8 and 5.3 TB/s; with four in flight 205 and 219).  16-bit values that the
// 256 MB cache behind L2 holds, eight workgroups to a CU and more, come faster than
// a wave asks for them: four chunks in flight (fp16, 32768 x 2048, both ways: 53 us
// against 58; bf16, 16384 x 6144: 94 against 90; fp16, 4099 x 2057: 12.1 against 11.2).
template <class F>
hipError_t dispatch(const MxQuantArgs& a, uint64_t chunks, F&& f) {
  const bool four = chunks >= 1u << 21 && chunks <= 1u << 23;
  auto by_u = [&](auto D) {
    if (four) f(D, std::integral_constant<int, 4>{});
    else f(D, std::integral_constant<int, 1>{});
  };
  if (a.dtype == MOE_DT_F32) f(std::integral_constant<int, MOE_DT_F32>{}, std::integral_constant<int, 1>{});
  else if (a.dtype == MOE_DT_BF16) by_u(std::integral_constant<int, MOE_DT_BF16>{});
  else by_u(std::integral_constant<int, MOE_DT_F16>{});
  return hipGetLastError();
}

// Calls launch(part, map, chunks) for runs of whole rows of at most 2^31 chunks (a
// row has 2^21 at most): a launch has to stay below 2^32 work items, and larger
// matrices fit the card.
template <class F>
hipError_t by_rows(const MxQuantArgs& a, F&& launch) {
  const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock;
  ChunkMap m;
  m.cpr = (uint32_t)(nb * (kMxBlock / kChunk));
  m.magic64 = ~0ull / m.cpr + 1;
  m.magic32 = ~0u / m.cpr + 1;
  const int64_t most = (int64_t)((1u << 31) / m.cpr), size = a.dtype == MOE_DT_F32 ? 4 : 2;
  for (int64_t r = 0; r < a.rows; r += most) {
    MxQuantArgs part = a;
    part.x = static_cast<uint8_t*>(a.x) + r * a.ld * size;
    part.codes = a.codes + r * nb * (kMxBlock / 2);
    part.scale = a.scale + r * nb;
    part.rows = std::min(most, a.rows - r);
    const hipError_t e = launch(part, m, (uint64_t)part.rows * m.cpr);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t s) {
  return by_rows(a, [&](const MxQuantArgs& p, const ChunkMap& m, uint64_t chunks) {
    return dispatch(p, chunks, [&](auto D, auto U) {
      constexpr int u = decltype(U)::value;
      hipLaunchKernelGGL((mx_quantize_kernel<decltype(D)::value, u>), dim3((unsigned)((chunks + 256 * u - 1) / (256 * u))),
                         dim3(256), 0, s, p, m, chunks);
    });
  });
}

hipError_t launch_mx_dequantize(const MxQuantArgs& a, hipStream_t s) {
  return by_rows(a, [&](const MxQuantArgs& p, const ChunkMap& m, uint64_t chunks) {
    return dispatch(p, chunks, [&](auto D, auto U) {
      constexpr int u = decltype(U)::value;
      hipLaunchKernelGGL((mx_dequantize_kernel<decltype(D)::value, u>), dim3((unsigned)((chunks + 256 * u - 1) / (256 * u))),
                         dim3(256), 0, s, p, m, chunks);
    });
  });
}

}  // namespace qmoe
