// Tokens' rows into expert order (dispatch), back with weights (collect), and the
// gradient of the way back.
//
// A workgroup goes by tokens: a token's row is read (written) once, its top_k
// rows in expert order are written (read) where inv_perm says.  All of it moves
// bytes and is bound by HBM.
#include <algorithm>

#include "rows_device.h"

namespace qmoe {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxK = 16;

// How tokens and the chunks of their rows lie over workgroups: rows of 64 chunks
// and more in `parts` workgroups of `threads` lanes, shorter ones 2^bits lanes a
// token.
struct TokenMap {
  int parts, threads, bits;
  int first;                // token of the launch's first workgroup
};

TokenMap token_map(int chunks) {
  if (chunks > 32) {
    const int parts = (chunks + kBlock - 1) / kBlock;
    const int each = (chunks + parts - 1) / parts;
    return {parts, (each + kWave - 1) / kWave * kWave, -1, 0};
  }
  int bits = 0;
  while ((1 << bits) < chunks) ++bits;
  return {1, kBlock, bits, 0};
}

// Calls f(workgroups, map) for runs of tokens of at most 2^31 work items: a launch
// has to stay below 2^32.
template <class F>
hipError_t by_tokens(TokenMap m, int T, F&& f) {
  const int most = m.bits < 0 ? (int)((1u << 31) / ((unsigned)m.parts * kBlock)) : 1 << 20;
  for (; m.first < T; m.first += most) {
    const unsigned n = (unsigned)std::min(most, T - m.first);
    f(m.bits < 0 ? n * m.parts : ((n << m.bits) + kBlock - 1) / kBlock, m);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Token and chunk of a lane; the token is uniform where rows are long.
template <bool LONG>
__device__ __forceinline__ void locate(const TokenMap& m, int& t, int& c) {
  if constexpr (LONG) {
    const unsigned row = blockIdx.x / (unsigned)m.parts;
    c = (blockIdx.x - row * m.parts) * blockDim.x + threadIdx.x;
    t = m.first + row;
  } else {
    const unsigned at = blockIdx.x * kBlock + threadIdx.x;
    t = m.first + (at >> m.bits);
    c = at & ((1u << m.bits) - 1);
  }
}

// Bytes [at, at + n) of a row of bytes, n <= 16.
__device__ __forceinline__ uint4 load_bytes16(const uint8_t* p, int n) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (n >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < n) w[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}
__device__ __forceinline__ void store_bytes16(uint8_t* p, int n, const uint4& v) {
  if (n >= 16) {
    __builtin_memcpy(p, &v, 16);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < n) p[i] = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
  }
}

struct CopyArgs {
  const uint8_t *x, *x_scale;
  uint8_t *rows, *row_scale;
  int64_t x_pitch, row_pitch;   // bytes
  int row_bytes, scale_bytes;
  int chunks;                   // of 16 bytes a row
  const int32_t* inv;
  int T, K, slots;
};

// Rows as they are, then their scales: chunk `chunks` and the following ones.
template <bool LONG>
__global__ void __launch_bounds__(kBlock) dispatch_copy_kernel(CopyArgs a, TokenMap m) {
  int t, c;
  locate<LONG>(m, t, c);
  if (t >= a.T) return;
  const bool scale = c >= a.chunks;
  const int at = (scale ? c - a.chunks : c) * 16;
  const int bytes = scale ? a.scale_bytes : a.row_bytes;
  if (at >= bytes) return;
  const uint8_t* src = scale ? a.x_scale + (int64_t)t * bytes : a.x + t * a.x_pitch;
  const uint4 v = load_bytes16(src + at, bytes - at);
  for (int i = 0; i < a.K; ++i) {
    const int slot = a.inv[(int64_t)t * a.K + i];
    if ((unsigned)slot >= (unsigned)a.slots) continue;
    uint8_t* dst = scale ? a.row_scale + (int64_t)slot * bytes : a.rows + slot * a.row_pitch;
    store_bytes16(dst + at, bytes - at, v);
  }
}

// Rows from fp32 to bf16 or back.
template <int DT, bool LONG>
__global__ void __launch_bounds__(kBlock) dispatch_cast_kernel(DispatchArgs a, TokenMap m) {
  int t, c;
  locate<LONG>(m, t, c);
  c *= kUnit;
  const int n = a.cols - c;
  if (t >= a.T || n <= 0) return;
  Unit<DT> u;
  float v[kUnit];
  load_unit(u, a.x.p, DT, (int64_t)t * a.x.ld + c, n);
  unit_floats(u, DT, v);
  for (int i = 0; i < a.K; ++i) {
    const int slot = a.inv[(int64_t)t * a.K + i];
    if ((unsigned)slot >= (unsigned)a.slots) continue;
    store_unit(a.rows.p, DT == MOE_DT_BF16 ? MOE_DT_F32 : MOE_DT_BF16, (int64_t)slot * a.rows.ld + c, n, v);
  }
}

template <int DT, bool LONG>
__global__ void __launch_bounds__(kBlock) collect_kernel(CollectArgs a, TokenMap m) {
  int t, c;
  locate<LONG>(m, t, c);
  c *= kUnit;
  const int n = a.cols - c;
  if (t >= a.T || n <= 0) return;
  float y[kUnit] = {};
  for (int i = 0; i < a.K; ++i) {
    const int slot = a.inv[(int64_t)t * a.K + i];
    if ((unsigned)slot >= (unsigned)a.slots) continue;
    const float w = a.w ? a.w[(int64_t)t * a.K + i] : 1.0f;
    Unit<DT> u;
    float v[kUnit];
    load_unit(u, a.rows.p, DT, (int64_t)slot * a.rows.ld + c, n);
    unit_floats(u, DT, v);
#pragma unroll
    for (int j = 0; j < kUnit; ++j) y[j] = fmaf(w, v[j], y[j]);
  }
  if (a.add.p) {
    Unit<kAnyDtype> u;
    float v[kUnit];
    load_unit(u, a.add.p, a.add.dtype, (int64_t)t * a.add.ld + c, n);
    unit_floats(u, a.add.dtype, v);
#pragma unroll
    for (int j = 0; j < kUnit; ++j) y[j] += v[j];
  }
  store_unit(a.y.p, a.y.dtype, (int64_t)t * a.y.ld + c, n, y);
}

// One token a workgroup (G == 256) or a wave: its rows one after the other.
template <int DT, int G>
__global__ void __launch_bounds__(kBlock) collect_grad_kernel(CollectGradArgs a) {
  __shared__ float lds[kMaxK][kBlock / kWave];
  const int lane = threadIdx.x % G;
  const int t = blockIdx.x * (kBlock / G) + __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  if (t >= a.T) return;
  for (int i = 0; i < a.K; ++i) {
    const int slot = a.inv[(int64_t)t * a.K + i];
    const bool on = (unsigned)slot < (unsigned)a.slots;
    const float w = a.w ? a.w[(int64_t)t * a.K + i] : 1.0f;
    float dot = 0.0f;
    if (on) {
      for (int c = lane * kUnit; c < a.cols; c += G * kUnit) {
        const int n = a.cols - c;
        Unit<kAnyDtype> d;
        Unit<DT> r;
        float dy[kUnit], v[kUnit];
        load_unit(d, a.dy.p, a.dy.dtype, (int64_t)t * a.dy.ld + c, n);
        unit_floats(d, a.dy.dtype, dy);
        if (a.dw) {
          load_unit(r, a.rows.p, DT, (int64_t)slot * a.rows.ld + c, n);
          unit_floats(r, DT, v);
#pragma unroll
          for (int j = 0; j < kUnit; ++j) dot = fmaf(dy[j], v[j], dot);
        }
        if (a.drows.p) {
#pragma unroll
          for (int j = 0; j < kUnit; ++j) v[j] = w * dy[j];
          store_unit(a.drows.p, DT, (int64_t)slot * a.drows.ld + c, n, v);
        }
      }
    }
    if (a.dw) {
      dot = wave_sum(dot);
      if (G == kWave) {
        if (lane == 0) a.dw[(int64_t)t * a.K + i] = dot;
      } else if ((threadIdx.x & 63) == 0) {
        lds[i][threadIdx.x >> 6] = dot;
      }
    }
  }
  if (G > kWave && a.dw) {
    __syncthreads();
    if (lane < a.K) a.dw[(int64_t)t * a.K + lane] = (lds[lane][0] + lds[lane][1]) + (lds[lane][2] + lds[lane][3]);
  }
}

template <class F>
hipError_t by_length(const TokenMap& map, int T, F&& f) {
  return by_tokens(map, T, [&](unsigned blocks, const TokenMap& m) {
    if (m.bits < 0) f(std::true_type{}, dim3(blocks), dim3(m.threads), m);
    else f(std::false_type{}, dim3(blocks), dim3(m.threads), m);
  });
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s) {
  if (a.x.dtype != a.rows.dtype) {
    return by_length(token_map((a.cols + kUnit - 1) / kUnit), a.T, [&](auto L, dim3 grid, dim3 block, const TokenMap& m) {
      constexpr bool l = decltype(L)::value;
      if (a.x.dtype == MOE_DT_F32) hipLaunchKernelGGL((dispatch_cast_kernel<MOE_DT_F32, l>), grid, block, 0, s, a, m);
      else hipLaunchKernelGGL((dispatch_cast_kernel<MOE_DT_BF16, l>), grid, block, 0, s, a, m);
    });
  }
  CopyArgs c{};
  c.x = static_cast<const uint8_t*>(a.x.p);
  c.rows = static_cast<uint8_t*>(a.rows.p);
  c.x_scale = a.x_scale;
  c.row_scale = a.row_scale;
  c.scale_bytes = a.scale_bytes;
  if (a.x.dtype == MOE_DT_MXFP4) {
    c.row_bytes = (a.cols + kMxBlock - 1) / kMxBlock * (kMxBlock / 2);
    c.x_pitch = c.row_pitch = c.row_bytes;
  } else {
    const int size = a.x.dtype == MOE_DT_F32 ? 4 : a.x.dtype == MOE_DT_BF16 ? 2 : 1;
    c.row_bytes = a.cols * size;
    c.x_pitch = a.x.ld * size;
    c.row_pitch = a.rows.ld * size;
  }
  c.chunks = (c.row_bytes + 15) / 16;
  c.inv = a.inv;
  c.T = a.T;
  c.K = a.K;
  c.slots = a.slots;
  return by_length(token_map(c.chunks + (c.scale_bytes + 15) / 16), a.T, [&](auto L, dim3 grid, dim3 block, const TokenMap& m) {
    hipLaunchKernelGGL((dispatch_copy_kernel<decltype(L)::value>), grid, block, 0, s, c, m);
  });
}

hipError_t launch_collect(const CollectArgs& a, hipStream_t s) {
  return by_length(token_map((a.cols + kUnit - 1) / kUnit), a.T, [&](auto L, dim3 grid, dim3 block, const TokenMap& m) {
    constexpr bool l = decltype(L)::value;
    if (a.rows.dtype == MOE_DT_F32) hipLaunchKernelGGL((collect_kernel<MOE_DT_F32, l>), grid, block, 0, s, a, m);
    else hipLaunchKernelGGL((collect_kernel<MOE_DT_BF16, l>), grid, block, 0, s, a, m);
  });
}

hipError_t launch_collect_grad(const CollectGradArgs& a, hipStream_t s) {
  auto launch = [&](auto D) {
    constexpr int d = decltype(D)::value;
    if (a.cols <= 1024)
      hipLaunchKernelGGL((collect_grad_kernel<d, kWave>), dim3((a.T + 3) / 4), dim3(kBlock), 0, s, a);
    else
      hipLaunchKernelGGL((collect_grad_kernel<d, kBlock>), dim3(a.T), dim3(kBlock), 0, s, a);
  };
  if (a.rows.dtype == MOE_DT_F32) launch(std::integral_constant<int, MOE_DT_F32>{});
  else launch(std::integral_constant<int, MOE_DT_BF16>{});
  return hipGetLastError();
}

}  // namespace qmoe
