// Grouped products over MXFP4 expert weights for few rows, their gradient for
// few rows, and the choice of the kernel.
//
// A few rows per expert: the weights are read once and bound the call (HBM),
// or the call is a few microseconds of latency.  So the rows come into LDS, the
// weights straight from global memory into the matrix units' operands, whole
// lines per row, and the four waves of a workgroup split the sum and add their
// parts up in LDS, in a fixed order.  One token, 8 of 256 experts, 4096 x 6144: 24.1
// us (107 MB at 4.4 TB/s; shortest of 60 runs 23.4); 64 tokens, 76 experts, 6144 x
// 2048: 156 us (145).
#include <algorithm>
#include <cmath>

#include "mxfp4_tile.h"

namespace qmoe {
namespace {

constexpr int kThinRows = 16;                   // rows of a unit
constexpr int kThinLds = kThinRows * 4 * 512;   // four steps of them

// At most this many units for R rows of E experts.
long max_units(const MatmulArgs& g, int BM) {
  return (long)g.R / BM + (g.offsets ? (long)std::min(g.E, g.R) : 1);
}

// Calls launch(first unit, workgroups) for runs of units of `per` workgroups each: a
// launch has to stay below 2^32 work items.
template <class F>
hipError_t by_units(long units, long per, int threads, F&& launch) {
  const long most = (1l << 31) / (per * threads);
  for (long u = 0; u < units; u += most) {
    launch((int)u, dim3((unsigned)(std::min(most, units - u) * per)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// RT x 16 outputs x up to 16 rows, for one or several neighbouring tiles of
// outputs.  A step is 256 inputs, a line of a row's codes: lane (lr, lq) takes
// blocks 2 lq and 2 lq + 1 of row lr.  Wave w takes steps w, w + 4, ... of a
// slab, the steps whose rows fit LDS (most calls have one slab, whose rows then
// stay for every tile; of 9 to 16 rows it holds four steps, one of each wave, and
// nothing is in flight from slab to slab: 76 of 256 experts, 6144 x 2048, 8 rows each
// 131 us, 9 rows 154; 6144 x 1024, one slab either way, 74 and 75).  Two of a wave's steps are in flight: with three or
// four, one token's gate and up (8 experts) took 24.3 and 27.6 us instead of
// 23.4, the registers costing more waves than the loads gain.
// ---------------------------------------------------------------------------
// 16-byte chunk c (8 bf16 inputs) of row r of a slab of S steps, at c ^ r ^ (r / 2
// and 4) of its row: the four groups of lanes in which a wave's 16-byte reads go
// mix rows 0 to 3 and 12 to 15 of a chunk with rows 4 to 11 of the chunk eight on.
__device__ __forceinline__ int slab_at(int r, int S, int c) { return r * (512 * S) + (c ^ r ^ ((r >> 1) & 4)) * 16; }

// EV: an even number of blocks per row, whose scales come in pairs.
template <bool MX, int RT, bool EV>
__device__ __forceinline__ void thin_tiles(const MatmulArgs& g, const RowUnit& u, int tile, int tiles, lds8_t* lds, lds8_t* parts) {
  constexpr int D = 2;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nb = g.K / kMxBlock, steps = (g.K + 255) / 256;

  const int64_t erow = (int64_t)u.e * g.N;
  const uint32_t wld = (uint32_t)(g.K / 2);
  const rsrc_t wr = make_rsrc(g.w_codes + erow * wld, (uint32_t)g.N * wld);
  const rsrc_t sr = make_rsrc(g.w_scale + erow * nb, (uint32_t)g.N * (uint32_t)nb);
  // both chunks of a step and their scales (low byte: the first); blocks past
  // K get zero codes and the scale 2^-127
  uint32_t w[D][RT][2][4], sb[D][RT];
  auto load_w = [&](int d, int n0, int s) {
    const int b = s * 8 + 2 * lq;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const uint32_t row = (uint32_t)(n0 + 16 * rt + lr);
      const uint32_t at = row * wld + 16u * b, st = row * (uint32_t)nb + (uint32_t)b;
      bload16(w[d][rt][0], wr, b < nb ? at : kOutside, 0);
      bload16(w[d][rt][1], wr, b + 1 < nb ? at + 16u : kOutside, 0);
      if constexpr (EV)
        sb[d][rt] = bload_u16(sr, b < nb ? st : kOutside, 0);
      else
        sb[d][rt] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(sr, b < nb ? st : kOutside, 0, 0) |
                    (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(sr, b + 1 < nb ? st + 1u : kOutside, 0, 0) << 8;
    }
  };
  f32x4 acc[RT];
  const int64_t arow = MX && lr < u.M ? source_row(g, u.r0 + lr) : -1;
  // step s of the call, S steps from s0 on being in LDS (bf16 rows)
  auto multiply = [&](int d, int s, int s0, int S) {
    if constexpr (MX) {
      // rows in MXFP4: as small as the weights, read by every wave directly
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = s * 8 + 2 * lq + h;
        uint4 x = make_uint4(0, 0, 0, 0);
        uint32_t xs = 0;
        if (arow >= 0 && b < nb) {
          x = static_cast<const uint4*>(g.a)[arow * nb + b];
          xs = g.a_scale[arow * nb + b];
        }
        const i32x8 X = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const i32x8 W = {(int)w[d][rt][h][0], (int)w[d][rt][h][1], (int)w[d][rt][h][2], (int)w[d][rt][h][3], 0, 0, 0, 0};
          acc[rt] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(W, X, acc[rt], 4, 4, 0, (int)(sb[d][rt] >> (8 * h)), 0, (int)xs);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // lanes past the rows repeat the last one; their results are dropped
          const bf16x8 x = __builtin_bit_cast(bf16x8, lds_read16(lds + slab_at(min(lr, u.M - 1), S, (s - s0) * 32 + (2 * lq + h) * 4 + i)));
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            acc[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                bf16_of(w[d][rt][h][i], __uint_as_float((sb[d][rt] >> (8 * h)) << 23)), x, acc[rt], 0, 0, 0);
        }
    }
  };
  auto stage = [&](int s0, int S) {
    if constexpr (!MX) {
      for (int i = tid; i < u.M * S * 32; i += 256) {
        const int r = i / (S * 32), c = i - r * (S * 32), k = s0 * 256 + c * 8;
        const int64_t src = source_row(g, u.r0 + r);
        u32x4 v = {0u, 0u, 0u, 0u};
        if (src >= 0 && k < g.K) v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(g.a) + src * g.lda + k);
        lds_write16(lds + slab_at(r, S, c), v);
      }
      __syncthreads();
    }
  };
  // steps per slab: all of them, or a multiple of the four waves
  const int fit = MX ? steps : kThinLds / (u.M * 512), slab = fit >= steps ? steps : fit & ~3;
  auto first_steps = [&](int n0, int s0, int S) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (wv + 4 * d < S) load_w(d, n0, s0 + wv + 4 * d);
  };
  if (slab == steps) {
    first_steps(tile * 16 * RT, 0, steps);
    stage(0, steps);
  }
  for (int t = tile; t < tile + tiles; ++t) {
    const int n0 = t * 16 * RT;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < steps; s0 += slab) {
      const int S = min(slab, steps - s0);
      if (slab != steps) {
        first_steps(n0, s0, S);
        __syncthreads();   // the last slab is read
        stage(s0, S);
      }
      for (int s = s0 + wv; s < s0 + S; s += 4 * D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (s + 4 * d < s0 + S) {
            multiply(d, s + 4 * d, s0, S);
            if (s + 4 * (d + D) < s0 + S) load_w(d, n0, s + 4 * (d + D));
          }
        }
      }
    }
    // the next tile's first steps
    if (slab == steps && t + 1 < tile + tiles) first_steps(n0 + 16 * RT, 0, steps);
    // the waves' parts, added in order
#pragma unroll
    for (int i = 0; i < RT; ++i) lds_write16(parts + ((wv * RT + i) * 64 + lane) * 16, __builtin_bit_cast(u32x4, acc[i]));
    __syncthreads();
    for (int i = wv; i < RT; i += 4) {
      f32x4 v = __builtin_bit_cast(f32x4, lds_read16(parts + (i * 64 + lane) * 16));
#pragma unroll
      for (int p = 1; p < 4; ++p) v += __builtin_bit_cast(f32x4, lds_read16(parts + ((p * RT + i) * 64 + lane) * 16));
      if (lr < u.M) store4(g, u.r0 + lr, n0 + 16 * i + 4 * lq, g.N, v);
    }
    if (t + 1 < tile + tiles) __syncthreads();   // the parts are read
  }
}

template <bool MX, int RT, bool EV>
__global__ void __launch_bounds__(256) mx_matmul_thin_kernel(MatmulArgs g, int nt, int per, int first) {
  __shared__ __attribute__((aligned(16))) uint8_t rows[MX ? 16 : kThinLds], parts[4 * RT * 1024];
  const int runs = (nt + per - 1) / per;
  const int ub = blockIdx.x / runs, tile = (blockIdx.x - ub * runs) * per;
  const RowUnit u = find_unit(g.offsets, g.E, g.R, kThinRows, first + ub, reinterpret_cast<int*>(parts));
  if (u.M <= 0) return;
  thin_tiles<MX, RT, EV>(g, u, tile, min(per, nt - tile), (lds8_t*)rows, (lds8_t*)parts);
}

template <bool MX>
hipError_t launch_thin(const MatmulArgs& g, hipStream_t s) {
  const long units = max_units(g, kThinRows);
  // 64 outputs a tile (a row's inputs are then read for four row tiles) where
  // that leaves every CU several, else 32 or 16 (64 tokens, down projection: 317 us
  // with 64, 331 with 32, 395 with 16; one token, gate and up: 24.4, 22.8, 27.8; 16
  // rows, 4096 x 4096, one expert: 18.5, 14.8, 13.0); with many tiles, two to a
  // workgroup, which looks its rows up and brings them into LDS once (64 tokens,
  // down projection: one 168 us, two 153, four 158)
  const int rt = units * ((g.N + 63) / 64) >= 1024 ? 4 : units * ((g.N + 31) / 32) >= 512 ? 2 : 1;
  const int nt = (g.N + 16 * rt - 1) / (16 * rt);
  const int per = units * nt >= 8192 ? 2 : 1;
  return by_units(units, (nt + per - 1) / per, 256, [&](int first, dim3 grid) {
    auto go = [&](auto RT) {
      constexpr int r = decltype(RT)::value;
      if (g.K % 64 == 0) hipLaunchKernelGGL((mx_matmul_thin_kernel<MX, r, true>), grid, dim3(256), 0, s, g, nt, per, first);
      else hipLaunchKernelGGL((mx_matmul_thin_kernel<MX, r, false>), grid, dim3(256), 0, s, g, nt, per, first);
    };
    if (rt == 4) go(std::integral_constant<int, 4>{});
    else if (rt == 2) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 1>{});
  });
}

// ---------------------------------------------------------------------------
// The gradient: 128 CW columns x up to 16 rows.  As in the kernel for many rows, a
// lane takes words of eight rows of the weights and regroups them along the
// sum; here two words, 16 columns, so that a row's share is a whole line.  Four
// waves take every fourth step of 32 terms.  Where that gives fewer than 128
// workgroups their address units bound the call, 17 requests per step: half the
// columns and twice the waves then (CW = 1, NW = 8), 4096 x 512 and one row 12.1
// us instead of 19.6, but 64 experts, 32 rows, 4096 x 4096 (512 workgroups) 91
// instead of 51.
// ---------------------------------------------------------------------------
template <int CW, int NW>
__device__ __forceinline__ void dx_thin_tile(const MatmulArgs& g, const RowUnit& u, int k0, lds8_t* lds) {
  constexpr int NT = 8 * CW;   // tiles of 16 columns
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nb = g.K / kMxBlock, steps = g.N / 32;
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t erow = (int64_t)u.e * g.N;
  const rsrc_t wr = make_rsrc(g.w_codes + erow * (g.K / 2), (uint32_t)g.N * (uint32_t)(g.K / 2));
  const rsrc_t sr = make_rsrc(g.w_scale + erow * nb, (uint32_t)g.N * (uint32_t)nb);
  const int k = k0 + 8 * CW * lr;
  const uint32_t wat = (uint32_t)(8 * lq) * (uint32_t)(g.K / 2) + (uint32_t)(k / 2);
  const uint32_t sat = (uint32_t)(8 * lq) * (uint32_t)nb + (uint32_t)(k / 32);
  // lanes past the rows repeat the last one
  const uint16_t* dy = static_cast<const uint16_t*>(g.a) + (int64_t)(u.r0 + min(lr, u.M - 1)) * g.lda + 8 * lq;
  for (int s = wv; s < steps; s += NW) {
    uint32_t w[8][CW];
    float sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t o = (uint32_t)(32 * s + j), at = k < g.K ? wat + o * (uint32_t)(g.K / 2) : kOutside;
      if constexpr (CW == 2) bload8(w[j], wr, at, 0);
      else w[j][0] = __builtin_amdgcn_raw_buffer_load_b32(wr, at, 0, 0);
      sc[j] = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b8(sr, k < g.K ? sat + o * (uint32_t)nb : kOutside, 0, 0) << 23);
    }
    const bf16x8 B = *reinterpret_cast<const bf16x8*>(dy + 32 * s);
    static_for<NT / 2>([&](auto T) {
      constexpr int t = decltype(T)::value;
      union {
        uint32_t x[4];
        bf16x8 v;
      } lo, hi;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[2 * m][t / 4], sc[2 * m], t % 4));
        const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[2 * m + 1][t / 4], sc[2 * m + 1], t % 4));
        lo.x[m] = __builtin_amdgcn_perm(b, a, 0x05040100u);
        hi.x[m] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      }
      acc[2 * t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo.v, B, acc[2 * t], 0, 0, 0);
      acc[2 * t + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi.v, B, acc[2 * t + 1], 0, 0, 0);
    });
  }
  // the waves' parts, added in order; four tiles to each of the first waves
#pragma unroll
  for (int t = 0; t < NT; ++t) lds_write16(lds + ((wv * NT + t) * 64 + lane) * 16, __builtin_bit_cast(u32x4, acc[t]));
  __syncthreads();
  if (4 * wv >= NT || lr >= u.M) return;
  f32x4 v[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    v[t] = __builtin_bit_cast(f32x4, lds_read16(lds + ((4 * wv + t) * 64 + lane) * 16));
#pragma unroll
    for (int p = 1; p < NW; ++p) v[t] += __builtin_bit_cast(f32x4, lds_read16(lds + ((p * NT + 4 * wv + t) * 64 + lane) * 16));
  }
  // tile 4 wv + t, result row 4 lq + i: column NT (4 lq + i) + 4 wv + t
#pragma unroll
  for (int i = 0; i < 4; ++i)
    store4(g, u.r0 + lr, k0 + NT * (4 * lq + i) + 4 * wv, g.K, f32x4{v[0][i], v[1][i], v[2][i], v[3][i]});
}

template <int CW, int NW>
__global__ void __launch_bounds__(64 * NW) mx_matmul_dx_thin_kernel(MatmulArgs g, int nt, int first) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[NW * CW * 8192];
  const int ub = blockIdx.x / nt, tile = blockIdx.x - ub * nt;
  const RowUnit u = find_unit(g.offsets, g.E, g.R, kThinRows, first + ub, reinterpret_cast<int*>(smem));
  if (u.M <= 0) return;
  dx_thin_tile<CW, NW>(g, u, tile * (128 * CW), (lds8_t*)smem);
}

template <int CW, int NW>
hipError_t launch_dx_thin(const MatmulArgs& g, hipStream_t s) {
  const int nt = (g.K + 128 * CW - 1) / (128 * CW);
  return by_units(max_units(g, kThinRows), nt, 64 * NW, [&](int first, dim3 grid) {
    hipLaunchKernelGGL((mx_matmul_dx_thin_kernel<CW, NW>), grid, dim3(64 * NW), 0, s, g, nt, first);
  });
}


// ---------------------------------------------------------------------------
// The choice.  The offsets lie on the device, so the host goes by R / E rows per
// expert and part of a run more for each.  Measured both ways on log-uniform draws
// (1 to 256 experts, 16 to 6144 outputs, 32 to 6144 inputs):
//
// - An item of 64 rows needs four rows per expert and 128 in all to be worth its
//   place (256 experts, 1024 rows, 2048 x 1024: 64 us against 71 with few-row
//   units; 8 experts, 32 rows, 4096 x 4096: 24 against 20), and items enough to
//   make up for its slower start: 32 of them forwards (512 rows, 512 x 4096: 20
//   against 23; 14 experts, 825 rows, 54 x 4768: 26 against 22), for the gradient
//   as many as there are in 512 few-row units (8 experts, 4096 rows, 512 x 512:
//   11 against 16; 1024 rows, 4096 x 512: 51 against 30).
// - Items of 256 x 256, one to a CU, take two thirds of the time per result, but
//   leave CUs idle in the last round of them: 4096 rows, 4096 x 4096, one expert
//   (256 items), 109 us against 165; eight experts (more than 256) 175 against
//   150.
// ---------------------------------------------------------------------------
double runs_of(const MatmulArgs& g, double rows, double part = 0.5) {
  return g.E == 1 ? std::ceil(g.R / rows) : g.R / rows + part * g.E;
}

// Whether items of 64 rows x 128 outputs, 1350 of which the chip ends in the time
// of one item of 256 x 256, end before those.  Up to 128 rows per expert lie in
// one run of the narrow form, 512 outputs wide, which takes less time, but not
// less than half of it; a last run in that form is half as many items.
bool mid_is_faster(const MatmulArgs& g, int outputs) {
  const double rows = (double)g.R / g.E;
  const double large = rows <= 128 ? std::ceil(g.E * std::ceil(outputs / 512.0) / 256) * std::max(rows, 64.0) / 128
                                   : std::ceil(runs_of(g, 256, 0.25) * std::ceil(outputs / 256.0) / 256);
  return runs_of(g, 64) * std::ceil(outputs / 128.0) / 1350 < large;
}

}  // namespace

hipError_t launch_mx_matmul(const MatmulArgs& g, bool a_mxfp4, hipStream_t s) {
  // sources past 32-bit offsets: the few-row kernel, which has 64-bit addresses (32768
  // rows of 256 experts, 4096 x 8192, gathered from 262144 rows: 11.5 ms, from 261000
  // 1.9)
  const int64_t ldb = a_mxfp4 ? g.K / 2 : g.lda * 2;
  const int64_t span = (g.index ? (int64_t)g.a_rows : kFatRows) * ldb;
  const bool near = span < (int64_t)kOutside;
  if (a_mxfp4) {
    // sixteen items of 256 x 256, of eight rows per expert or more (8 experts, 256
    // rows, 4096 x 4096: 26 us against 43; 8 items, 512 rows, 1024 x 4096, and fewer
    // rows per expert alike within 1 us either way)
    if (near && g.R >= 8 * (int64_t)g.E && (int64_t)g.R * g.N >= 16 * 256 * 256) return launch_mx_matmul4_large(g, s);
    return launch_thin<true>(g, s);
  }
  if (near && g.R >= 128 && g.R >= 4 * (int64_t)g.E && runs_of(g, 64) * std::ceil(g.N / 128.0) >= 32)
    return mid_is_faster(g, g.N) ? launch_mx_matmul_mid(g, s) : launch_mx_matmul_large(g, s);
  return launch_thin<false>(g, s);
}

hipError_t launch_mx_matmul_dx(const MatmulArgs& g, hipStream_t s) {
  if (g.R >= 4 * (int64_t)g.E && g.R >= 128 && kFatRows * g.lda * 2 < (int64_t)kOutside &&
      runs_of(g, 16) * std::ceil(g.K / 256.0) >= 512)
    return mid_is_faster(g, g.K) ? launch_mx_matmul_dx_mid(g, s) : launch_mx_matmul_dx_large(g, s);
  return max_units(g, kThinRows) * ((g.K + 255) / 256) < 128 ? launch_dx_thin<1, 8>(g, s) : launch_dx_thin<2, 4>(g, s);
}

}  // namespace qmoe
