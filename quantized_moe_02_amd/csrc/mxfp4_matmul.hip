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
#include <algorithm>

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

// Eight codes as bf16 with their block's scale (an fp32 whose exponent it is).
__device__ __forceinline__ bf16x8 bf16_of(uint32_t w, float s) {
  union {
    bf16x2 p[4];
    bf16x8 v;
  } A;
  A.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  A.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  A.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  A.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return A.v;
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

// ---------------------------------------------------------------------------
// Large products.  One workgroup of eight waves per CU; a work item is up to
// 256 rows of one expert times 256 outputs (waves 4 x 2), or up to 128 rows
// times 512 outputs (8 x 1): either way a wave holds 64 outputs x 128 rows in
// its accumulators, and a K block costs the CU 64 KB of LDS reads for 2048
// (bf16) MFMAs.  The weights go from global memory straight into registers
// (no other wave of the 8 x 1 form needs them), the rows of `a` through LDS by
// direct loads, two stages deep: block kb + 1 is requested when block kb has
// landed, a K block's MFMAs (two waves per SIMD) taking longer than the loads.
// ---------------------------------------------------------------------------
constexpr int kFatRows = 256, kFatThreads = 512;
constexpr int kStageBytes = 64 * 1024;

// Work item of workgroup b: workgroups go round-robin over the 8 XCDs, and
// each XCD's share is a contiguous range, so that the output tiles of one run
// of rows meet in one L2.
__device__ __forceinline__ int xcd_item(int b, int total) {
  const int x = b & 7, q = total >> 3, r = total & 7;
  return x * q + min(x, r) + (b >> 3);
}


struct FatItem {
  int e, r0, M, tile;
  bool wide;   // 4 x 2 waves: 256 outputs; else 8 x 1: 512
};

// Items in order of expert, output tile, run of up to 256 rows, so that what an
// XCD works on at a time shares weights as well as rows; a last run of at most
// 128 rows takes the narrow form, after the others.  All 512 threads call it.
__device__ __forceinline__ bool find_item(const int32_t* offsets, int E, int R, int ntw, int ntn, FatItem& it) {
  __shared__ int ws[4], hit[4], tot;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  int lo = 0, cnt = 0;
  if (!offsets) {
    cnt = t == 0 ? R : 0;
  } else if (t < E) {
    lo = min(max(offsets[t], 0), R);
    cnt = min(max(offsets[t + 1], lo), R) - lo;
  }
  const int rem = cnt & (kFatRows - 1);
  const int wide = cnt / kFatRows + (rem > kFatRows / 2);   // runs of the wide form
  const int u = wide * ntw + (rem > 0 && rem <= kFatRows / 2 ? ntn : 0);
  int inc = u;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(inc, d, 64);
    if (lane >= d) inc += v;
  }
  if (lane == 63 && wv < 4) ws[wv] = inc;
  __syncthreads();
  if (wv < 4)
    for (int i = 0; i < wv; ++i) inc += ws[i];
  if (t == 255) tot = inc;
  __syncthreads();
  const int total = tot;
  if ((int)blockIdx.x >= total) return false;
  const int w = xcd_item(blockIdx.x, total);
  if (wv < 4 && w >= inc - u && w < inc) {
    const int k = w - (inc - u);
    const int run = k < wide * ntw ? k % wide : wide;
    hit[0] = t;
    hit[1] = lo + run * kFatRows;
    hit[2] = min(kFatRows, cnt - run * kFatRows);
    hit[3] = k < wide * ntw ? k / wide : k - wide * ntw;
  }
  __syncthreads();
  it.e = __builtin_amdgcn_readfirstlane(hit[0]);
  it.r0 = __builtin_amdgcn_readfirstlane(hit[1]);
  it.M = __builtin_amdgcn_readfirstlane(hit[2]);
  it.tile = __builtin_amdgcn_readfirstlane(hit[3]);
  it.wide = it.M > kFatRows / 2;
  return true;
}

constexpr uint32_t kOutside = 0xff000000u;   // offset past every descriptor here, with room for a row's length

// 16 bytes per lane from buffer offset `off` into LDS at dst + 16 lane.
__device__ __forceinline__ void to_lds16(const rsrc_t& r, uint8_t* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
}

// Stores four consecutive outputs of one row (col % 4 == 0).
__device__ __forceinline__ void store4(const MatmulArgs& g, bool vec, int row, int col, const f32x4& v) {
  const int64_t i = (int64_t)row * g.ldo + col;
  if (vec && col + 4 <= g.N) {
    if (g.out_bf16) {
      typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
      bf16x4 o = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
      *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(g.out) + i) = o;
    } else {
      *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + i) = v;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (col + j < g.N) store_out(g, row, col + j, v[j]);
}

// LDS of one stage: rows of 256 bytes (bf16: 128 inputs) or 128 bytes (MXFP4:
// 256 inputs), 16-byte chunk c of row r at chunk c ^ (r mod 16) of its row, or
// c ^ (r / 2 mod 8): the 16 rows that one operand read touches then lie on
// distinct banks.
template <bool MX>
struct FatShape {
  static constexpr int kK = MX ? 256 : 128;             // inputs per K block
  static constexpr int kRowBytes = MX ? 128 : 256;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kWC = MX ? 2 : 1;                // 16-byte weight chunks per lane and row tile
  static __device__ __forceinline__ int place(int row, int c) {
    return MX ? c ^ ((row >> 1) & 7) : c ^ (row & 15);
  }
};

struct FatLds {
  uint8_t *st0, *st1;     // stages of K blocks
  uint32_t *sc0, *sc1;    // scales of MXFP4 rows, one stage each
  uint8_t* ws;            // weight scales: two groups of 16 blocks, 16 bytes per output
};

// SL: the scales of 16 blocks of an output are 16 aligned bytes (K % 128 ==
// 0), which come into LDS one group ahead: a scale byte per lane costs the
// address units as much as 16 bytes of codes.  Otherwise lanes load bytes.
template <bool MX, bool SL, int WT, int CT>
__device__ __forceinline__ void fat_tile(const MatmulArgs& g, const FatItem& it, const FatLds& lds) {
  using F = FatShape<MX>;
  constexpr int WN = 8 / WT, RT = 4, ROWS = 16 * CT * WT;
  constexpr int SLOTS = ROWS * F::kChunks, NA = (SLOTS + kFatThreads - 1) / kFatThreads;
  constexpr int GB = 16 / (F::kK / kMxBlock);   // K blocks per group of scales
  static_assert(ROWS * F::kRowBytes <= kStageBytes, "a stage fits");
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % WN, wt = wv / WN;
  const int n0 = it.tile * (64 * WN) + wn * 64;
  const int nb = g.K / kMxBlock, nkb = (g.K + F::kK - 1) / F::kK;

  // rows of `a`: this thread's chunk of each load
  const int64_t ldb = MX ? g.K / 2 : g.lda * 2;
  const uint8_t* abase = static_cast<const uint8_t*>(g.a) + (g.index ? 0 : (int64_t)it.r0 * ldb);
  const rsrc_t ar = make_rsrc(abase, kOutside);
  uint32_t aoff[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int slot = i * kFatThreads + tid, row = slot / F::kChunks;
    aoff[i] = kOutside;
    if (row < it.M) {
      const int64_t src = g.index ? source_row(g, it.r0 + row) : row;
      if (src >= 0) aoff[i] = (uint32_t)(src * ldb) + 16u * F::place(row, slot % F::kChunks);
    }
  }
  // MXFP4 rows: thread t < 2 ROWS carries four scale bytes of row t / 2
  const rsrc_t asr = make_rsrc(MX ? g.a_scale + (g.index ? 0 : (int64_t)it.r0 * nb) : nullptr, kOutside);
  uint32_t asoff = kOutside;
  if (MX && tid < 2 * ROWS && tid / 2 < it.M) {
    const int64_t src = g.index ? source_row(g, it.r0 + tid / 2) : tid / 2;
    if (src >= 0) asoff = (uint32_t)(src * nb) + 4u * (tid & 1);
  }
  // weights: rows past N lie past the descriptors
  const int64_t erow = (int64_t)it.e * g.N;
  const rsrc_t wr = make_rsrc(g.w_codes + erow * (g.K / 2), (uint32_t)g.N * (uint32_t)(g.K / 2));
  const rsrc_t sr = make_rsrc(g.w_scale + erow * nb, (uint32_t)g.N * (uint32_t)nb);
  const uint32_t woff = (uint32_t)(n0 + lr) * (uint32_t)(g.K / 2) + 16u * F::kWC * lq;
  const uint32_t soff = (uint32_t)(n0 + (SL ? lane : lr)) * (uint32_t)nb + (SL ? 0u : (uint32_t)(F::kWC * lq));

  uint32_t wq[2][RT][F::kWC][4], wsc[2][RT], asc = 0;
  auto issue_a = [&](auto P, int kb, int i) {
    constexpr int p = decltype(P)::value;
    if (i * kFatThreads + wv * 64 >= SLOTS) return;
    uint32_t off = aoff[i] + (uint32_t)kb * F::kRowBytes;
    if constexpr (MX || !SL) {   // chunks past K
      const int slot = i * kFatThreads + tid, c = F::place(slot / F::kChunks, slot % F::kChunks);
      off = kb * F::kK + c * (F::kK / F::kChunks) >= g.K ? kOutside : off;
    }
    to_lds16(ar, (p ? lds.st1 : lds.st0) + (i * kFatThreads + wv * 64) * 16, off);
  };
  auto issue_w = [&](auto P, int kb, int rt) {
    constexpr int p = decltype(P)::value;
#pragma unroll
    for (int c = 0; c < F::kWC; ++c)
      bload16(wq[p][rt][c], wr, woff + (uint32_t)rt * 16u * (uint32_t)(g.K / 2) + (uint32_t)kb * (F::kK / 2) + 16u * c, 0);
    if constexpr (!SL) {
      // blocks past K: the next row's scales, which may be NaN, times zeros
      const int b = kb * (F::kK / 32) + F::kWC * lq;
      const uint32_t so = soff + (uint32_t)rt * 16u * (uint32_t)nb + (uint32_t)kb * (F::kK / 32);
      wsc[p][rt] = __builtin_amdgcn_raw_buffer_load_b8(sr, b < nb ? so : kOutside, 0, 0);
      if constexpr (MX)
        wsc[p][rt] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(sr, b + 1 < nb ? so + 1 : kOutside, 0, 0) << 8;
    }
  };
  // K block kb's scales of the rows (MXFP4), and the weight scales of its group if kb starts one
  auto issue_s = [&](int kb) {
    if constexpr (MX) {
      if constexpr (SL) {
        asc = __builtin_amdgcn_raw_buffer_load_b32(asr, kb * 8 + 4 * (tid & 1) < nb ? asoff + (uint32_t)kb * 8u : kOutside, 0, 0);
      } else {
        asc = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          asc |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(asr, kb * 8 + 4 * (tid & 1) + j < nb ? asoff + (uint32_t)(kb * 8 + j) : kOutside, 0, 0) << (8 * j);
      }
    }
    if constexpr (SL) {
      if (wt == 0 && kb % GB == 0)
        to_lds16(sr, lds.ws + ((kb / GB) & 1) * (512 * 16) + wn * 1024, soff + (uint32_t)kb * (F::kK / 32));
    }
  };
  // the weight scales of K block kb, from LDS
  auto read_ws = [&](auto P, int kb) {
    constexpr int p = decltype(P)::value;
    if constexpr (SL) {
      const uint8_t* b = lds.ws + ((kb / GB) & 1) * (512 * 16) + (wn * 64 + lr) * 16 + (kb % GB) * (F::kK / 32) + F::kWC * lq;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        wsc[p][rt] = MX ? *reinterpret_cast<const uint16_t*>(b + rt * 256) : b[rt * 256];
      // a group that ends past K holds the next row's scales there
      if ((kb + 1) * F::kK > g.K && kb * (F::kK / 32) + F::kWC * lq >= nb) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) wsc[p][rt] = 0;
      }
    }
  };

  f32x4 acc[RT][CT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[rt][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Multiplies K block kb in sub-steps of HB column tiles, the operands of the
  // next one read from LDS while this one's MFMAs run.  The requests for block
  // kb + 1 are spread over the first half of the sub-steps: issued at once they
  // would stall every wave until the address units have taken them all.
  constexpr int HB = CT < 2 ? 1 : 2, SUB = CT / HB;
  constexpr int STEPS = MX ? 2 : 4, NSUB = STEPS * SUB, IS = NSUB > 1 ? NSUB / 2 : 1;
  auto block = [&](auto P, int kb) {
    constexpr int p = decltype(P)::value;
    using Q = std::integral_constant<int, 1 - p>;
    const uint8_t* st = p ? lds.st1 : lds.st0;
    if constexpr (MX) {
      if (tid < 2 * ROWS) (p ? lds.sc1 : lds.sc0)[tid] = asc;
    }
    // block kb has landed, in every wave; nobody reads the other stage any more
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    read_ws(P, kb);
    uint32_t ts[CT];
    if constexpr (MX) {
#pragma unroll
      for (int c = 0; c < CT; ++c)
        ts[c] = reinterpret_cast<const uint16_t*>(p ? lds.sc1 : lds.sc0)[((wt * CT + c) * 16 + lr) * 4 + lq];
    }
    __builtin_amdgcn_sched_barrier(0);
    const int kn = min(kb + 1, nkb - 1);   // the last block is requested twice: no branch
    bf16x8 A[RT];
    uint4 B[2][HB];
    auto read_b = [&](int j) {   // column tiles HB (j % SUB) .. of step j / SUB
      const int s = j / SUB;
#pragma unroll
      for (int c = 0; c < HB; ++c) {
        const int row = (wt * CT + HB * (j % SUB) + c) * 16 + lr;
        B[j & 1][c] = *reinterpret_cast<const uint4*>(st + row * F::kRowBytes + 16 * F::place(lr, (MX ? 2 : 4) * lq + s));
      }
    };
    read_b(0);
    if constexpr (!MX) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) A[rt] = bf16_of(wq[p][rt][0][0], __uint_as_float(wsc[p][rt] << 23));
    }
#pragma unroll
    for (int j = 0; j < NSUB; ++j) {
      const int s = j / SUB;
      if (j + 1 < NSUB) read_b(j + 1);
      if (j < IS) {
#pragma unroll
        for (int i = 0; i < NA; ++i)
          if (i % IS == j) issue_a(Q{}, kn, i);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          if (rt % IS == j) issue_w(Q{}, kn, rt);
        if (j == 0) issue_s(kn);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int c = 0; c < HB; ++c) {
          const int ct = HB * (j % SUB) + c;
          if constexpr (MX) {
            const uint32_t* w = wq[p][rt][s % F::kWC];
            const i32x8 Av = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
            const uint4 v = B[j & 1][c];
            const i32x8 Bv = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
            acc[rt][ct] = s == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(Av, Bv, acc[rt][ct], 4, 4, 0, (int)wsc[p][rt], 0, (int)ts[ct])
                                 : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(Av, Bv, acc[rt][ct], 4, 4, 1, (int)wsc[p][rt], 1, (int)ts[ct]);
          } else {
            acc[rt][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[rt], __builtin_bit_cast(bf16x8, B[j & 1][c]), acc[rt][ct], 0, 0, 0);
          }
        }
        // the next step's operand, in the registers that these MFMAs are done with
        if constexpr (!MX)
          if (j % SUB == SUB - 1 && s + 1 < STEPS)
            A[rt] = bf16_of(wq[p][rt][0][s + 1], __uint_as_float(wsc[p][rt] << 23));
      }
      // the next reads first, then the next codes' conversion between the MFMAs
      __builtin_amdgcn_sched_group_barrier(0x100, HB, 0);
#pragma unroll
      for (int i = 0; i < HB * RT; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  issue_s(0);
#pragma unroll
  for (int i = 0; i < NA; ++i) issue_a(std::integral_constant<int, 0>{}, 0, i);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) issue_w(std::integral_constant<int, 0>{}, 0, rt);
  for (int kb = 0; kb < nkb; kb += 2) {
    block(std::integral_constant<int, 0>{}, kb);
    if (kb + 1 < nkb) block(std::integral_constant<int, 1>{}, kb + 1);
  }

  const bool vec = g.ldo % 4 == 0;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int row = (wt * CT + c) * 16 + lr;
    if (row >= it.M) continue;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) store4(g, vec, it.r0 + row, n0 + 16 * rt + 4 * lq, acc[rt][c]);
  }
}

template <bool MX, bool SL>
__global__ void __launch_bounds__(kFatThreads, 2) mx_matmul_fat_kernel(MatmulArgs g, int ntw, int ntn) {
  __shared__ __attribute__((aligned(16))) uint8_t st0[kStageBytes / (MX ? 2 : 1)];
  __shared__ __attribute__((aligned(16))) uint8_t st1[kStageBytes / (MX ? 2 : 1)];
  __shared__ __attribute__((aligned(16))) uint8_t wsl[SL ? 2 * 512 * 16 : 16];
  __shared__ uint32_t sc0[MX ? 512 : 1], sc1[MX ? 512 : 1];
  FatItem it;
  if (!find_item(g.offsets, g.E, g.R, ntw, ntn, it)) return;
  const FatLds lds{st0, st1, sc0, sc1, wsl};
  if (it.wide) {
    if (it.M > 192) fat_tile<MX, SL, 2, 8>(g, it, lds);
    else fat_tile<MX, SL, 2, 6>(g, it, lds);
  } else {
    if (it.M > 96) fat_tile<MX, SL, 1, 8>(g, it, lds);
    else if (it.M > 64) fat_tile<MX, SL, 1, 6>(g, it, lds);
    else if (it.M > 32) fat_tile<MX, SL, 1, 4>(g, it, lds);
    else if (it.M > 16) fat_tile<MX, SL, 1, 2>(g, it, lds);
    else fat_tile<MX, SL, 1, 1>(g, it, lds);
  }
}

}  // namespace

hipError_t launch_mx_matmul(const MatmulArgs& g, bool a_mxfp4, hipStream_t s) {
  // few rows per expert, or too few outputs to give a quarter of the CUs an
  // item: the small kernel; sources past 32-bit offsets too
  const int64_t ldb = a_mxfp4 ? g.K / 2 : g.lda * 2;
  const int64_t span = (g.index ? (int64_t)g.a_rows : kFatRows) * ldb;
  if (g.R >= 8 * (int64_t)g.E && (int64_t)g.R * g.N >= 64 * 256 * 256 && span < (int64_t)kOutside) {
    const int ntw = (g.N + 255) / 256, ntn = (g.N + 511) / 512;
    const dim3 grid((unsigned)(((long)g.R / kFatRows + std::min(g.E, g.R)) * ntw));
    const bool sl = g.K % 128 == 0;
    auto* k = a_mxfp4 ? (sl ? mx_matmul_fat_kernel<true, true> : mx_matmul_fat_kernel<true, false>)
                      : (sl ? mx_matmul_fat_kernel<false, true> : mx_matmul_fat_kernel<false, false>);
    hipLaunchKernelGGL(k, grid, dim3(kFatThreads), 0, s, g, ntw, ntn);
    return hipGetLastError();
  }
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
