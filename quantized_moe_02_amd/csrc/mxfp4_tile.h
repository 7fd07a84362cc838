// Device helpers of the MXFP4 products: runs of rows, work items, operands and
// stores.
//
// MFMA operands (a wave of 64, lane = 16 lq + lr): of a 16 x 16 tile, lane
// (lr, lq) feeds row lr of A and column lr of B with the same inputs, any
// assignment of inputs to (step, lq, element) being valid as long as A and B
// share it, and holds rows 4 lq .. 4 lq + 3 of column lr of the result.  A is
// the weights (rows: output features) and B the rows of `a`, so a lane ends up
// with four consecutive outputs of one row.
#pragma once

#include "operators_internal.h"
#include "qmoe_device.h"

namespace qmoe {

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


// s_waitcnt immediate: all but the n most recent vector memory ops, and every
// LDS read (gfx9 encoding: vmcnt in bits 3-0 and 15-14, lgkmcnt in 11-8).
__host__ __device__ constexpr int waitcnt_vm_lds(int n) { return (n & 15) | (7 << 4) | ((n >> 4) << 14); }

}  // namespace qmoe
