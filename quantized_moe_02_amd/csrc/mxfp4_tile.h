// Device helpers of the MXFP4 products: runs of rows, work items, operands and
// stores.
//
// MFMA operands: of a 16 x 16 tile, lane 16 lq + lr feeds row lr of A and
// column lr of B with the same inputs, any assignment of inputs to (step, lq,
// element) being valid as long as A and B share it, and holds rows 4 lq ..
// 4 lq + 3 of column lr of the result; of a 32 x 32 tile, lane 32 lh + ln row
// and column ln, and rows 8 q + 4 lh .. + 3 of column ln.  A is the weights
// (rows: output features) and B the rows of `a`, so a lane ends up with four
// consecutive outputs of one row.
//
// One wave alone issues the 32 x 32 shapes at the matrix units' rate, but the
// 16 x 16 ones at 60% of it; two waves of a SIMD reach it with either
// (measured, registers only: bf16 2.30 / 1.46 and 2.37 / 2.35 PFLOP/s, MXFP4
// 8.3 / 4.8 and 8.5 / 7.9).
#pragma once

#include "operators_internal.h"
#include "qmoe_device.h"

namespace qmoe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct RowUnit {
  int e, r0, M;   // expert, first row, rows (0: no such unit)
};

// Unit `b` of the rows cut into runs of at most BM rows of one expert: thread
// i counts the units of expert i, a scan over the 256 threads finds the expert
// that holds unit b.  Called by every thread, 256 or more; offsets are clamped to
// ascending values in [0, R], so no row outside the output is ever touched.
// `sh` is eight words of LDS, free again when it returns.
__device__ __forceinline__ RowUnit find_unit(const int32_t* offsets, int E, int R, int BM, int b, int* sh) {
  if (!offsets) {
    const int r0 = b * BM;
    return RowUnit{0, r0, max(0, min(BM, R - r0))};
  }
  int *wave_sum = sh, *hit = sh + 4;
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
  if (lane == 63 && wv < 4) wave_sum[wv] = inc;
  if (t == 0) hit[2] = 0;
  __syncthreads();
  if (wv < 4)
    for (int i = 0; i < wv; ++i) inc += wave_sum[i];
  if (wv < 4 && b >= inc - u && b < inc) {
    const int k = b - (inc - u);
    hit[0] = t;
    hit[1] = lo + k * BM;
    hit[2] = min(BM, cnt - k * BM);
  }
  __syncthreads();
  const RowUnit found{__builtin_amdgcn_readfirstlane(hit[0]), __builtin_amdgcn_readfirstlane(hit[1]),
                  __builtin_amdgcn_readfirstlane(hit[2])};
  __syncthreads();
  return found;
}

// Stores four consecutive outputs of one row, at whatever alignment its pitch
// leaves them (global stores need none on this target).
__device__ __forceinline__ void store4(const MatmulArgs& g, int row, int col, int cols, const f32x4& v) {
  const int64_t i = (int64_t)row * g.ldo + col;
  if (col + 4 <= cols) {
    if (g.out_bf16) {
      typedef __bf16 bf16x4 __attribute__((ext_vector_type(4), aligned(2)));
      *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(g.out) + i) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    } else {
      typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
      *reinterpret_cast<f32x4_any*>(static_cast<float*>(g.out) + i) = v;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + j < cols) {
      if (g.out_bf16) static_cast<__bf16*>(g.out)[i + j] = (__bf16)v[j];
      else static_cast<float*>(g.out)[i + j] = v[j];
    }
  }
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

// Items in order of expert, group of four output tiles, run of up to RUN rows, tile,
// so that what an XCD works on at a time shares rows as well as weights in its L2
// (MXFP4 rows, 28672 of 4 experts, 4096 x 2048: 231 us with single tiles, 226 with
// two, 214 with four, 216 with eight; bf16 rows 417, 400, 385, 395); a last run of
// at most half of RUN takes the narrow form, after the others.  Every thread calls
// it, 256 of them or more.
constexpr int kTileGroup = 4;
template <int RUN = kFatRows>
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
  const int rem = cnt & (RUN - 1);
  const int wide = cnt / RUN + (rem > RUN / 2);   // runs of the wide form
  const int u = wide * ntw + (rem > 0 && rem <= RUN / 2 ? ntn : 0);
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
    const bool full = k < wide * ntw;
    const int group = k / (max(wide, 1) * kTileGroup), tiles = min(kTileGroup, ntw - group * kTileGroup);
    const int j = k - group * wide * kTileGroup;
    const int run = full ? j / tiles : wide;
    hit[0] = t;
    hit[1] = lo + run * RUN;
    hit[2] = min(RUN, cnt - run * RUN);
    hit[3] = full ? group * kTileGroup + j % tiles : k - wide * ntw;
  }
  __syncthreads();
  it.e = __builtin_amdgcn_readfirstlane(hit[0]);
  it.r0 = __builtin_amdgcn_readfirstlane(hit[1]);
  it.M = __builtin_amdgcn_readfirstlane(hit[2]);
  it.tile = __builtin_amdgcn_readfirstlane(hit[3]);
  it.wide = it.M > RUN / 2;
  return true;
}

constexpr uint32_t kOutside = 0xff000000u;   // offset past every descriptor here, with room for a row's length

// 16 bytes per lane from buffer offset `off` into LDS at dst + 16 lane.
__device__ __forceinline__ void to_lds16(const rsrc_t& r, uint8_t* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
}

// A buffer descriptor as four words, for inline assembly.
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 raw_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// 16 bytes per lane from buffer offset `off` into LDS address dst + 16 lane, past
// the compiler's bookkeeping: it tells only a few such loads apart and waits
// for all of them before LDS reads that it cannot prove apart, where this
// pipeline counts its loads itself.  The load has no register result.
__device__ __forceinline__ void to_lds16_raw(const i32x4& r, uint32_t dst, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(off), "s"(r) : "m0");
}
// LDS by 32-bit address.
typedef __attribute__((address_space(3))) uint8_t lds8_t;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3), may_alias)) u32x4 lds_u32x4;
typedef __attribute__((address_space(3), may_alias)) u32x2 lds_u32x2;
__device__ __forceinline__ uint32_t lds_addr(const lds8_t* p) { return (uint32_t)(uintptr_t)p; }
__device__ __forceinline__ u32x4 lds_read16(const lds8_t* p) {
  return *reinterpret_cast<const lds_u32x4*>(p);
}
__device__ __forceinline__ uint32_t lds_read4(const lds8_t* p) {
  typedef __attribute__((address_space(3), may_alias)) uint32_t word;
  return *reinterpret_cast<const word*>(p);
}
__device__ __forceinline__ void lds_write16(lds8_t* p, u32x4 v) { *reinterpret_cast<lds_u32x4*>(p) = v; }
__device__ __forceinline__ void lds_write8(lds8_t* p, u32x2 v) { *reinterpret_cast<lds_u32x2*>(p) = v; }

// 16 scale bytes of a row starting at byte `off` of a descriptor whose base is
// 4-byte aligned.
struct ScaleWords {
  uint32_t w[5];
  __device__ __forceinline__ void load(const rsrc_t& r, uint32_t off) {
    uint32_t v[4];
    bload16(v, r, off & ~3u, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
    w[4] = __builtin_amdgcn_raw_buffer_load_b32(r, (off & ~3u) + 16u, 0, 0);
  }
  // keeps the first `valid` bytes, the others 0
  __device__ __forceinline__ u32x4 bytes(uint32_t off, int valid) const {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = __builtin_amdgcn_alignbyte(w[i + 1], w[i], off & 3u);
      const int left = valid - 4 * i;
      o[i] = left >= 4 ? x : left > 0 ? x & (0xffffffffu >> (32 - 8 * left)) : 0u;
    }
    return u32x4{o[0], o[1], o[2], o[3]};
  }
};

// Orders this wave's LDS accesses between lanes: the hardware keeps a wave's
// accesses in order, the compiler only each lane's.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Results leave through LDS: the lanes of a store from the accumulators hold 4
// outputs of as many rows, 16-byte requests, where the vector cache takes a
// line in one.  A wave lays its rows out at RB + 16 bytes each (rows 16 apart
// in the bank row, so that neither side of the exchange has conflicts) and
// writes them out RB bytes at a time, at whatever alignment the rows' pitch
// leaves them.  `out_cols` bounds the columns.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2), may_alias));
template <int RB>
__device__ __forceinline__ void store_rows(const MatmulArgs& g, const lds8_t* t, int rows, int row0, int col0, int out_cols) {
  constexpr int LPR = RB / 16, RPI = 64 / LPR;   // lanes per row, rows per instruction
  const int lane = threadIdx.x & 63, c = lane % LPR;
  const int es = g.out_bf16 ? 2 : 4, per = 16 / es;
  const int col = col0 + c * per;
  const bool vec = col + per <= out_cols;
  // whole lines need not stay in L2, which the operands need (MXFP4 rows, 28672 rows,
  // 4096 x 1024: 144 us with plain stores, 124 with these); parts of lines have to
  // meet there (bf16 rows, 28672 rows, 4088 x 32: 72 us, with these 117)
  const bool lines = ((reinterpret_cast<uintptr_t>(g.out) | (uintptr_t)(g.ldo * es)) & 127) == 0;
  uint8_t* o = static_cast<uint8_t*>(g.out) + ((int64_t)row0 * g.ldo + col) * es;
  wave_sync();
  if (lines && col0 + RB / es <= out_cols) {
    for (int r = lane / LPR; r < rows; r += RPI)
      __builtin_nontemporal_store(lds_read16(t + r * (RB + 16) + c * 16), reinterpret_cast<u32x4_any*>(o + (int64_t)r * g.ldo * es));
    wave_sync();
    return;
  }
  for (int r = lane / LPR; r < rows; r += RPI) {
    const u32x4 v = lds_read16(t + r * (RB + 16) + c * 16);
    uint8_t* p = o + (int64_t)r * g.ldo * es;
    if (vec) {
      *reinterpret_cast<u32x4_any*>(p) = v;
    } else if (g.out_bf16) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < out_cols) reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < out_cols) reinterpret_cast<uint32_t*>(p)[j] = v[j];
    }
  }
  wave_sync();   // the next results may take their place
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// s_waitcnt immediate: all but the n most recent vector memory ops, and every
// LDS read (gfx9 encoding: vmcnt in bits 3-0 and 15-14, lgkmcnt in 11-8).
__host__ __device__ constexpr int waitcnt_vm_lds(int n) { return (n & 15) | (7 << 4) | ((n >> 4) << 14); }

}  // namespace qmoe
