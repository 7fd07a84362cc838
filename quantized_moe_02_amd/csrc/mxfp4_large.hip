// Grouped products of bf16 rows and MXFP4 expert weights, for many rows.
//
// One workgroup of eight waves per CU; a work item is up to 256 rows of one
// expert times 256 outputs (waves 4 x 2), or up to 128 rows times 512 outputs
// (8 x 1): either way a wave holds 64 outputs x 128 rows in its accumulators,
// and 128 inputs cost the CU 256 KB of LDS reads for 8192 cycles of MFMAs per
// pair of waves.  The weights go from global memory straight into registers
// and become bf16 there, four conversions per eight codes, in the shadow of
// the MFMAs; the rows of `a` go through LDS by direct loads.  128 inputs per
// stage, two stages: a K block's MFMAs take longer than the next block's loads.
//
// The hand-over between stages comes before a block's last step, whose
// operands are in registers by then, so that the first reads of the next block
// and its first conversion run beside those MFMAs.
#include <algorithm>

#include "mxfp4_tile.h"

namespace qmoe {
namespace {

constexpr int kBlk = 128;                        // inputs per stage
constexpr int kStage = kFatRows * kBlk * 2;      // 64 KB

// LDS: two stages, rows of 256 bytes, 16-byte chunk c of row r at c ^ (r mod
// 16); then two groups of weight scales, 16 bytes per output.
constexpr int kLdsS = 2 * kStage, kLds = kLdsS + 2 * 512 * 16;
static_assert(8 * 128 * (128 + 16) <= kLds, "the results fit");

// SL: K % 128 == 0.  Every stage is full, and 16 scales of an output are
// aligned words, which come into LDS by direct loads; otherwise they pass
// through registers, which shift them into place.
template <bool SL, int WT, int CT>
__device__ __forceinline__ void large_tile(const MatmulArgs& g, const FatItem& it, lds8_t* lds) {
  constexpr int WN = 8 / WT, RT = 2, ROWS = 32 * CT * WT, NA = ROWS * 16 / kFatThreads;
  const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, lh = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % WN, wt = wv / WN;
  const int n0 = it.tile * (64 * WN);
  const int nb = g.K / kMxBlock, nkb = (g.K + kBlk - 1) / kBlk;

  // rows of `a`: load i brings row i * 32 + tid / 16, this thread always the same chunk of it
  const int64_t ldb = g.lda * 2;
  const i32x4 ar = raw_rsrc(static_cast<const uint8_t*>(g.a) + (g.index ? 0 : (int64_t)it.r0 * ldb), kOutside);
  const int chunk = (tid & 15) ^ ((tid >> 4) & 15);
  uint32_t aoff[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int row = i * 32 + (tid >> 4);
    const int64_t src = row < it.M ? (g.index ? source_row(g, it.r0 + row) : (int64_t)row) : (int64_t)-1;
    aoff[i] = src >= 0 ? (uint32_t)(src * ldb) + 16u * chunk : kOutside;
  }
  // weights: rows past N lie past the descriptors
  const int64_t erow = (int64_t)it.e * g.N;
  const rsrc_t wr = make_rsrc(g.w_codes + erow * (g.K / 2), (uint32_t)g.N * (uint32_t)(g.K / 2));
  const uint32_t woff = (uint32_t)(n0 + wn * 64 + ln) * (uint32_t)(g.K / 2) + 16u * lh;
  // scales: thread t < 64 WN carries those of output n0 + t
  const uint8_t* sbase = g.w_scale + erow * nb;
  const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(sbase) & 3);
  const i32x4 sr_raw = raw_rsrc(sbase - mis, ((uint32_t)g.N * (uint32_t)nb + mis + 3u) & ~3u);
  const rsrc_t sr = make_rsrc(sbase - mis, ((uint32_t)g.N * (uint32_t)nb + mis + 3u) & ~3u);
  const uint32_t soff = n0 + tid < g.N ? mis + (uint32_t)(n0 + tid) * (uint32_t)nb : kOutside;

  ScaleWords sw;
  auto issue_s = [&](int grp) {
    if (wv >= WN) return;
    if constexpr (SL) to_lds16_raw(sr_raw, lds_addr(lds) + kLdsS + (grp & 1) * 8192 + wv * 1024, soff + 16u * (uint32_t)grp);
    else sw.load(sr, soff + 16u * (uint32_t)grp);
  };
  auto write_s = [&](int grp) {
    if constexpr (!SL) {
      if (wv < WN)
        *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(lds + kLdsS + (grp & 1) * 8192 + tid * 16) =
            sw.bytes(soff, soff < kOutside ? nb - 16 * grp : 0);
    }
  };
  uint32_t wq[2][RT][2][4];   // chunk 2 c + lh of the block, c = 0, 1
  uint32_t sc[2][RT][2];
  auto issue_a = [&](auto P, int kb, int i) {
    constexpr int p = decltype(P)::value;
    const bool past = !SL && kb * kBlk + chunk * 8 >= g.K;
    to_lds16_raw(ar, lds_addr(lds) + p * kStage + (i * kFatThreads + wv * 64) * 16,
             past ? kOutside : aoff[i] + (uint32_t)kb * (kBlk * 2));
  };
  auto issue_w = [&](auto P, int kb, int i) {   // i < 4
    constexpr int p = decltype(P)::value;
    bload16(wq[p][i >> 1][i & 1], wr, woff + (uint32_t)(i >> 1) * 32u * (uint32_t)(g.K / 2) + (uint32_t)kb * 64u + 32u * (i & 1), 0);
  };
  auto read_s = [&](auto P, int kb) {
    constexpr int p = decltype(P)::value;
    const lds8_t* b = lds + kLdsS + ((kb >> 2) & 1) * 8192 + (wn * 64 + ln) * 16 + (kb & 3) * 4 + lh;
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[p][i >> 1][i & 1] = b[(i >> 1) * 512 + 2 * (i & 1)];
  };

  f32x16 acc[RT][CT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[rt][c][i] = 0.0f;

  // step j < 8 of a block: word j % 4 of chunk 2 (j / 4) + lh, eight inputs a lane
  bf16x8 A[2][RT], B[2][CT];
  auto read_b = [&](auto P, int j) {
    const lds8_t* st = lds + decltype(P)::value * kStage;
    const int c = (2 * (j >> 2) + lh) * 4 + (j & 3);
#pragma unroll
    for (int t = 0; t < CT; ++t)
      B[j & 1][t] = __builtin_bit_cast(bf16x8, lds_read16(st + ((wt * CT + t) * 32 + ln) * 256 + 16 * (c ^ (ln & 15))));
  };
  auto convert = [&](auto P, int j) {
    constexpr int p = decltype(P)::value;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      A[j & 1][rt] = bf16_of(wq[p][rt][j >> 2][j & 3], __uint_as_float(sc[p][rt][j >> 2] << 23));
  };
  auto block = [&](auto P, int kb) {
    constexpr int p = decltype(P)::value;
    using Q = std::integral_constant<int, 1 - p>;
    const int kn = min(kb + 1, nkb - 1);   // past the end: the last block again, never used
    const int grp = (kb >> 2) + 1;
    if ((kb & 3) == 0) issue_s(grp);
    if ((kb & 3) == 2) write_s(grp);
    static_for<8>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (j < 7) {
        read_b(P, j + 1);
      } else {
        // this wave has read block kb and its loads of block kb + 1 have
        // landed; past the barrier both hold for every wave
        __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(0));
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        read_s(Q{}, kb + 1);
        read_b(Q{}, 0);
      }
      if constexpr (j < 4) {
#pragma unroll
        for (int i = 0; i < NA; ++i)
          if (i % 4 == j) issue_a(Q{}, kn, i);
        issue_w(Q{}, kn, j);
      }
      if constexpr (j < 7) convert(P, j + 1);
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          acc[rt][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A[j & 1][rt], B[j & 1][t], acc[rt][t], 0, 0, 0);
      if constexpr (j == 7) convert(Q{}, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  issue_s(0);
#pragma unroll
  for (int i = 0; i < NA; ++i) issue_a(std::integral_constant<int, 0>{}, 0, i);
#pragma unroll
  for (int i = 0; i < 4; ++i) issue_w(std::integral_constant<int, 0>{}, 0, i);
  write_s(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(0));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  read_s(std::integral_constant<int, 0>{}, 0);
  read_b(std::integral_constant<int, 0>{}, 0);
  convert(std::integral_constant<int, 0>{}, 0);
  for (int kb = 0; kb < nkb; kb += 2) {
    block(std::integral_constant<int, 0>{}, kb);
    if (kb + 1 < nkb) block(std::integral_constant<int, 1>{}, kb + 1);
  }

  // every wave's reads and loads are done: LDS takes the results
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  lds8_t* t = lds + wv * (CT * 32 * (RT * 64 + 16));
  const int row0 = it.r0 + wt * CT * 32, rows = min(it.M - wt * CT * 32, CT * 32);
  if (g.out_bf16) {
    constexpr int RB = RT * 64;
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(t + (c * 32 + ln) * (RB + 16) + rt * 64 + 16 * q + 8 * lh) =
              u32x2{pack_bf16(acc[rt][c][4 * q], acc[rt][c][4 * q + 1]), pack_bf16(acc[rt][c][4 * q + 2], acc[rt][c][4 * q + 3])};
    store_rows<RB>(g, t, rows, row0, n0 + wn * 64, g.N);
  } else {
    // half of the outputs at a time
    constexpr int RB = RT * 64;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int rt = 0; rt < RT / 2; ++rt)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16& v = acc[h * (RT / 2) + rt][c];
            *reinterpret_cast<__attribute__((address_space(3))) f32x4*>(t + (c * 32 + ln) * (RB + 16) + rt * 128 + 32 * q + 16 * lh) =
                f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          }
      store_rows<RB>(g, t, rows, row0, n0 + wn * 64 + h * (RT / 2) * 32, g.N);
    }
  }
}

template <bool SL>
__global__ void __launch_bounds__(kFatThreads, 2) mx_matmul_large_kernel(MatmulArgs g, int ntw, int ntn) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  FatItem it;
  if (!find_item(g.offsets, g.E, g.R, ntw, ntn, it)) return;
  lds8_t* lds = (lds8_t*)smem;
  if (it.wide) {
    if (it.M > 192) large_tile<SL, 2, 4>(g, it, lds);
    else large_tile<SL, 2, 3>(g, it, lds);
  } else {
    if (it.M > 96) large_tile<SL, 1, 4>(g, it, lds);
    else if (it.M > 64) large_tile<SL, 1, 3>(g, it, lds);
    else if (it.M > 32) large_tile<SL, 1, 2>(g, it, lds);
    else large_tile<SL, 1, 1>(g, it, lds);
  }
}

}  // namespace

hipError_t launch_mx_matmul_large(const MatmulArgs& g, hipStream_t s) {
  const int ntw = (g.N + 255) / 256, ntn = (g.N + 511) / 512;
  const dim3 grid((unsigned)(((long)g.R / kFatRows + std::min(g.E, g.R)) * ntw));
  hipLaunchKernelGGL(g.K % kBlk == 0 ? mx_matmul_large_kernel<true> : mx_matmul_large_kernel<false>, grid,
                     dim3(kFatThreads), 0, s, g, ntw, ntn);
  return hipGetLastError();
}

}  // namespace qmoe
