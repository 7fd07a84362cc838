// Grouped products over MXFP4 expert weights for many rows.
#include <algorithm>

#include "mxfp4_tile.h"

namespace qmoe {
namespace {

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

hipError_t launch_mx_matmul_large(const MatmulArgs& g, bool a_mxfp4, hipStream_t s) {
  const int ntw = (g.N + 255) / 256, ntn = (g.N + 511) / 512;
  const dim3 grid((unsigned)(((long)g.R / kFatRows + std::min(g.E, g.R)) * ntw));
  const bool sl = g.K % 128 == 0;
  auto* k = a_mxfp4 ? (sl ? mx_matmul_fat_kernel<true, true> : mx_matmul_fat_kernel<true, false>)
                    : (sl ? mx_matmul_fat_kernel<false, true> : mx_matmul_fat_kernel<false, false>);
  hipLaunchKernelGGL(k, grid, dim3(kFatThreads), 0, s, g, ntw, ntn);
  return hipGetLastError();
}

}  // namespace qmoe
