// Grouped products of bf16 rows and MXFP4 expert weights, for many rows.
//
// One workgroup of eight waves per CU; a work item is up to 256 rows of one
// expert times 256 outputs (waves 4 x 2), or up to 128 rows times 512 outputs
// (8 x 1): either way a wave holds 64 outputs x 128 rows in its accumulators,
// and 128 inputs cost the CU 256 KB of LDS reads for 4096 cycles of MFMAs on
// every SIMD.  The weights go from global memory straight into registers and
// become bf16 there, four conversions per eight codes, between the MFMAs; the
// rows of `a` go through LDS by direct loads.  128 inputs per stage, two
// stages: a K block's MFMAs take longer than the next block's loads.
//
// 4096 tokens, 8 of 256 experts, 4096 x 6144: 1.45 to 1.56 ms on average from card to
// card, 1.06 to 1.14 PFLOP/s (a library product of 16384^3 in bf16: 1.36), MFMAs busy
// in 57 % of the cycles; what is left is mostly an item's start and end.  32x32x16 MFMAs with half the LDS reads took
// 1.60 to 1.72 ms.
//
// The next block's requests are spread over the first half of a block: issued
// at once they stall every wave until the address units have taken them all
// (1.94 against 1.59 ms for gate and up of 256 experts over 4096 tokens).
#include <algorithm>

#include "mxfp4_tile.h"

namespace qmoe {
namespace {

constexpr int kBlk = 128;                        // inputs per stage
constexpr int kStage = kFatRows * kBlk * 2;      // 64 KB
constexpr int kMidRows = 64, kMidOut = 128, kMidThreads = 256;
constexpr int kMidStage = kMidRows * kBlk * 2;   // 16 KB

// A wave's 16-byte reads go in four groups, one of them lanes 0 to 3, 12 to 15 and
// 20 to 27 (two chunks, four apart, of eight rows each): with this they lie on
// distinct banks, while at chunk c ^ r they would meet in pairs.
__device__ __forceinline__ int turn(int r) { return (r & 15) ^ ((r << 1) & 8); }

struct LdsL {
  // stages: rows of 256 bytes, 16-byte chunk c of row r at c ^ turn(r)
  uint8_t *st0, *st1;
  uint8_t* ws;          // weight scales: two groups of 16 bytes per output
};
// the results take the place of the stages, four waves in each, half of a wave's rows at a time
static_assert(4 * 64 * (128 + 16) <= kStage, "half of the results fits");

// SL: the scales of 16 blocks of an output are 16 aligned bytes (K % 128 ==
// 0), which come into LDS one group ahead: a scale byte per lane costs the
// address units as much as 16 bytes of codes.  Otherwise lanes load bytes.
// NW waves, NW / WT x WT; a wave's tile is 16 RT outputs x 16 CT rows.
template <bool SL, int NW, int WT, int RT, int CT>
__device__ __forceinline__ void large_tile(const MatmulArgs& g, const FatItem& it, const LdsL& lds) {
  constexpr int WN = NW / WT, ROWS = 16 * CT * WT, THREADS = 64 * NW, WOUT = 16 * RT;
  constexpr int SLOTS = ROWS * 16, NA = (SLOTS + THREADS - 1) / THREADS;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % WN, wt = wv / WN;
  const int n0 = it.tile * (WOUT * WN);
  const int nb = g.K / kMxBlock, nkb = (g.K + kBlk - 1) / kBlk;

  // load i brings rows THREADS / 16 i + tid / 16, this thread always the same chunk of its row
  const int chunk = (tid & 15) ^ turn(tid >> 4);
  const int64_t ldb = g.lda * 2;
  const rsrc_t ar = make_rsrc(static_cast<const uint8_t*>(g.a) + (g.index ? 0 : (int64_t)it.r0 * ldb), kOutside);
  uint32_t aoff[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int row = i * (THREADS / 16) + (tid >> 4);
    const int64_t src = row < it.M ? (g.index ? source_row(g, it.r0 + row) : (int64_t)row) : (int64_t)-1;
    aoff[i] = src >= 0 ? (uint32_t)(src * ldb) + 16u * chunk : kOutside;
  }
  // weights: lane (lr, lq) takes block lq of row lr; rows past N lie past the descriptors
  const int64_t erow = (int64_t)it.e * g.N;
  const uint32_t wld = (uint32_t)(g.K / 2);
  const rsrc_t wr = make_rsrc(g.w_codes + erow * wld, (uint32_t)g.N * wld);
  const uint32_t woff = (uint32_t)(n0 + wn * WOUT + lr) * wld + 16u * lq;
  const rsrc_t sr = make_rsrc(g.w_scale + erow * nb, (uint32_t)g.N * (uint32_t)nb);
  const uint32_t soff = (uint32_t)(n0 + (SL ? wv * 64 + lane : wn * WOUT + lr)) * (uint32_t)nb + (SL ? 0u : (uint32_t)lq);

  uint32_t wq[2][RT][4], wsc[2][RT];
  auto issue_a = [&](auto P, int kb, int i) {
    if (i * THREADS + wv * 64 >= SLOTS) return;
    const bool past = !SL && kb * kBlk + chunk * 8 >= g.K;
    to_lds16(ar, (decltype(P)::value ? lds.st1 : lds.st0) + (i * THREADS + wv * 64) * 16,
             past ? kOutside : aoff[i] + (uint32_t)kb * (kBlk * 2));
  };
  auto issue_w = [&](auto P, int kb, int rt) {
    constexpr int p = decltype(P)::value;
    bload16(wq[p][rt], wr, woff + (uint32_t)rt * 16u * wld + (uint32_t)kb * 64u, 0);
    // blocks past K: the next row's scales, which may be NaN, times zeros
    if constexpr (!SL)
      wsc[p][rt] = __builtin_amdgcn_raw_buffer_load_b8(
          sr, kb * 4 + lq < nb ? soff + (uint32_t)rt * 16u * (uint32_t)nb + (uint32_t)kb * 4u : kOutside, 0, 0);
  };
  auto issue_s = [&](int kb) {   // the scales of block kb's group, if it starts one
    if constexpr (SL) {
      if (wv < WOUT * WN / 64 && (kb & 3) == 0)
        to_lds16(sr, lds.ws + ((kb >> 2) & 1) * 8192 + wv * 1024, soff + (uint32_t)kb * 4u);
    }
  };
  auto read_s = [&](auto P, int kb) {
    if constexpr (SL) {
      const uint8_t* b = lds.ws + ((kb >> 2) & 1) * 8192 + (wn * WOUT + lr) * 16 + (kb & 3) * 4 + lq;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) wsc[decltype(P)::value][rt] = b[rt * 256];
    }
  };

  f32x4 acc[RT][CT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[rt][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Sub-step j of a block: HB column tiles, from HB (j % SUB) on, of step j /
  // SUB, which takes word j / SUB of every lane's 32 inputs.
  constexpr int HB = CT < 2 ? 1 : 2, SUB = CT / HB, NSUB = 4 * SUB, IS = NSUB / 2;
  auto block = [&](auto P, int kb) {
    constexpr int p = decltype(P)::value;
    using Q = std::integral_constant<int, 1 - p>;
    const uint8_t* st = p ? lds.st1 : lds.st0;
    // block kb has landed, in every wave; nobody reads the other stage any more
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    read_s(P, kb);
    __builtin_amdgcn_sched_barrier(0);
    const int kn = min(kb + 1, nkb - 1);   // the last block is requested twice: no branch
    bf16x8 A[RT];
    uint4 B[2][HB];
    auto read_b = [&](int j) {
#pragma unroll
      for (int c = 0; c < HB; ++c)
        B[j & 1][c] = *reinterpret_cast<const uint4*>(st + ((wt * CT + HB * (j % SUB) + c) * 16 + lr) * 256 + 16 * ((4 * lq + j / SUB) ^ turn(lr)));
    };
    read_b(0);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) A[rt] = bf16_of(wq[p][rt][0], __uint_as_float(wsc[p][rt] << 23));
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
          acc[rt][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[rt], __builtin_bit_cast(bf16x8, B[j & 1][c]), acc[rt][ct], 0, 0, 0);
        }
        // the next step's operand, in the registers that these MFMAs are done with
        if (j % SUB == SUB - 1 && s < 3) A[rt] = bf16_of(wq[p][rt][s + 1], __uint_as_float(wsc[p][rt] << 23));
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
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  issue_s(0);
#pragma unroll
  for (int i = 0; i < NA; ++i) issue_a(I0{}, 0, i);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) issue_w(I0{}, 0, rt);
  for (int kb = 0; kb < nkb; kb += 2) {
    block(I0{}, kb);
    if (kb + 1 < nkb) block(I1{}, kb + 1);
  }

  // every wave's reads and loads are done: LDS takes the results
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  constexpr int HC = (CT + 1) / 2, RB = 32 * RT;   // column tiles at a time, bytes of a row
  lds8_t* t = (lds8_t*)(wv < NW / 2 ? lds.st0 : lds.st1) + (wv % (NW / 2)) * (HC * 16 * (RB + 16));
#pragma unroll
  for (int c0 = 0; c0 < CT; c0 += HC) {
    const int row0 = (wt * CT + c0) * 16, rows = min(it.M - row0, HC * 16);
    if (g.out_bf16) {
#pragma unroll
      for (int c = 0; c < HC; ++c)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          if (c0 + c < CT)
            lds_write8(t + (c * 16 + lr) * (RB + 16) + rt * 32 + lq * 8,
                       u32x2{pack_bf16(acc[rt][c0 + c][0], acc[rt][c0 + c][1]), pack_bf16(acc[rt][c0 + c][2], acc[rt][c0 + c][3])});
      store_rows<RB>(g, t, rows, it.r0 + row0, n0 + wn * WOUT, g.N);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {   // half of the outputs
#pragma unroll
        for (int c = 0; c < HC; ++c)
#pragma unroll
          for (int rt = 0; rt < RT / 2; ++rt)
            if (c0 + c < CT) lds_write16(t + (c * 16 + lr) * (RB + 16) + rt * 64 + lq * 16, __builtin_bit_cast(u32x4, acc[RT / 2 * h + rt][c0 + c]));
        store_rows<RB>(g, t, rows, it.r0 + row0, n0 + wn * WOUT + h * (WOUT / 2), g.N);
      }
    }
  }
}

template <bool SL>
__global__ void __launch_bounds__(kFatThreads, 2) mx_matmul_large_kernel(MatmulArgs g, int ntw, int ntn) {
  __shared__ __attribute__((aligned(16))) uint8_t st0[kStage], st1[kStage];
  __shared__ __attribute__((aligned(16))) uint8_t ws[SL ? 2 * 512 * 16 : 16];
  FatItem it;
  if (!find_item(g.offsets, g.E, g.R, ntw, ntn, it)) return;
  const LdsL lds{st0, st1, ws};
  if (it.wide) {
    if (it.M > 192) large_tile<SL, 8, 2, 4, 8>(g, it, lds);
    else large_tile<SL, 8, 2, 4, 6>(g, it, lds);
  } else {
    if (it.M > 96) large_tile<SL, 8, 1, 4, 8>(g, it, lds);
    else if (it.M > 64) large_tile<SL, 8, 1, 4, 6>(g, it, lds);
    else if (it.M > 32) large_tile<SL, 8, 1, 4, 4>(g, it, lds);
    else if (it.M > 16) large_tile<SL, 8, 1, 4, 2>(g, it, lds);
    else large_tile<SL, 8, 1, 4, 1>(g, it, lds);
  }
}

// Products too small to give every CU an item of 256 x 256: 128 outputs x 64
// rows on four waves, three workgroups per CU.  Twice the LDS reads per MFMA,
// but eight times the items: 512 rows, 4096 x 4096 in 29 us (600 TFLOP/s), where
// units of 16 rows take 87, and 8 experts, 4096 rows, 512 x 4096 in 32 instead
// of 100.  Bound by the latency of the next block's loads, where a CU has one
// workgroup, else by the LDS.
template <bool SL>
__global__ void __launch_bounds__(kMidThreads, 2) mx_matmul_mid_kernel(MatmulArgs g, int nt) {
  __shared__ __attribute__((aligned(16))) uint8_t st0[kMidStage], st1[kMidStage];
  __shared__ __attribute__((aligned(16))) uint8_t ws[SL ? 8192 + kMidOut * 16 : 16];
  FatItem it;
  if (!find_item<kMidRows>(g.offsets, g.E, g.R, nt, nt, it)) return;
  const LdsL lds{st0, st1, ws};
  if (it.M > 32) large_tile<SL, 4, 1, 2, 4>(g, it, lds);
  else if (it.M > 16) large_tile<SL, 4, 1, 2, 2>(g, it, lds);
  else large_tile<SL, 4, 1, 2, 1>(g, it, lds);
}

}  // namespace

hipError_t launch_mx_matmul_large(const MatmulArgs& g, hipStream_t s) {
  const int ntw = (g.N + 255) / 256, ntn = (g.N + 511) / 512;
  const dim3 grid((unsigned)(((long)g.R / kFatRows + std::min(g.E, g.R)) * ntw));
  hipLaunchKernelGGL(g.K % kBlk == 0 ? mx_matmul_large_kernel<true> : mx_matmul_large_kernel<false>, grid,
                     dim3(kFatThreads), 0, s, g, ntw, ntn);
  return hipGetLastError();
}

hipError_t launch_mx_matmul_mid(const MatmulArgs& g, hipStream_t s) {
  const int nt = (g.N + kMidOut - 1) / kMidOut;
  const dim3 grid((unsigned)(((long)g.R / kMidRows + std::min(g.E, g.R)) * nt));
  hipLaunchKernelGGL(g.K % kBlk == 0 ? mx_matmul_mid_kernel<true> : mx_matmul_mid_kernel<false>, grid,
                     dim3(kMidThreads), 0, s, g, nt);
  return hipGetLastError();
}

}  // namespace qmoe
