// Grouped products with both sides in MXFP4, for many rows.
//
// A work item is up to 256 rows times 256 outputs on one workgroup of four
// waves, one per SIMD with all 512 registers: 128 x 128 each (runs of up to 128
// rows: 64 outputs x 128 rows each).  A scaled MFMA takes 32 cycles for 4 KB of
// operands, so both sides come through LDS, where a wave tile of 128 x 128
// costs the CU 64 KB of reads per 1024 cycles of MFMAs, half of what LDS
// delivers.
//
// What bounds it is the vector cache, which keeps about 80 requests to L2 in
// flight per CU, whatever their size: with 128 inputs (64 bytes) of a row per
// stage, half a line per request, it delivered 17 bytes a cycle where the
// MFMAs ask for 32.  So a stage holds 256 inputs, a whole line per row, and
// LDS two stages.  Block kb + 1's operands for the first step are read, and
// block kb + 2 is requested, once every wave has block kb's last step in
// registers; the requests are spread over the following steps.
//
// 16384 tokens, 8 of 256 experts, 4096 x 6144: 1.97 to 2.13 ms on average from card
// to card, beside 0.05 for quantising the tokens, 3.1 to 3.3 PFLOP/s, MFMAs busy in 43
// % of the cycles.
//
// Scales: 16 blocks of a row at a time.  Where a row's bytes may start
// anywhere, a thread loads the five aligned words around them, shifts them into
// place, clears what lies past K and writes 16 bytes to LDS.
#include <algorithm>

#include "mxfp4_tile.h"

namespace qmoe {
namespace {

constexpr int kThreads4 = 256;
constexpr int kBlk4 = 256;    // inputs per stage

// LDS: two stages of each side, rows of 128 bytes, 16-byte chunk c of row r at
// c ^ (r / 2 mod 8); then two groups of scales of each side, 16 bytes per row.
constexpr int kLdsA = 0, kLdsW = 65536, kLdsAs = 131072, kLdsWs = kLdsAs + 8192, kLds4 = kLdsWs + 8192;
static_assert(4 * 128 * (256 + 16) <= kLds4, "the results fit");

// SL: K % 256 == 0.  Every stage is full, and 16 scales of a row are aligned
// words, which come by direct loads too.
template <bool SL, int RT, int WT, int CT>
__device__ __forceinline__ void tile4(const MatmulArgs& g, const FatItem& it, lds8_t* lds) {
  constexpr int NA = 8, NV = 16;   // direct loads per thread and stage: rows, both
  const int tid = threadIdx.x, lane = tid & 63, ln = lane & 31, lh = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv / WT, wt = wv % WT;
  const int nb = g.K / kMxBlock, nkb = (g.K + kBlk4 - 1) / kBlk4;
  const int n0 = it.tile * 256;

  const int64_t ldb = g.K / 2;
  const int64_t first = g.index ? 0 : it.r0;
  const i32x4 ar = raw_rsrc(static_cast<const uint8_t*>(g.a) + first * ldb, kOutside);
  const int64_t erow = (int64_t)it.e * g.N;
  const i32x4 wr = raw_rsrc(g.w_codes + erow * ldb, (uint32_t)g.N * (uint32_t)ldb);
  auto row_of = [&](int i) {   // row of `a` behind row i of the run, relative to the descriptor; -1: none
    return i < it.M ? (g.index ? source_row(g, it.r0 + i) : (int64_t)i) : (int64_t)-1;
  };
  const int chunk = (tid & 7) ^ ((tid >> 4) & 7);   // this thread's chunk of a row, the same in each load
  uint32_t aoff[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int64_t src = row_of(i * 32 + (tid >> 3));
    aoff[i] = src >= 0 ? (uint32_t)(src * ldb) + 16u * chunk : kOutside;
  }
  const uint32_t woff = (uint32_t)(n0 + (tid >> 3)) * (uint32_t)ldb + 16u * chunk;

  // scales: thread t carries row t of the weights' tile and row t of the run.
  // The descriptors start at the aligned word before the first byte and end
  // with the word of the last one.
  const uint8_t* sb[2] = {g.w_scale + erow * nb, g.a_scale + first * nb};
  const int srows[2] = {g.N, g.index ? g.a_rows : it.M};
  uint32_t soff[2];
  rsrc_t sr[2];
  i32x4 sr_raw[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(sb[j]) & 3);
    sr[j] = make_rsrc(sb[j] - mis, ((uint32_t)srows[j] * (uint32_t)nb + mis + 3u) & ~3u);
    sr_raw[j] = raw_rsrc(sb[j] - mis, ((uint32_t)srows[j] * (uint32_t)nb + mis + 3u) & ~3u);
    const int64_t row = j == 0 ? (int64_t)(n0 + tid) : row_of(tid);
    soff[j] = row >= 0 && row < srows[j] ? mis + (uint32_t)(row * nb) : kOutside;
  }

  ScaleWords sw[2];
  auto issue_s = [&](int grp) {
    if constexpr (SL) {
      to_lds16_raw(sr_raw[0], lds_addr(lds) + kLdsWs + (grp & 1) * 4096 + wv * 1024, soff[0] + 16u * (uint32_t)grp);
      to_lds16_raw(sr_raw[1], lds_addr(lds) + kLdsAs + (grp & 1) * 4096 + wv * 1024, soff[1] + 16u * (uint32_t)grp);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) sw[j].load(sr[j], soff[j] + 16u * (uint32_t)grp);
    }
  };
  auto write_s = [&](int grp) {
    if constexpr (SL) return;
    const int valid = nb - 16 * grp;
    lds_write16(lds + kLdsWs + (grp & 1) * 4096 + tid * 16, sw[0].bytes(soff[0], soff[0] < kOutside ? valid : 0));
    lds_write16(lds + kLdsAs + (grp & 1) * 4096 + tid * 16, sw[1].bytes(soff[1], soff[1] < kOutside ? valid : 0));
  };
  // load i < NV of block kb into the stage at byte p (0 or 32768) of each side
  auto issue = [&](uint32_t p, int kb, int i) {
    const bool past = !SL && kb * 8 + chunk >= nb;
    if (i < NA)
      to_lds16_raw(ar, lds_addr(lds) + kLdsA + p + (i * 4 + wv) * 1024, past ? kOutside : aoff[i % NA] + (uint32_t)kb * 128u);
    else
      to_lds16_raw(wr, lds_addr(lds) + kLdsW + p + ((i - NA) * 4 + wv) * 1024,
                   past ? kOutside : woff + (uint32_t)(i - NA) * 32u * (uint32_t)ldb + (uint32_t)kb * 128u);
  };

  f32x16 acc[RT][CT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[rt][c][i] = 0.0f;

  // operands of step t < 4 of a block, 64 inputs: chunk 2 t + lh of each row
  u32x4 W[2][RT], A[2][CT];
  uint32_t ws[2][RT], as[2][CT];
  // part i < 4 of the operands of step t of block kb, from the stage at p
  auto read = [&](uint32_t p, auto T, int kb, int i) {
    constexpr int t = decltype(T)::value, s = t & 1;
    const int at = ln * 128 + 16 * ((2 * t + lh) ^ ((ln >> 1) & 7));
    // scales of steps t and t + 1, from an even step on: bytes 0 and 2 of the word,
    // in the upper half of the wave bytes 1 and 3
    constexpr int m = t >> 1;
    const int grp = ((kb >> 1) & 1) * 4096 + (kb & 1) * 8 + 4 * m + ln * 16;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      if (rt == i) {
        W[s][rt] = lds_read16(lds + kLdsW + p + (wn * RT + rt) * 4096 + at);
        if constexpr (s == 0) ws[m][rt] = lds_read4(lds + kLdsWs + grp + (wn * RT + rt) * 512) >> (8 * lh);
      }
#pragma unroll
    for (int c = 0; c < CT; ++c)
      if (c == i) {
        A[s][c] = lds_read16(lds + kLdsA + p + (wt * CT + c) * 4096 + at);
        if constexpr (s == 0) as[m][c] = lds_read4(lds + kLdsAs + grp + (wt * CT + c) * 512) >> (8 * lh);
      }
  };
  auto handover = [&]() {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // Step t of block kb: in four parts, requests, the next step's reads (first)
  // and MFMAs.  Requests: half of block kb + 2 in step 3, into the stage that
  // its barrier freed, the other half of block kb + 1 in step 0, which leaves
  // two steps for the last of them to land.
  using I0 = std::integral_constant<int, 0>;
  auto block = [&](int kb) {
    const uint32_t p = (uint32_t)(kb & 1) * 32768u, q = p ^ 32768u;
    const int k1 = min(kb + 1, nkb - 1), k2 = min(kb + 2, nkb - 1);   // past the end: never read
    const int grp = (kb >> 1) + 1;
    static_for<4>([&](auto T) {
      constexpr int t = decltype(T)::value, s = t & 1;
      if constexpr (t == 3) handover();   // block kb is read, block kb + 1 has landed, in every wave
      if (t == 0 && (kb & 1) == 0) issue_s(grp);
      if (t == 2 && (kb & 1) == 0) write_s(grp);
      static_for<4>([&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (t == 3) {
          issue(p, k2, 2 * i);
          issue(p, k2, 2 * i + 1);
        } else if constexpr (t == 0) {
          issue(q, k1, 8 + 2 * i);
          issue(q, k1, 9 + 2 * i);
        }
        if constexpr (i < 2) {
#pragma unroll
          for (int j = 2 * i; j < 2 * i + 2; ++j) {
            if constexpr (t == 3) read(q, I0{}, kb + 1, j);
            else read(p, std::integral_constant<int, t + 1>{}, kb, j);
          }
        }
#pragma unroll
        for (int j = 0; j < RT * CT; ++j)
          if (j * 4 / (RT * CT) == i) {
            const int c = j / RT, rt = j % RT;
            const u32x4 w = W[s][rt], x = A[s][c];
            const i32x8 wv8 = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
            const i32x8 xv8 = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
            acc[rt][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv8, xv8, acc[rt][c], 4, 4, 2 * s, (int)ws[t >> 1][rt], 2 * s, (int)as[t >> 1][c]);
          }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  };
  issue_s(0);
#pragma unroll
  for (int i = 0; i < NV; ++i) issue(0u, 0, i);
#pragma unroll
  for (int i = 0; i < 8; ++i) issue(32768u, min(1, nkb - 1), i);
  write_s(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(8));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < 4; ++i) read(0u, I0{}, 0, i);
  for (int kb = 0; kb < nkb; ++kb) block(kb);
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
          lds_write8(t + (c * 32 + ln) * (RB + 16) + rt * 64 + 16 * q + 8 * lh,
                   u32x2{pack_bf16(acc[rt][c][4 * q], acc[rt][c][4 * q + 1]), pack_bf16(acc[rt][c][4 * q + 2], acc[rt][c][4 * q + 3])});
    store_rows<RB>(g, t, rows, row0, n0 + wn * RT * 32, g.N);
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
            lds_write16(t + (c * 32 + ln) * (RB + 16) + rt * 128 + 32 * q + 16 * lh, __builtin_bit_cast(u32x4, f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]}));
          }
      store_rows<RB>(g, t, rows, row0, n0 + wn * RT * 32 + h * (RT / 2) * 32, g.N);
    }
  }
}

template <bool SL>
__global__ void __launch_bounds__(kThreads4, 1) mx_matmul4_kernel(MatmulArgs g, int nt) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds4];
  FatItem it;
  if (!find_item(g.offsets, g.E, g.R, nt, nt, it)) return;
  lds8_t* lds = (lds8_t*)smem;
  if (it.wide) {
    if (it.M > 192) tile4<SL, 4, 2, 4>(g, it, lds);
    else tile4<SL, 4, 2, 3>(g, it, lds);
  } else {
    if (it.M > 96) tile4<SL, 2, 1, 4>(g, it, lds);
    else if (it.M > 64) tile4<SL, 2, 1, 3>(g, it, lds);
    else if (it.M > 32) tile4<SL, 2, 1, 2>(g, it, lds);
    else tile4<SL, 2, 1, 1>(g, it, lds);
  }
}

}  // namespace

hipError_t launch_mx_matmul4_large(const MatmulArgs& g, hipStream_t s) {
  const int nt = (g.N + 255) / 256;
  const dim3 grid((unsigned)(((long)g.R / kFatRows + std::min(g.E, g.R)) * nt));
  hipLaunchKernelGGL(g.K % kBlk4 == 0 ? mx_matmul4_kernel<true> : mx_matmul4_kernel<false>, grid, dim3(kThreads4), 0, s, g, nt);
  return hipGetLastError();
}

}  // namespace qmoe
