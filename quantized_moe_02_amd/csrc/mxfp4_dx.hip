// Gradient of the grouped products with respect to their rows, for many rows:
// dx[r][i] = sum_j dy[r][j] W[j][i].
//
// The sum runs over the weights' rows, while their codes are packed along the
// columns, and the matrix units want eight consecutive terms of the sum per
// lane.  So a lane takes one word of codes (eight columns) from each of eight
// rows j: the conversion turns byte t of a word into bf16 columns 2t and 2t + 1
// of its row, with the row's scale, and two byte permutes per row pair regroup
// them into the operands of row tiles 2t and 2t + 1.  Lane (lr, lq) thereby
// feeds column 8 lr + tile of a 128-column strip, and holds, of the result,
// the 32 consecutive columns 32 lq .. 32 lq + 31 of row lr of each column tile.
//
// Eight waves per CU, each 128 columns x 64 rows: 2 x 4 waves for runs of up to
// 256 rows, 4 x 2 for up to 128.  dy and the codes come into LDS by direct
// loads, 64 terms of the sum per stage, three stages: block kb + 2 is requested
// while block kb is multiplied.  The scales (one byte per row j and 32 columns)
// go through registers into LDS, transposed, so that a lane reads the eight it
// needs at once.
//
// 4096 tokens, 8 of 256 experts, 4096 x 6144: 1.59 to 1.72 ms on average from card to
// card, 0.96 to 1.04 PFLOP/s, MFMAs busy in 51 % of the cycles, with three other vector
// instructions to each.
#include <algorithm>

#include "mxfp4_tile.h"

namespace qmoe {
namespace {

constexpr int kDxTerms = 64;   // terms of the sum per stage
constexpr int kMidRows = 64;

struct DxLds {
  uint8_t *dy[3], *cd[3], *sc[3];
};

template <int NW, int WT, int CT>
__device__ __forceinline__ void dx_tile(const MatmulArgs& g, const FatItem& it, const DxLds& lds) {
  constexpr int WN = NW / WT, ROWS = 16 * CT * WT, THREADS = 64 * NW;
  constexpr int CB = 64 * WN;              // bytes of codes per weight row of the tile
  constexpr int SB = 4 * WN;               // scales per weight row of the tile
  constexpr int DSLOTS = ROWS * 8, NA = (DSLOTS + THREADS - 1) / THREADS;
  constexpr int NC = kDxTerms * CB / 16 / THREADS, NV = NA + NC;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % WN, wt = wv / WN;
  const int k0 = it.tile * (128 * WN);
  const int nb = g.K / kMxBlock, nkb = (g.N + kDxTerms - 1) / kDxTerms;

  // Every wave issues the same NV loads per block, which the waits count on;
  // slots past the tile's rows lie in the stage too.
  static_assert(NA * THREADS * 16 <= NW * 4096 && (NW == 8 || WT == 2), "a stage holds every slot");
  // dy: rows of 128 bytes, 16-byte chunk c of row r at c ^ (r / 2 mod 8)
  const uint8_t* abase = static_cast<const uint8_t*>(g.a) + (int64_t)it.r0 * g.lda * 2;
  const rsrc_t ar = make_rsrc(abase, kOutside);
  uint32_t aoff[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int slot = i * THREADS + tid, row = slot >> 3, c = (slot & 7) ^ ((row >> 1) & 7);
    aoff[i] = row < it.M ? (uint32_t)((int64_t)row * g.lda * 2) + 16u * c : kOutside;
  }
  const int ac = (tid & 7) ^ ((tid >> 4) & 7);   // this thread's chunk, the same for each load
  // codes: the words that the four lq of a read touch (rows 8 apart) on
  // distinct banks.  Rows of 256 bytes: 64-byte unit u at u ^ (j / 8 mod 4);
  // of 128 bytes: rows j and j ^ 1 exchanged by j / 16, unit u at u ^ (j / 8 mod 2)
  auto code_at = [](int j, int u) {   // byte offset of unit u of row j
    return WN == 4 ? j * 256 + ((u ^ (j >> 3)) & 3) * 64 : (j ^ ((j >> 4) & 1)) * 128 + ((u ^ (j >> 3)) & 1) * 64;
  };
  const int64_t erow = (int64_t)it.e * g.N;
  const rsrc_t wr = make_rsrc(g.w_codes + erow * (g.K / 2), (uint32_t)g.N * (uint32_t)(g.K / 2));
  uint32_t coff[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int slot = i * THREADS + tid;
    const int jr = slot / (CB / 16), p = slot % (CB / 16);       // row and chunk in LDS
    const int j = WN == 4 ? jr : jr ^ ((jr >> 4) & 1);
    const int u = WN == 4 ? ((p >> 2) ^ (j >> 3)) & 3 : ((p >> 2) ^ (j >> 3)) & 1;
    coff[i] = (uint32_t)j * (uint32_t)(g.K / 2) + (uint32_t)k0 / 2 + (uint32_t)(u * 64 + (p & 3) * 16);
  }
  // scales: lane j of wave 0 carries row j's SB bytes, from the aligned word
  // before them on
  const uint8_t* sbase = g.w_scale + erow * nb;
  const uint32_t smis = (uint32_t)(reinterpret_cast<uintptr_t>(sbase) & 3);
  const rsrc_t sr = make_rsrc(sbase - smis, ((uint32_t)g.N * (uint32_t)nb + smis + 3u) & ~3u);
  const uint32_t soff = smis + (uint32_t)lane * (uint32_t)nb + (uint32_t)k0 / 32;
  uint32_t sw[SB / 4 + 1];

  auto issue_s = [&](int kb) {
    const uint32_t o = (soff + (uint32_t)kb * (kDxTerms * (uint32_t)nb)) & ~3u;
#pragma unroll
    for (int i = 0; i <= SB / 4; ++i) sw[i] = __builtin_amdgcn_raw_buffer_load_b32(sr, o + 4u * i, 0, 0);
  };
  auto write_s = [&](auto P, int kb) {
    const uint32_t sh = (soff + (uint32_t)kb * (kDxTerms * (uint32_t)nb)) & 3u;
    uint8_t* d = lds.sc[decltype(P)::value] + lane;
#pragma unroll
    for (int i = 0; i < SB / 4; ++i) {
      // rows past N: zero codes times a scale that must not be NaN
      const uint32_t w = kb * kDxTerms + lane < g.N ? __builtin_amdgcn_alignbyte(sw[i + 1], sw[i], sh) : 0u;
#pragma unroll
      for (int b = 0; b < 4; ++b) d[(4 * i + b) * kDxTerms] = (uint8_t)(w >> (8 * b));
    }
  };
  auto issue_a = [&](auto P, int kb, int i) {
    const uint32_t off = kb * kDxTerms + ac * 8 >= g.N ? kOutside : aoff[i] + (uint32_t)kb * (kDxTerms * 2);
    to_lds16(ar, lds.dy[decltype(P)::value] + (i * THREADS + wv * 64) * 16, off);
  };
  auto issue_c = [&](auto P, int kb, int i) {
    to_lds16(wr, lds.cd[decltype(P)::value] + (i * THREADS + wv * 64) * 16,
             coff[i] + (uint32_t)kb * (kDxTerms * (uint32_t)(g.K / 2)));
  };

  f32x4 acc[8][CT];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  // operands of one step of 32 terms
  uint32_t cw[2][8];
  uint2 ss[2];
  bf16x8 B[2][CT];
  auto read_step = [&](auto P, int s) {
    constexpr int p = decltype(P)::value;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int row = (wt * CT + c) * 16 + lr;
      B[s][c] = *reinterpret_cast<const bf16x8*>(lds.dy[p] + row * 128 + 16 * ((4 * s + lq) ^ ((lr >> 1) & 7)));
    }
    ss[s] = *reinterpret_cast<const uint2*>(lds.sc[p] + (wn * 4 + (lr >> 2)) * kDxTerms + 32 * s + 8 * lq);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      cw[s][j] = *reinterpret_cast<const uint32_t*>(lds.cd[p] + code_at(32 * s + 8 * lq + j, wn) + 4 * lr);
  };
  auto multiply = [&](int s) {
    // the conversion takes the exponent field of its scale operand and no other bit
    float sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = j < 4 ? ss[s].x : ss[s].y;
      sc[j] = __uint_as_float((j & 3) == 3 ? w >> 1 : w << (23 - 8 * (j & 3)));
    }
    static_for<4>([&](auto T) {
      constexpr int t = decltype(T)::value;
      union {
        uint32_t u[4];
        bf16x8 v;
      } lo, hi;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t a = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[s][2 * m], sc[2 * m], t));
        const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cw[s][2 * m + 1], sc[2 * m + 1], t));
        lo.u[m] = __builtin_amdgcn_perm(b, a, 0x05040100u);
        hi.u[m] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      }
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        acc[2 * t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo.v, B[s][c], acc[2 * t][c], 0, 0, 0);
        acc[2 * t + 1][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi.v, B[s][c], acc[2 * t + 1][c], 0, 0, 0);
      }
    });
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  auto block = [&](auto P, int kb) {
    constexpr int p = decltype(P)::value;
    using N1 = std::integral_constant<int, (p + 1) % 3>;
    using N2 = std::integral_constant<int, (p + 2) % 3>;
    const int k2 = min(kb + 2, nkb - 1);   // past the end: the last block again, never read
    if (wv == 0) {
      write_s(N1{}, min(kb + 1, nkb - 1));
      issue_s(k2);
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) issue_a(N2{}, k2, i);
#pragma unroll
    for (int i = 0; i < NC; ++i) issue_c(N2{}, k2, i);
    read_step(P, 1);
    multiply(0);
    // this wave's reads of block kb and its loads of block kb + 1 are done;
    // after the barrier that holds for every wave
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(NV));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    read_step(N1{}, 0);
    multiply(1);
  };
  if (wv == 0) {
    issue_s(0);
    write_s(I0{}, 0);
    issue_s(min(1, nkb - 1));
  }
#pragma unroll
  for (int i = 0; i < NA; ++i) issue_a(I0{}, 0, i);
#pragma unroll
  for (int i = 0; i < NC; ++i) issue_c(I0{}, 0, i);
#pragma unroll
  for (int i = 0; i < NA; ++i) issue_a(I1{}, min(1, nkb - 1), i);
#pragma unroll
  for (int i = 0; i < NC; ++i) issue_c(I1{}, min(1, nkb - 1), i);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(NV));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  read_step(I0{}, 0);
  for (int kb = 0; kb < nkb; kb += 3)
    static_for<3>([&](auto J) {
      if (kb + decltype(J)::value < nkb) block(J, kb + decltype(J)::value);
    });
  // every wave's reads and loads are done: LDS takes the results, a wave's
  // 16 rows x 128 columns at a time
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  lds8_t* t;
  if constexpr (NW == 8) t = (lds8_t*)(wv < 4 ? lds.dy[0] : lds.dy[1]) + (wv & 3) * (16 * (256 + 16));
  else t = (lds8_t*)(wv < 1 ? lds.dy[0] : wv < 2 ? lds.dy[1] : wv < 3 ? lds.dy[2] : lds.cd[0]);
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int row0 = (wt * CT + c) * 16, rows = min(it.M - row0, 16);
    if (g.out_bf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        lds_write16(t + lr * 272 + lq * 64 + i * 16,
                    u32x4{pack_bf16(acc[0][c][i], acc[1][c][i]), pack_bf16(acc[2][c][i], acc[3][c][i]),
                          pack_bf16(acc[4][c][i], acc[5][c][i]), pack_bf16(acc[6][c][i], acc[7][c][i])});
      store_rows<256>(g, t, rows, it.r0 + row0, k0 + wn * 128, g.K);
    } else {
      // 64 columns at a time: lanes lq 0 and 1, then 2 and 3
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if ((lq >> 1) == h) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lds_write16(t + lr * 272 + (lq & 1) * 128 + i * 32,
                        __builtin_bit_cast(u32x4, f32x4{acc[0][c][i], acc[1][c][i], acc[2][c][i], acc[3][c][i]}));
            lds_write16(t + lr * 272 + (lq & 1) * 128 + i * 32 + 16,
                        __builtin_bit_cast(u32x4, f32x4{acc[4][c][i], acc[5][c][i], acc[6][c][i], acc[7][c][i]}));
          }
        }
        store_rows<256>(g, t, rows, it.r0 + row0, k0 + wn * 128 + h * 64, g.K);
      }
    }
  }
}

__global__ void __launch_bounds__(kFatThreads, 2) mx_matmul_dx_fat_kernel(MatmulArgs g, int ntw, int ntn) {
  __shared__ __attribute__((aligned(16))) uint8_t dy0[32768], dy1[32768], dy2[32768];
  __shared__ __attribute__((aligned(16))) uint8_t cd0[16384], cd1[16384], cd2[16384];
  __shared__ __attribute__((aligned(16))) uint8_t sc0[1024], sc1[1024], sc2[1024];
  FatItem it;
  if (!find_item(g.offsets, g.E, g.R, ntw, ntn, it)) return;
  const DxLds lds{{dy0, dy1, dy2}, {cd0, cd1, cd2}, {sc0, sc1, sc2}};
  if (it.wide) {
    if (it.M > 192) dx_tile<8, 4, 4>(g, it, lds);
    else dx_tile<8, 4, 3>(g, it, lds);
  } else {
    if (it.M > 96) dx_tile<8, 2, 4>(g, it, lds);
    else if (it.M > 64) dx_tile<8, 2, 3>(g, it, lds);
    else if (it.M > 32) dx_tile<8, 2, 2>(g, it, lds);
    else dx_tile<8, 2, 1>(g, it, lds);
  }
}

// Results too few to give every CU an item of 256 x 256: 256 columns x 64 rows
// on four waves, three workgroups per CU.  8 experts, 4096 rows, 512 x 4096: 32
// us, in units of 16 rows 70, in items of 256 x 256 40.  A wave alone on its SIMD
// has an instruction of its conversions issued every 9 cycles, two together one
// every 5: a workgroup alone on its CU takes 0.78 us per 64 terms.
__global__ void __launch_bounds__(256, 3) mx_matmul_dx_mid_kernel(MatmulArgs g, int nt) {
  __shared__ __attribute__((aligned(16))) uint8_t dy0[8192], dy1[8192], dy2[8192];
  __shared__ __attribute__((aligned(16))) uint8_t cd0[8192], cd1[8192], cd2[8192];
  __shared__ __attribute__((aligned(16))) uint8_t sc0[512], sc1[512], sc2[512];
  FatItem it;
  if (!find_item<kMidRows>(g.offsets, g.E, g.R, nt, nt, it)) return;
  const DxLds lds{{dy0, dy1, dy2}, {cd0, cd1, cd2}, {sc0, sc1, sc2}};
  if (it.wide) dx_tile<4, 2, 2>(g, it, lds);
  else dx_tile<4, 2, 1>(g, it, lds);
}

}  // namespace

hipError_t launch_mx_matmul_dx_mid(const MatmulArgs& g, hipStream_t s) {
  const int nt = (g.K + 255) / 256;
  const dim3 grid((unsigned)(((long)g.R / kMidRows + std::min(g.E, g.R)) * nt));
  hipLaunchKernelGGL(mx_matmul_dx_mid_kernel, grid, dim3(256), 0, s, g, nt);
  return hipGetLastError();
}

hipError_t launch_mx_matmul_dx_large(const MatmulArgs& g, hipStream_t s) {
  const int ntw = (g.K + 255) / 256, ntn = (g.K + 511) / 512;
  const dim3 grid((unsigned)(((long)g.R / kFatRows + std::min(g.E, g.R)) * ntw));
  hipLaunchKernelGGL(mx_matmul_dx_fat_kernel, grid, dim3(kFatThreads), 0, s, g, ntw, ntn);
  return hipGetLastError();
}

}  // namespace qmoe
