// Grouped products with both sides in MXFP4, for many rows.
//
// A work item is up to 256 rows times 256 outputs on one workgroup of four
// waves, one per SIMD with all 512 registers: 128 x 128 each (runs of up to 128
// rows: 64 outputs x 128 rows each).  A scaled MFMA takes 16 cycles for 2 KB of
// operands, so both sides come through LDS, where a wave tile of 128 x 128
// costs the CU 64 KB of reads per 1024 cycles of MFMAs, half of what LDS
// delivers; taken from global memory into registers, as the bf16 product takes
// its weights, the operands would need more requests than the address units
// answer.  128 inputs per stage, four stages by direct loads: block kb + 4 is
// requested when every wave has block kb in registers; the operands of block
// kb + 1 are read from LDS while block kb is multiplied.
//
// Scales: 16 blocks of a row at a time.  A row's bytes may start anywhere, so
// a thread loads the five aligned words around them, shifts them into place,
// clears what lies past K and writes 16 bytes to LDS.
#include <algorithm>

#include "mxfp4_tile.h"

namespace qmoe {
namespace {

constexpr int kThreads4 = 256;
constexpr int kBlk4 = 128;    // inputs per stage

struct Lds4 {
  uint8_t *a[4], *w[4];   // rows of 64 bytes, 16-byte chunk c of row r at c ^ (r / 4 mod 4)
  uint8_t *as, *ws;       // scales: two groups of 16 bytes per row
};

// A buffer descriptor as four words, for inline assembly.
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 raw_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// 16 bytes per lane from buffer offset `off` into LDS at dst + 16 lane, past
// the compiler's bookkeeping: it tells only a few such loads apart and waits
// for all of them before LDS reads that it cannot prove apart, where this
// pipeline counts its loads itself.  The load has no register result.
__device__ __forceinline__ void to_lds16_raw(const i32x4& r, uint8_t* dst, uint32_t off) {
  const uint32_t d = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)dst;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(__builtin_amdgcn_readfirstlane(d)), "v"(off), "s"(r) : "m0");
}

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
  __device__ __forceinline__ uint4 bytes(uint32_t off, int valid) const {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = __builtin_amdgcn_alignbyte(w[i + 1], w[i], off & 3u);
      const int left = valid - 4 * i;
      o[i] = left >= 4 ? x : left > 0 ? x & (0xffffffffu >> (32 - 8 * left)) : 0u;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

// SL: K % 128 == 0.  Every stage is full, and 16 scales of a row are aligned
// words, which come by direct loads too.
template <bool SL, int RT, int WT, int CT>
__device__ __forceinline__ void tile4(const MatmulArgs& g, const FatItem& it, const Lds4& lds) {
  constexpr int NA = 4, NV = 8;   // direct loads per thread and stage: rows, both
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
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
  const int chunk = (tid & 3) ^ ((tid >> 4) & 3);   // this thread's chunk of a row, the same in each load
  uint32_t aoff[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int64_t src = row_of(i * 64 + (tid >> 2));
    aoff[i] = src >= 0 ? (uint32_t)(src * ldb) + 16u * chunk : kOutside;
  }
  const uint32_t woff = (uint32_t)(n0 + (tid >> 2)) * (uint32_t)ldb + 16u * chunk;

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
      to_lds16_raw(sr_raw[0], lds.ws + (grp & 1) * 4096 + wv * 1024, soff[0] + 16u * (uint32_t)grp);
      to_lds16_raw(sr_raw[1], lds.as + (grp & 1) * 4096 + wv * 1024, soff[1] + 16u * (uint32_t)grp);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) sw[j].load(sr[j], soff[j] + 16u * (uint32_t)grp);
    }
  };
  auto write_s = [&](int grp) {
    if constexpr (SL) return;
    const int valid = nb - 16 * grp;
    *reinterpret_cast<uint4*>(lds.ws + (grp & 1) * 4096 + tid * 16) = sw[0].bytes(soff[0], soff[0] < kOutside ? valid : 0);
    *reinterpret_cast<uint4*>(lds.as + (grp & 1) * 4096 + tid * 16) = sw[1].bytes(soff[1], soff[1] < kOutside ? valid : 0);
  };
  auto issue = [&](auto P, int kb, int i) {   // load i < NV of block kb
    constexpr int p = decltype(P)::value;
    const bool past = !SL && kb * 4 + chunk >= nb;
    if (i < NA)
      to_lds16_raw(ar, lds.a[p] + (i * 4 + wv) * 1024, past ? kOutside : aoff[i % NA] + (uint32_t)kb * 64u);
    else
      to_lds16_raw(wr, lds.w[p] + ((i - NA) * 4 + wv) * 1024,
                   past ? kOutside : woff + (uint32_t)(i - NA) * 64u * (uint32_t)ldb + (uint32_t)kb * 64u);
  };

  f32x4 acc[RT][CT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[rt][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  uint4 W[2][RT], A[2][CT];
  uint32_t ws[2][RT], as[2][CT];
  const int at = lr * 64 + 16 * (lq ^ ((lr >> 2) & 3));
  // part i < 8 of block kb's operands, from stage P into operand set P mod 2
  auto read = [&](auto P, int kb, int i) {
    constexpr int p = decltype(P)::value, s = p & 1;
    const int grp = ((kb >> 2) & 1) * 4096 + (kb & 3) * 4 + lq + lr * 16;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
      if (rt % 8 == i) {
        W[s][rt] = *reinterpret_cast<const uint4*>(lds.w[p] + (wn * RT + rt) * 1024 + at);
        ws[s][rt] = lds.ws[grp + (wn * RT + rt) * 256];
      }
#pragma unroll
    for (int c = 0; c < CT; ++c)
      if (c % 8 == i) {
        A[s][c] = *reinterpret_cast<const uint4*>(lds.a[p] + (wt * CT + c) * 1024 + at);
        as[s][c] = lds.as[grp + (wt * CT + c) * 256];
      }
  };
  auto block = [&](auto P, int kb) {
    constexpr int p = decltype(P)::value, s = p & 1;
    using N1 = std::integral_constant<int, (p + 1) % 4>;
    // block kb is in this wave's registers and its loads of block kb + 1 are in
    // LDS; past the barrier that holds for every wave
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(2 * NV));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const int grp = (kb >> 2) + 1;
    if (p == 0) issue_s(grp);
    if (p == 2) write_s(grp);
    // in eight parts: one request, an eighth of the reads, an eighth of the MFMAs
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      issue(P, min(kb + 4, nkb - 1), i);   // past the end: never read
      read(N1{}, kb + 1, i);
#pragma unroll
      for (int j = 0; j < RT * CT; ++j)
        if (j * 8 / (RT * CT) == i) {
          const int c = j / RT, rt = j % RT;
          const i32x8 wv8 = {(int)W[s][rt].x, (int)W[s][rt].y, (int)W[s][rt].z, (int)W[s][rt].w, 0, 0, 0, 0};
          const i32x8 av8 = {(int)A[s][c].x, (int)A[s][c].y, (int)A[s][c].z, (int)A[s][c].w, 0, 0, 0, 0};
          acc[rt][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv8, av8, acc[rt][c], 4, 4, 0, (int)ws[s][rt], 0, (int)as[s][c]);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  issue_s(0);
  static_for<4>([&](auto J) {
#pragma unroll
    for (int i = 0; i < NV; ++i) issue(J, min(decltype(J)::value, nkb - 1), i);
  });
  write_s(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lds(3 * NV));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < 8; ++i) read(std::integral_constant<int, 0>{}, 0, i);
  for (int kb = 0; kb < nkb; kb += 4)
    static_for<4>([&](auto J) {
      if (kb + decltype(J)::value < nkb) block(J, kb + decltype(J)::value);
    });
  __builtin_amdgcn_s_waitcnt(0);   // the loads past the end

  const bool vec = g.ldo % 4 == 0;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int row = (wt * CT + c) * 16 + lr;
    if (row >= it.M) continue;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) store4(g, vec, it.r0 + row, n0 + (wn * RT + rt) * 16 + 4 * lq, acc[rt][c]);
  }
}

template <bool SL>
__global__ void __launch_bounds__(kThreads4, 1) mx_matmul4_kernel(MatmulArgs g, int nt) {
  __shared__ __attribute__((aligned(16))) uint8_t a0[16384], a1[16384], a2[16384], a3[16384];
  __shared__ __attribute__((aligned(16))) uint8_t w0[16384], w1[16384], w2[16384], w3[16384];
  __shared__ __attribute__((aligned(16))) uint8_t as[8192], ws[8192];
  FatItem it;
  if (!find_item(g.offsets, g.E, g.R, nt, nt, it)) return;
  const Lds4 lds{{a0, a1, a2, a3}, {w0, w1, w2, w3}, as, ws};
  if (it.wide) {
    if (it.M > 192) tile4<SL, 8, 2, 8>(g, it, lds);
    else tile4<SL, 8, 2, 6>(g, it, lds);
  } else {
    if (it.M > 96) tile4<SL, 4, 1, 8>(g, it, lds);
    else if (it.M > 64) tile4<SL, 4, 1, 6>(g, it, lds);
    else if (it.M > 32) tile4<SL, 4, 1, 4>(g, it, lds);
    else if (it.M > 16) tile4<SL, 4, 1, 2>(g, it, lds);
    else tile4<SL, 4, 1, 1>(g, it, lds);
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
