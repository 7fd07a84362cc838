// Device code shared by the row operators: eight neighbouring values of a row
// (a "unit") are what a lane holds, 16 bytes of bf16 or 32 of fp32.
#pragma once

#include "qmoe_device.h"
#include "rows_internal.h"

namespace qmoe {

constexpr int kUnit = 8;
// dtype of a matrix known at compile time, or only at run time, or bf16 of a matrix that
// is read once and whose lines go first when room is needed (read_once)
constexpr int kAnyDtype = -1;
constexpr int kBf16Once = 0x100 | MOE_DT_BF16;
template <int DT>
constexpr bool kIsBf16 = DT == MOE_DT_BF16 || DT == kBf16Once;
template <int DT>
constexpr int kPlain = kIsBf16<DT> ? (int)MOE_DT_BF16 : DT;

// Where a lane's unit lies in its row.  A row's last values come with those before
// them, as whole units that end where the row ends: `skip` of the eight are another
// lane's too, who comes to the same results and may store the same values.  Loads and
// stores then need no path for parts of a unit, whose waits would end the flow of the
// loads behind it (SwiGLU, norm and sums of 1502 columns: within 5 % of 1504).  Sums
// leave the skipped values out.  TAIL: units start where they would and end early, for
// rows of less than eight values and for results that overwrite what other lanes read.
template <bool TAIL>
struct Span {
  int c;       // column of the first value
  int n;       // own values of the unit; 0 and less: none
  int skip;    // values before the own ones (8 and more: no own ones)
  __device__ __forceinline__ Span(int unit, int cols) {
    const int begin = unit * kUnit;
    n = cols - begin;
    c = TAIL ? begin : min(begin, cols - kUnit);
    skip = begin - c;
  }
};

template <int DT>
struct Unit {
  uint32_t w[kIsBf16<DT> ? 4 : 8];
};

template <int DT>
__device__ __forceinline__ bool is_bf16(int dtype) {
  if constexpr (DT == kAnyDtype) return dtype == MOE_DT_BF16;
  return kIsBf16<DT>;
}

// The first n < 8 values of a row's last unit come and go as a run of four, one of
// two and one of one (those that n has), so in three accesses at most.  WORDS of
// dwords hold eight values.
template <int WORDS>
__device__ __forceinline__ void load_tail(uint32_t (&w)[WORDS], const uint8_t* p, int n) {
  constexpr int kSize = WORDS / 2, kHalf = WORDS / 2, kQuarter = WORDS / 4;   // bytes a value; dwords of four, of two
  const bool has4 = n & 4;
  uint32_t four[kHalf] = {}, two[kQuarter] = {}, one = 0;
  if (has4) __builtin_memcpy(four, p, 4 * kSize);
  if (n & 2) __builtin_memcpy(two, p + (n & 4) * kSize, 2 * kSize);
  if (n & 1) __builtin_memcpy(&one, p + (n & 6) * kSize, kSize);
  uint32_t v[WORDS];
#pragma unroll
  for (int i = 0; i < kHalf; ++i) {
    const uint32_t t = i < kQuarter ? two[i % kQuarter] : 0u;
    v[i] = has4 ? four[i] : t;
    v[kHalf + i] = has4 ? t : 0u;
  }
  // behind an even number of values
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i * kQuarter] = v[i * kQuarter] | ((n & 6) == 2 * i ? one : 0u);
  if constexpr (kQuarter == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[2 * i + 1] = v[2 * i + 1];
  }
}

template <int WORDS>
__device__ __forceinline__ void store_tail(uint8_t* p, const uint32_t (&w)[WORDS], int n) {
  constexpr int kSize = WORDS / 2, kHalf = WORDS / 2, kQuarter = WORDS / 4;
  const uint32_t has4 = n & 4 ? ~0u : 0u;
  uint32_t four[kHalf], two[kQuarter], one = 0;
#pragma unroll
  for (int i = 0; i < kHalf; ++i) four[i] = w[i];
#pragma unroll
  for (int i = 0; i < kQuarter; ++i) two[i] = (w[kHalf + i] & has4) | (w[i] & ~has4);
#pragma unroll
  for (int i = 0; i < 4; ++i) one |= (n & 6) == 2 * i ? w[i * kQuarter] : 0u;
  if (n & 4) __builtin_memcpy(p, four, 4 * kSize);
  if (n & 2) __builtin_memcpy(p + (n & 4) * kSize, two, 2 * kSize);
  if (n & 1) __builtin_memcpy(p + (n & 6) * kSize, &one, kSize);
}

// Values [at, at + 8) of a matrix in memory; TAIL: those past the first n as zeros
// (n <= 0: none is read).
template <bool TAIL, int DT>
__device__ __forceinline__ void load_unit(Unit<DT>& u, const void* base, int dtype, int64_t at, int n) {
  constexpr int kWords = kIsBf16<DT> ? 4 : 8;
#pragma unroll
  for (int i = 0; i < kWords; ++i) u.w[i] = 0;
  if constexpr (DT == kBf16Once && !TAIL) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + at));
#pragma unroll
    for (int i = 0; i < 4; ++i) u.w[i] = v[i];
  } else if (is_bf16<DT>(dtype)) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + at * 2;
    uint32_t w[4] = {};
    if (!TAIL || n >= kUnit) __builtin_memcpy(w, p, 16);
    else if (n > 0) load_tail(w, p, n);
#pragma unroll
    for (int i = 0; i < 4; ++i) u.w[i] = w[i];
  } else if constexpr (kWords == 8) {
    const uint8_t* p = static_cast<const uint8_t*>(base) + at * 4;
    if (!TAIL || n >= kUnit) __builtin_memcpy(u.w, p, 32);
    else if (n > 0) load_tail(u.w, p, n);
  }
}

template <int DT>
__device__ __forceinline__ void unit_floats(const Unit<DT>& u, int dtype, float (&v)[kUnit]) {
  if (is_bf16<DT>(dtype)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(u.w[i]);
      v[2 * i + 1] = bf16_hi(u.w[i]);
    }
  } else if constexpr (!kIsBf16<DT>) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = __uint_as_float(u.w[i]);
  }
}

// Hides a unit's values from the optimiser, so that what was made of them before is
// made again instead of being kept.
template <int DT>
__device__ __forceinline__ void forget_values(Unit<DT>& u) {
#pragma unroll
  for (int i = 0; i < (kIsBf16<DT> ? 4 : 8); ++i) opaque(u.w[i]);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// Rounds eight values to a dtype and back.
__device__ __forceinline__ void round_to(int dtype, float (&v)[kUnit]) {
  if (dtype != MOE_DT_BF16) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = pack_bf16(v[2 * i], v[2 * i + 1]);
    v[2 * i] = bf16_lo(w);
    v[2 * i + 1] = bf16_hi(w);
  }
}

// 16 bytes to memory, past the caches where the results are more than they hold.
__device__ __forceinline__ void store16(uint8_t* p, const uint32_t* w, bool past_cache) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
  const u32x4 v = {w[0], w[1], w[2], w[3]};
  if (past_cache) {
    // the empty statements keep the two stores from becoming one ordinary one
    asm volatile("");
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
    asm volatile("");
  } else {
    *reinterpret_cast<u32x4*>(p) = v;
  }
}

// Eight values to [at, at + 8) of a matrix; TAIL: the first n > 0 of them.
template <bool TAIL>
__device__ __forceinline__ void store_unit(void* base, int dtype, int64_t at, int n, const float (&v)[kUnit],
                                           bool past_cache = false) {
  if (dtype == MOE_DT_BF16) {
    uint8_t* p = static_cast<uint8_t*>(base) + at * 2;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if (!TAIL || n >= kUnit) store16(p, w, past_cache);
    else store_tail(p, w, n);
  } else {
    uint8_t* p = static_cast<uint8_t*>(base) + at * 4;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
    if (!TAIL || n >= kUnit) {
      store16(p, w, past_cache);
      store16(p + 16, w + 4, past_cache);
    } else {
      store_tail(p, w, n);
    }
  }
}

// Largest magnitude of eight values as fp32 bits, which order like the values,
// infinities and NaN last.
__device__ __forceinline__ uint32_t top_bits(const float (&v)[kUnit]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// Scale of an E4M3 row from its largest magnitude.  Below 2^-126 a scale would
// lose bits, and its reciprocal could overflow.
__device__ __forceinline__ float e4m3_scale(uint32_t top) {
  if (top >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(top) / 448.0f, 0x1p-126f);
}

// x / scale from the rounded reciprocal, one correction: the product alone would
// put about one code in 10^6 on the other side of a tie.
__device__ __forceinline__ float quotient(float x, float scale, float inv) {
  const float v = x * inv;
  return fmaf(fmaf(-v, scale, x), inv, v);
}

// E4M3 codes of eight values of a row with this scale (NaN: all codes 0).  A
// quotient may pass 448 by a unit in the last place of fp32; E4M3 rounds
// everything below 464 to 448.
__device__ __forceinline__ uint2 e4m3_codes(const float (&v)[kUnit], float scale) {
  if (scale != scale) return make_uint2(0u, 0u);
  const float inv = 1.0f / scale;
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = quotient(v[4 * i + j], scale, inv);
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(d[0], d[1], 0, false);
    q = __builtin_amdgcn_cvt_pk_fp8_f32(d[2], d[3], q, true);
    w[i] = (uint32_t)q;
  }
  return make_uint2(w[0], w[1]);
}

// Eight code bytes; TAIL: the first n > 0 of them.
template <bool TAIL>
__device__ __forceinline__ void store_bytes(uint8_t* p, int n, uint2 q) {
  if (!TAIL || n >= kUnit) {
    __builtin_memcpy(p, &q, 8);
    return;
  }
  if (n & 4) __builtin_memcpy(p, &q.x, 4);
  const uint32_t rest = n & 4 ? q.y : q.x;
  if (n & 2) {
    const uint16_t two = (uint16_t)rest;
    __builtin_memcpy(p + (n & 4), &two, 2);
  }
  if (n & 1) p[n & 6] = (uint8_t)(n & 2 ? rest >> 16 : rest);
}

// The own values of a unit first, then zeros.
__device__ __forceinline__ void own_first(float (&v)[kUnit], int skip) {
  if (skip == 0) return;
  if (skip & 4) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = i < 4 ? v[(i + 4) % kUnit] : 0.0f;
  }
  if (skip & 2) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = i < 6 ? v[(i + 2) % kUnit] : 0.0f;
  }
  if (skip & 1) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = i < 7 ? v[(i + 1) % kUnit] : 0.0f;
  }
  if (skip >= kUnit) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = 0.0f;
  }
}

// MXFP4 of a block of 32 that four neighbouring lanes hold, eight values each
// (values past the row's end zeros): this lane's codes and the block's scale
// byte, as moe_mxfp4_quantize makes them.
__device__ __forceinline__ uint32_t mxfp4_codes(const float (&v)[kUnit], uint32_t& byte) {
  uint32_t m = top_bits(v);
  m = max(m, dpp<kDppXor1>(m));
  m = max(m, dpp<kDppXor2>(m));
  const uint32_t e = m >> 23;
  byte = e == 255u ? 255u : (uint32_t)max((int)e - 2, 0);
  if (e == 255u) return 0;
  const float s = __uint_as_float(byte << 23);   // the conversion uses the exponent alone, 0 for 2^-127
  uint32_t q = 0;
  static_for<4>([&](auto I) {
    constexpr int i = decltype(I)::value;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2 * i], v[2 * i + 1], s, i);
  });
  return q;
}

// Reductions over G = 4, 8 .. 64 neighbouring lanes, every lane with the result.
template <int G, class T, class F>
__device__ __forceinline__ T lanes_reduce(T v, F&& join) {
  auto step = [&](auto ctrl) {
    constexpr int c = decltype(ctrl)::value;
    if constexpr (sizeof(T) == 8) v = join(v, dppd<c>(v));
    else v = join(v, __builtin_bit_cast(T, dpp<c>(__builtin_bit_cast(uint32_t, v))));
  };
  step(std::integral_constant<int, kDppXor1>{});
  step(std::integral_constant<int, kDppXor2>{});
  if constexpr (G >= 8) step(std::integral_constant<int, kDppHalfMirror>{});
  if constexpr (G >= 16) step(std::integral_constant<int, kDppMirror>{});
  auto swap = [&](auto m) {
    if constexpr (sizeof(T) == 8) {
      T a, b;
      swap_pair<decltype(m)::value>(v, a, b);
      v = join(a, b);
    } else {
      int a, b;
      swap_pair<decltype(m)::value>(__builtin_bit_cast(int, v), a, b);
      v = join(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
    }
  };
  if constexpr (G >= 32) swap(std::integral_constant<int, 16>{});
  if constexpr (G >= 64) swap(std::integral_constant<int, 32>{});
  return v;
}

// Over the G lanes that share a row: up to a wave, or the whole workgroup through
// `lds`, which holds one value a wave and is free again after the next barrier.
template <int G, class T, class F>
__device__ __forceinline__ T group_reduce(T v, T* lds, F&& join) {
  if constexpr (G <= kWave) return lanes_reduce<G>(v, join);
  v = lanes_reduce<kWave>(v, join);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int i = 1; i < G / kWave; ++i) v = join(v, lds[i]);
  return v;
}
template <int G>
__device__ __forceinline__ double group_sum(double v, double* lds) {
  return group_reduce<G>(v, lds, [](double a, double b) { return a + b; });
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t* lds) {
  return group_reduce<G>(v, lds, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// Workgroups go to the eight XCDs in turn.  In order they are numbered so that
// neighbours run on one XCD.  Where rows end inside a line, both writers of the line
// then meet in one L2 instead of each sending a part of it to memory (bf16, dispatch
// of 8000 tokens to 8 rows of 2056 73 us against 81, of 4104 128 against 133; SwiGLU
// and gradient of 20000 x 2056 131 against 140); with rows of whole lines taking
// turns is better (dispatch to 8 rows of 6144 165 us against 172).  The norm, the sums
// and their gradient are within 2 % either way, and take turns.
__device__ __forceinline__ unsigned block_number(bool in_order) {
  if (!in_order) return blockIdx.x;
  const unsigned n = gridDim.x, xcd = blockIdx.x & 7, each = n >> 3, more = n & 7;
  return xcd * each + min(xcd, more) + (blockIdx.x >> 3);
}
// Whether the norm's results go past the caches: more of them than the 256 MB behind
// L2 hold only push out what is yet to be read.  Norm of 16384 x 6144 bf16 with the
// kernel that quantises its result 183 us past the caches and 190 through them (alone
// 133 and 140); of 8192 rows, which the next kernel finds there, 89 and 85.  The
// gradient of collect is faster past them by itself (4096 tokens, 403 MB: 173 us, 182),
// but the products that read its rows lose more (811 us in all, 806), and so it is with
// SwiGLU (32768 x 2048 and what quantises it: 99 us, 89).
inline bool past_cache(int64_t bytes) { return bytes > (int64_t)256 << 20; }

// Whether the rows of a matrix end inside lines.
inline bool ragged_lines(const void* p, int64_t pitch_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch_bytes) & 127) != 0;
}

// Whether the bf16 rows of a matrix are read with kBf16Once.  Inputs that the caches
// cannot hold then leave them to what is written, for the next reader: SwiGLU of 32768 x
// 2048 66 us against 69, right after gu was written 162 against 172 for both; norm of
// 16384 x 6144 with its gradient, x written before, 344 against 372, of 8192 (96 MB each)
// 174 against 200.  Under that the caches still hold what was written last, and it comes
// slower so: norm of 4096 right after x 50 us against 47, SwiGLU of 8000 x 1024 11.6
// against 10.4.  Rows that end inside lines are read in part by two workgroups (norm of
// 24000 x 1503 60 us against 58), fp32 rows in two requests a line (SwiGLU and gradient
// of 10000 x 2056 183 against 153).
constexpr int64_t kOnceBytes = (int64_t)96 << 20;
inline bool read_once(const RowMat& m, int64_t rows, int64_t cols) {
  return !m.p || (m.dtype == MOE_DT_BF16 && rows * cols * 2 >= kOnceBytes && !ragged_lines(m.p, m.ld * 2));
}

constexpr int kMapBlock = 256;

// Row and chunk of a lane; the row is uniform over the workgroup if LONG.
template <bool LONG>
__device__ __forceinline__ void locate(const RowMap& m, int& row, int& chunk) {
  if constexpr (LONG) {
    const unsigned b = block_number(m.in_order), r = b / (unsigned)m.parts;
    chunk = (b - r * m.parts) * blockDim.x + threadIdx.x;
    row = m.first + r;
  } else {
    const unsigned at = block_number(m.in_order) * kMapBlock + threadIdx.x;
    row = m.first + (at >> m.bits);
    chunk = at & ((1u << m.bits) - 1);
  }
}

inline RowMap row_map(int chunks, bool in_order) {
  if (chunks > 32) {
    const int parts = (chunks + kMapBlock - 1) / kMapBlock;
    const int each = (chunks + parts - 1) / parts;
    return {parts, (each + kWave - 1) / kWave * kWave, -1, 0, in_order};
  }
  int bits = 0;
  while ((1 << bits) < chunks) ++bits;
  return {1, kMapBlock, bits, 0, in_order};
}

// Work items of a launch, which has to stay below 2^32 of them.
constexpr int64_t kMostItems = 1ll << 31;

// Calls f(first row, workgroups) for runs of rows where a workgroup of `block` lanes
// takes `per` of them.
template <class F>
hipError_t by_runs(int rows, int block, int per, F&& f) {
  const int64_t most = kMostItems / block * per;
  for (int64_t r = 0; r < rows; r += most) {
    f((int)r, dim3((unsigned)(((rows - r < most ? rows - r : most) + per - 1) / per)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Calls f(LONG, TAIL, grid, block, map), the first two as integral constants, for runs
// of rows.  LONG_TAIL: long rows may need tails too, where a result may lie over an
// input; others do for less than eight columns alone.
template <bool LONG_TAIL, class F>
hipError_t by_rows(RowMap m, int rows, bool tail, F&& f) {
  const int64_t most = m.bits < 0 ? kMostItems / ((int64_t)m.parts * kMapBlock) : kMostItems >> 5;
  for (int64_t r = 0; r < rows; r += most) {
    const unsigned n = (unsigned)(rows - r < most ? rows - r : most);
    m.first = (int)r;
    if (m.bits >= 0) {
      const dim3 dense((unsigned)((((int64_t)n << m.bits) + kMapBlock - 1) / kMapBlock));
      if (tail) f(std::false_type{}, std::true_type{}, dense, dim3(kMapBlock), m);
      else f(std::false_type{}, std::false_type{}, dense, dim3(kMapBlock), m);
    } else if (LONG_TAIL && tail) {
      f(std::true_type{}, std::integral_constant<bool, LONG_TAIL>{}, dim3(n * m.parts), dim3(m.threads), m);
    } else {
      f(std::true_type{}, std::false_type{}, dim3(n * m.parts), dim3(m.threads), m);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qmoe
