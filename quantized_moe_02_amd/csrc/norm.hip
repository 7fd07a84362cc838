// Root-mean-square norm with the residual's addition, and its gradient.
//
//   h = x + residual,  y = h m w  with  m = 1 / sqrt(mean(h^2) + eps)
//   g = dy w,  dx = dh + m (g - h m^2 mean(g h)),  dw = sum over rows of dy h m
//
// Both move bytes and are bound by HBM.  A row lies in the registers of the G lanes
// that share it, U units of eight values a lane, so that it is read once for its sums
// and its results alike; it stays there as it came (bf16 as bf16) and is widened again
// after the sums, which halves the registers.  Rows of up to 512 columns take the 4 to
// 64 lanes that they fill, of up to 1536 a wave, of up to 8192 a workgroup of 256, then
// of 512 or 1024; past 32768 (gradient: 16384) they are read again from L2.
//
// Sums over a row are float64: squares of fp32 values leave fp32's range, and fp64
// additions do not show beside the bytes.  m, the products and y are fp32, each result
// rounded once.
//
// dw: a workgroup of the gradient takes rows in turn and sums its columns in registers, in
// fp32 over eight rows; runs of eight are added in float64, in LDS (rows past 16384 columns:
// in the workgroup's own part in memory).  A second launch adds the workgroups' sums in
// float64, in order.  No atomics, the same bits every time.
//
// Measured, averages: 16384 x 6144 bf16 with residual 133 us (805 MB, 6.1 TB/s), with
// E4M3 rows beside 155 (906 MB, 5.8 TB/s); followed by its gradient 133 + 147, and 5 to
// join 512 parts (1.61 GB in all, 5.7 TB/s).  1 x 6144 3.8 us, 64 x 6144 fp32 onto bf16 to
// MXFP4 5.5: the latency of one row.  1027 x 2057 fp32 7 us, its gradient 11.5 + 4: the
// launches, and three rows one after the other.  24000 x 1503 bf16 58 us (5.0 TB/s).
// 1627 x 8815 with fp32 dy 65 us for both against 42 at a copy's rate: one workgroup of
// 512 a CU (a second would have to do with 128 registers and 80 KB of LDS) waits for each
// row.
#include <algorithm>

#include "rows_device.h"

namespace qmoe {
namespace {

// Lanes of a workgroup whose rows take G lanes each, and its rows.
constexpr int block_of(int g) { return g > 256 ? g : 256; }
constexpr int kWide = 1024;      // lanes for rows that are read again

// MXFP4 of a unit's own values; all lanes of a quad take part, also those past the
// row's end.
__device__ __forceinline__ void put_mxfp4(const NormArgs& a, int64_t row, int unit, int skip, float (&v)[kUnit]) {
  uint32_t byte;
  own_first(v, skip);
  const uint32_t q = mxfp4_codes(v, byte);
  const int nb = (a.cols + kMxBlock - 1) / kMxBlock;
  if (unit < nb * 4) {
    static_cast<uint32_t*>(a.q)[row * nb * 4 + unit] = q;
    if (unit % 4 == 0) static_cast<uint8_t*>(a.q_scale)[row * nb + unit / 4] = (uint8_t)byte;
  }
}

__device__ __forceinline__ float inverse_rms(double sum, int cols, float eps) {
  return (float)(1.0 / sqrt(sum / cols + (double)eps));
}

// Sum of squares of a unit's own values.
__device__ __forceinline__ double squares(const float (&h)[kUnit], int skip) {
  double sum = 0;
  if (skip == 0) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) sum += (double)h[i] * h[i];
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) sum += i >= skip ? (double)h[i] * h[i] : 0.0;
  }
  return sum;
}

// h of a unit, rounded to the stream's type, from x and the residual.
template <int XT, int RT>
__device__ __forceinline__ void add_residual(const NormArgs& a, const Unit<XT>& x, const Unit<RT>& r, float (&h)[kUnit]) {
  unit_floats(x, a.x.dtype, h);
  if (a.res.p) {
    float v[kUnit];
    unit_floats(r, a.res.dtype, v);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) h[i] += v[i];
    round_to(RT == kAnyDtype ? a.res.dtype : kPlain<RT>, h);
  }
}

// h of a unit between the sum and its use: bf16 where it is that, else fp32.
template <int DT>
__device__ __forceinline__ void hold(Unit<DT>& u, const float (&h)[kUnit]) {
  if constexpr (kIsBf16<DT>) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u.w[i] = pack_bf16(h[2 * i], h[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) u.w[i] = __float_as_uint(h[i]);
  }
}

// RT is h's type, with or without a residual.  Nothing is stored before the whole row is
// read: h may be the residual itself, and the last lanes of a row read values of the ones
// before them.
template <int XT, int RT, int G, int U, bool TAIL>
__global__ void __launch_bounds__(block_of(G)) rmsnorm_kernel(NormArgs a) {
  constexpr int kRows = block_of(G) / G;
  __shared__ double sums[block_of(G) / kWave];
  __shared__ uint32_t tops[block_of(G) / kWave];
  const int lane = threadIdx.x % G;
  int64_t row = a.first + (int64_t)blockIdx.x * kRows;
  if constexpr (G < kWave) row += threadIdx.x / G;
  else if constexpr (G == kWave) row += __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  if (row >= a.rows) return;
  Unit<XT> x[U];
  Unit<RT> r[U];
  Unit<kAnyDtype> w[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Span<TAIL> p(u * G + lane, a.cols);
    load_unit<TAIL>(x[u], a.x.p, a.x.dtype, row * a.x.ld + p.c, p.n);
    if (a.res.p) load_unit<TAIL>(r[u], a.res.p, a.res.dtype, row * a.res.ld + p.c, p.n);
    load_unit<TAIL>(w[u], a.w, a.w_dtype, p.c, p.n);
  }
  double sum = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float h[kUnit];
    add_residual(a, x[u], r[u], h);
    sum += squares(h, Span<TAIL>(u * G + lane, a.cols).skip);
    hold(r[u], h);
  }
  const float m = inverse_rms(group_sum<G>(sum, sums), a.cols, a.eps);
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Span<TAIL> p(u * G + lane, a.cols);
    float h[kUnit], v[kUnit];
    forget_values(r[u]);       // else the fp32 values stay in registers all along
    unit_floats(r[u], RT, h);
    if (a.h.p && p.n > 0) store_unit<TAIL>(a.h.p, a.h.dtype, row * a.h.ld + p.c, p.n, h, a.past_cache);
    unit_floats(w[u], a.w_dtype, v);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = h[i] * m * v[i];
    if (a.y.p && p.n > 0) store_unit<TAIL>(a.y.p, a.y.dtype, row * a.y.ld + p.c, p.n, v, a.past_cache);
    if (a.q && a.q_dtype == MOE_DT_MXFP4) put_mxfp4(a, row, u * G + lane, p.skip, v);
    if (a.q && a.q_dtype == MOE_DT_E4M3) top = max(top, top_bits(v));
  }
  if (a.q && a.q_dtype == MOE_DT_E4M3) {
    const float scale = e4m3_scale(group_max<G>(top, tops));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Span<TAIL> p(u * G + lane, a.cols);
      float h[kUnit], v[kUnit];
      unit_floats(r[u], RT, h);
      unit_floats(w[u], a.w_dtype, v);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) v[i] = h[i] * m * v[i];
      if (p.n > 0) store_bytes<TAIL>(static_cast<uint8_t*>(a.q) + row * a.cols + p.c, p.n, e4m3_codes(v, scale));
    }
    if (lane == 0) static_cast<float*>(a.q_scale)[row] = scale;
  }
}

// Rows past the registers of a workgroup, read again for each pass over them.  h,
// which may be the residual itself, is written with the last reading.
__global__ void __launch_bounds__(kWide) rmsnorm_wide_kernel(NormArgs a) {
  __shared__ double sums[kWide / kWave];
  __shared__ uint32_t tops[kWide / kWave];
  const int64_t row = a.first + (int64_t)blockIdx.x;
  const int units = (a.cols + kMxBlock - 1) / kMxBlock * 4;     // whole quads of lanes
  auto read = [&](int c, float (&h)[kUnit]) {
    Unit<kAnyDtype> x, r;
    load_unit<true>(x, a.x.p, a.x.dtype, row * a.x.ld + c, a.cols - c);
    if (a.res.p) load_unit<true>(r, a.res.p, a.res.dtype, row * a.res.ld + c, a.cols - c);
    add_residual(a, x, r, h);
  };
  auto normed = [&](int c, float m, float (&h)[kUnit]) {
    Unit<kAnyDtype> w;
    float wv[kUnit];
    load_unit<true>(w, a.w, a.w_dtype, c, a.cols - c);
    unit_floats(w, a.w_dtype, wv);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) h[i] = h[i] * m * wv[i];
  };
  double sum = 0;
  float h[kUnit];
  for (int u = threadIdx.x; u < units; u += kWide) {
    read(u * kUnit, h);
    sum += squares(h, 0);
  }
  const float m = inverse_rms(group_sum<kWide>(sum, sums), a.cols, a.eps);
  float scale = 0.0f;
  if (a.q && a.q_dtype == MOE_DT_E4M3) {
    uint32_t top = 0;
    for (int u = threadIdx.x; u < units; u += kWide) {
      read(u * kUnit, h);
      normed(u * kUnit, m, h);
      top = max(top, top_bits(h));
    }
    scale = e4m3_scale(group_max<kWide>(top, tops));
    if (threadIdx.x == 0) static_cast<float*>(a.q_scale)[row] = scale;
  }
  for (int u = threadIdx.x; u < units; u += kWide) {
    const int c = u * kUnit, n = a.cols - c;
    read(c, h);
    if (a.h.p && n > 0) store_unit<true>(a.h.p, a.h.dtype, row * a.h.ld + c, n, h);
    normed(c, m, h);
    if (a.y.p && n > 0) store_unit<true>(a.y.p, a.y.dtype, row * a.y.ld + c, n, h);
    if (!a.q) continue;
    if (a.q_dtype == MOE_DT_MXFP4) put_mxfp4(a, row, u, 0, h);
    else if (n > 0) store_bytes<true>(static_cast<uint8_t*>(a.q) + row * a.cols + c, n, e4m3_codes(h, scale));
  }
}

// Sums over a row that the gradient needs.
struct RowSums {
  double squares, product;     // of h; of g * h
};

// m and m^2 * mean(g * h) of a row.
__device__ __forceinline__ void row_factors(RowSums s, int cols, float eps, float& m, float& k) {
  const double r = 1.0 / sqrt(s.squares / cols + (double)eps);
  m = (float)r;
  k = (float)(s.product / cols * r * r);
}

// Sum of dy * w * h over a unit's own values.
__device__ __forceinline__ double product(const float (&dy)[kUnit], const float (&w)[kUnit], const float (&h)[kUnit], int skip) {
  double sum = 0;
  if (skip == 0) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) sum += (double)(dy[i] * w[i]) * h[i];
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) sum += i >= skip ? (double)(dy[i] * w[i]) * h[i] : 0.0;
  }
  return sum;
}

// Weights beside bf16 rows are bf16 too, but for any types.
template <int DT>
constexpr int weight_dtype() { return kIsBf16<DT> ? MOE_DT_BF16 : kAnyDtype; }

// Rows whose share of dw is summed in fp32 before it is added to the float64 sums: about as
// exact as float64 alone (16384 x 6144 bf16 dw off by 7.1e-8 of its norm, 4.9e-8 by the final
// rounding, 1.1e-7 with all 32 rows of a workgroup in fp32) at an eighth of its LDS traffic
// (with fp32 sums alone: 20000 x 2000 129.5 us against 127.7, 16384 x 6144 282 both).
constexpr int kDwRun = 8;

// Workgroups take rows in turn and hold dw's sums over theirs, each lane its own in LDS.
// As in the norm, nothing of a row is stored before all of it is read.  DT is the type of h,
// dh and dx, YT that of dy.
template <int DT, int YT, int G, int U, bool TAIL>
__global__ void __launch_bounds__(block_of(G)) rmsnorm_grad_kernel(NormGradArgs a) {
  constexpr int kBlock = block_of(G), kRows = kBlock / G;
  __shared__ double lds[2][2][kBlock / kWave];
  __shared__ double sums[U][kUnit][kBlock + (kRows > 1 ? 8 : 0)];     // a row's columns in banks of their own
  const int lane = threadIdx.x % G;
  int64_t row = (int64_t)blockIdx.x * kRows;
  if constexpr (G < kWave) row += threadIdx.x / G;
  else if constexpr (G == kWave) row += __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  Unit<weight_dtype<DT>()> wr[U];
  float acc[U][kUnit] = {};
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Span<TAIL> p(u * G + lane, a.cols);
    load_unit<TAIL>(wr[u], a.w, a.w_dtype, p.c, p.n);
  }
  auto total = [&](int u, int i, bool first) { return (first ? 0.0 : sums[u][i][threadIdx.x]) + acc[u][i]; };
  int turn = 0, run = 0;
  bool first = true;           // no run of rows is in the sums yet
  for (; row < a.rows; row += (int64_t)gridDim.x * kRows, turn ^= 1) {
    Unit<DT> hr[U], dr[U];
    Unit<YT> yr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Span<TAIL> p(u * G + lane, a.cols);
      load_unit<TAIL>(hr[u], a.h.p, a.h.dtype, row * a.h.ld + p.c, p.n);
      load_unit<TAIL>(yr[u], a.dy.p, a.dy.dtype, row * a.dy.ld + p.c, p.n);
      if (a.dh.p) load_unit<TAIL>(dr[u], a.dh.p, a.dh.dtype, row * a.dh.ld + p.c, p.n);
    }
    // while the row is on its way
    if (a.dw && run == kDwRun) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          sums[u][i][threadIdx.x] = total(u, i, first);
          acc[u][i] = 0.0f;
        }
      }
      first = false;
      run = 0;
    }
    ++run;
    RowSums s{0, 0};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int skip = Span<TAIL>(u * G + lane, a.cols).skip;
      float w[kUnit], h[kUnit], dy[kUnit];
      unit_floats(wr[u], a.w_dtype, w);
      unit_floats(hr[u], a.h.dtype, h);
      unit_floats(yr[u], a.dy.dtype, dy);
      s.squares += squares(h, skip);
      s.product += product(dy, w, h, skip);
    }
    s.squares = group_sum<G>(s.squares, lds[turn][0]);
    s.product = group_sum<G>(s.product, lds[turn][1]);
    float m, k;
    row_factors(s, a.cols, a.eps, m, k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Span<TAIL> p(u * G + lane, a.cols);
      float dx[kUnit], w[kUnit], h[kUnit], dy[kUnit];
      forget_values(wr[u]);      // else the fp32 values stay in registers all along
      forget_values(hr[u]);
      forget_values(yr[u]);
      unit_floats(wr[u], a.w_dtype, w);
      unit_floats(hr[u], a.h.dtype, h);
      unit_floats(yr[u], a.dy.dtype, dy);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        dx[i] = m * (dy[i] * w[i] - h[i] * k);
        acc[u][i] += dy[i] * (h[i] * m);
      }
      if (a.dh.p) {
        float d[kUnit];
        unit_floats(dr[u], a.dh.dtype, d);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) dx[i] += d[i];
      }
      if (p.n > 0) store_unit<TAIL>(a.dx.p, a.dx.dtype, row * a.dx.ld + p.c, p.n, dx, a.past_cache);
    }
  }
  if (!a.dw) return;
  float* part = gridDim.x == 1 ? a.dw : static_cast<float*>(a.part) + (int64_t)blockIdx.x * a.cols;
  if constexpr (kRows > 1) {       // the sums of the workgroup's rows, in order
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) sums[u][i][threadIdx.x] = total(u, i, first);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kBlock) {
      const int unit = c / kUnit, i = c - Span<TAIL>(unit, a.cols).c;
      double v = 0;
#pragma unroll 8
      for (int r = 0; r < kRows; ++r) v += sums[unit / G][i][r * G + unit % G];
      part[c] = (float)v;
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Span<TAIL> p(u * G + lane, a.cols);
      float v[kUnit];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) v[i] = (float)total(u, i, first);
      if (p.n > 0) store_unit<TAIL>(part, MOE_DT_F32, p.c, p.n, v);
    }
  }
}

// Longer rows: read twice, kWideTurns of them for each reading and writing of dweight's
// sums, which lie in the workgroup's own part: as float64, but where it takes no more rows
// than that (T float), whose sums are written once.
constexpr int kWideTurns = 4;
template <class T>
__global__ void __launch_bounds__(kWide) rmsnorm_grad_wide_kernel(NormGradArgs a) {
  constexpr int kTurns = kWideTurns;
  __shared__ double lds[2][2][kWide / kWave];
  __shared__ float factors[kTurns][2];          // m and k of the rows in turn
  T* part = gridDim.x == 1 ? reinterpret_cast<T*>(a.dw) : static_cast<T*>(a.part) + (int64_t)blockIdx.x * a.cols;   // one: T float
  auto read = [&](int64_t row, int c, float (&h)[kUnit], float (&dy)[kUnit]) {
    Unit<kAnyDtype> v;
    const int n = a.cols - c;
    load_unit<true>(v, a.h.p, a.h.dtype, row * a.h.ld + c, n);
    unit_floats(v, a.h.dtype, h);
    load_unit<true>(v, a.dy.p, a.dy.dtype, row * a.dy.ld + c, n);
    unit_floats(v, a.dy.dtype, dy);
  };
  auto weight = [&](int c, float (&w)[kUnit]) {
    Unit<kAnyDtype> v;
    load_unit<true>(v, a.w, a.w_dtype, c, a.cols - c);
    unit_floats(v, a.w_dtype, w);
  };
  // hides that rows ascend, else an address of each matrix for each loop over them is kept
  auto row_of = [](int row) {
    uint32_t r = row;
    opaque(r);
    return (int64_t)r;
  };
  const int step = gridDim.x;
  float h[kUnit], dy[kUnit], w[kUnit];
  for (int first = blockIdx.x; first < a.rows; first += kTurns * step) {
    const int turns = min(kTurns, (a.rows - first + step - 1) / step);
#pragma unroll 1
    for (int t = 0; t < turns; ++t) {
      const int64_t row = row_of(first + t * step);
      RowSums s{0, 0};
      for (int c = threadIdx.x * kUnit; c < a.cols; c += kWide * kUnit) {
        read(row, c, h, dy);
        weight(c, w);
        s.squares += squares(h, 0);
        s.product += product(dy, w, h, 0);
      }
      s.squares = group_sum<kWide>(s.squares, lds[t % 2][0]);
      s.product = group_sum<kWide>(s.product, lds[t % 2][1]);
      if (threadIdx.x == 0) row_factors(s, a.cols, a.eps, factors[t][0], factors[t][1]);
    }
    __syncthreads();
    for (int c = threadIdx.x * kUnit; c < a.cols; c += kWide * kUnit) {
      const int n = a.cols - c;
      weight(c, w);
      double sum[kUnit] = {};
      if (sizeof(T) == 8 && a.dw && first != blockIdx.x) {
        if (n >= kUnit) {
          __builtin_memcpy(sum, part + c, sizeof(sum));
        } else {
#pragma unroll
          for (int i = 0; i < kUnit - 1; ++i)
            if (i < n) sum[i] = part[c + i];
        }
      }
#pragma unroll 1
      for (int t = 0; t < turns; ++t) {
        const int64_t row = row_of(first + t * step);
        const float m = factors[t][0], k = factors[t][1];
        read(row, c, h, dy);
        float v[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          v[i] = m * (dy[i] * w[i] - h[i] * k);
          sum[i] += dy[i] * (h[i] * m);
        }
        if (a.dh.p) {
          Unit<kAnyDtype> u;
          load_unit<true>(u, a.dh.p, a.dh.dtype, row * a.dh.ld + c, n);
          unit_floats(u, a.dh.dtype, h);
#pragma unroll
          for (int i = 0; i < kUnit; ++i) v[i] += h[i];
        }
        store_unit<true>(a.dx.p, a.dx.dtype, row * a.dx.ld + c, n, v);
      }
      if (!a.dw) continue;
      T v[kUnit];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) v[i] = (T)sum[i];
      if (n >= kUnit) {
        __builtin_memcpy(part + c, v, sizeof(v));
      } else {
#pragma unroll
        for (int i = 0; i < kUnit - 1; ++i)
          if (i < n) part[c + i] = v[i];
      }
    }
  }
}

// dw[c] = sum of the workgroups' parts: 32 columns a workgroup, eight lanes to a part,
// the shares of the parts joined in order.
constexpr int kDwCols = 32;
template <class T>
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const T* part, int parts, int cols, float* dw) {
  constexpr int kShares = 1024 / 8, kGroups = 1024 / kDwCols;
  __shared__ double lds[kShares][kDwCols];
  const int lane = threadIdx.x % 8, share = threadIdx.x / 8;
  const int c = blockIdx.x * kDwCols + lane * 4;
  double v[4] = {};
#pragma unroll 8
  for (int p = share; p < parts; p += kShares) {
    T x[4] = {};
    const T* at = part + (int64_t)p * cols + c;
    if (c + 4 <= cols) {
      __builtin_memcpy(x, at, sizeof(x));
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (c + i < cols) x[i] = at[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += x[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) lds[share][lane * 4 + i] = v[i];
  __syncthreads();
  const int col = threadIdx.x % kDwCols, group = threadIdx.x / kDwCols;
  double sum = 0;
#pragma unroll
  for (int i = 0; i < kShares / kGroups; ++i) sum += lds[group * (kShares / kGroups) + i][col];
  __syncthreads();
  lds[group][col] = sum;
  __syncthreads();
  if (group == 0 && blockIdx.x * kDwCols + col < cols) {
#pragma unroll
    for (int i = 1; i < kGroups; ++i) sum += lds[i][col];
    dw[blockIdx.x * kDwCols + col] = (float)sum;
  }
}

__global__ void __launch_bounds__(256) fill_zero_kernel(float* p, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// The most workgroups of the gradient, so parts of dw's sums: two per CU.  More would
// hide more latency, but their parts cost more (16384 x 6144 bf16, norm and gradient:
// 512 of them 299 us, 1024 314).  Rows past 8192 columns leave room for one per CU.
constexpr int kGradBlocks = 512;

// Calls f(lanes, units, tail) as integral constants for rows of up to MOST columns,
// g() for longer ones.  Lanes that a row fills to two thirds and more, fewer of them with
// more units before more with fewer (bf16 norm of 4000 x 9000 64 us with 512 of three
// against 81 with 1024 of two, 2000 x 14000 49 with 512 of four against 54, 2000 x 20000
// 77 with 1024 of three against 87 with four).  1024 lanes have 128 registers each, of which
// four units of fp32 rows are three short (12 bytes of scratch a lane).
template <int MOST, class F, class H>
void by_shape(int cols, F&& f, H&& g) {
  using std::integral_constant;
  const int units = (cols + kUnit - 1) / kUnit;
  auto at = [&](auto G, auto U) { f(G, U, std::false_type{}); };
  if (cols > MOST) g();
  else if (cols < kUnit) f(integral_constant<int, 4>{}, integral_constant<int, 1>{}, std::true_type{});
  else if (units <= 4) at(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (units <= 8) at(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (units <= 16) at(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (units <= 32) at(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (units <= 64) at(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (units <= 128) at(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (units <= 192) at(integral_constant<int, 64>{}, integral_constant<int, 3>{});
  else if (units <= 256) at(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (units <= 512) at(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (units <= 768) at(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  else if (units <= 1024) at(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else if (units <= 1536) at(integral_constant<int, 512>{}, integral_constant<int, 3>{});
  else if (units <= 2048) at(integral_constant<int, 512>{}, integral_constant<int, 4>{});
  else if constexpr (MOST > 16384) {
    if (units <= 3 * 1024) at(integral_constant<int, 1024>{}, integral_constant<int, 3>{});
    else at(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  }
}

// Calls f of two dtypes as integral constants.
template <class F>
void by_dtypes(int a, int b, F&& f) {
  using F32 = std::integral_constant<int, MOE_DT_F32>;
  using Bf16 = std::integral_constant<int, MOE_DT_BF16>;
  if (a == MOE_DT_F32 && b == MOE_DT_F32) f(F32{}, F32{});
  else if (a == MOE_DT_F32) f(F32{}, Bf16{});
  else if (b == MOE_DT_F32) f(Bf16{}, F32{});
  else f(Bf16{}, Bf16{});
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& args, hipStream_t s) {
  NormArgs a = args;
  a.past_cache = past_cache((int64_t)a.rows * a.cols * ((a.h.p ? element(a.h.dtype) : 0) + (a.y.p ? element(a.y.dtype) : 0)));
  hipError_t e = hipSuccess;
  by_shape<32768>(
      a.cols,
      [&](auto G, auto U, auto T) {
        constexpr int g = decltype(G)::value;
        e = by_runs(a.rows, block_of(g), block_of(g) / g, [&](int first, dim3 grid) {
          a.first = first;
          auto launch = [&](auto X, auto R) {
            hipLaunchKernelGGL((rmsnorm_kernel<decltype(X)::value, decltype(R)::value, g, decltype(U)::value, decltype(T)::value>),
                               grid, dim3(block_of(g)), 0, s, a);
          };
          if constexpr (!decltype(T)::value) {
            using Once = std::integral_constant<int, kBf16Once>;
            if (read_once(a.x, a.rows, a.cols) && read_once(a.res, a.rows, a.cols)) return launch(Once{}, Once{});
          }
          by_dtypes(a.x.dtype, a.res.p ? a.res.dtype : a.x.dtype, launch);
        });
      },
      [&] {
        e = by_runs(a.rows, kWide, 1, [&](int first, dim3 grid) {
          a.first = first;
          hipLaunchKernelGGL(rmsnorm_wide_kernel, grid, dim3(kWide), 0, s, a);
        });
      });
  return e;
}

size_t norm_grad_part_bytes(int rows, int cols) {
  const size_t most = cols > kNormGradCols ? kGradBlocks / 2 * sizeof(double) : kGradBlocks * sizeof(float);
  return std::min(std::max(rows, 1) * (cols > kNormGradCols ? sizeof(double) : sizeof(float)), most) * cols;
}

hipError_t launch_rmsnorm_grad(const NormGradArgs& args, hipStream_t s) {
  NormGradArgs a = args;
  a.past_cache = past_cache((int64_t)a.rows * a.cols * element(a.dx.dtype));
  if (a.rows == 0) {
    hipLaunchKernelGGL(fill_zero_kernel, dim3((a.cols + 255) / 256), dim3(256), 0, s, a.dw, a.cols);
    return hipGetLastError();
  }
  // workgroups of `per` rows at a time, each as many times as the others
  int blocks = 0;
  bool deep = false;           // parts in float64
  auto grid = [&](int per, int most) {
    const int steps = (a.rows + per - 1) / per;
    int turns = (steps + most - 1) / most;
    // few: one workgroup, which needs no launch to join the parts (norm and gradient of 8
    // x 300 rows through Python 13.8 us against 15.5; 8 x 1000 17.9, 8 x 6144 22.1)
    if (a.dw && steps <= (a.cols <= 64 * kUnit ? 8 : 4)) turns = steps;
    return dim3(blocks = (steps + turns - 1) / turns);
  };
  by_shape<kNormGradCols>(
      a.cols,
      [&](auto G, auto U, auto T) {
        auto launch = [&](auto D, auto Y) {
          // bf16 rows of up to 2048 columns by a wave each, without barriers (norm and
          // gradient of 20000 x 2000 129 us against 144); fp32 rows take too many registers
          // for that (8000 x 1600 88 us against 82), and the norm alone has more of them in
          // flight by workgroups (20000 x 2000 60 us against 64)
          constexpr bool wave = kIsBf16<decltype(D)::value> && decltype(G)::value == 256 && decltype(U)::value == 1;
          constexpr int g = wave ? kWave : decltype(G)::value, u = wave ? 4 : decltype(U)::value;
          hipLaunchKernelGGL((rmsnorm_grad_kernel<decltype(D)::value, decltype(Y)::value, g, u, decltype(T)::value>),
                             grid(block_of(g) / g, g > 256 ? kGradBlocks / 2 : kGradBlocks), dim3(block_of(g)), 0, s, a);
        };
        const bool same = a.dx.dtype == a.h.dtype && (a.h.dtype == MOE_DT_F32 || a.w_dtype == MOE_DT_BF16);
        if constexpr (!decltype(T)::value) {
          using Once = std::integral_constant<int, kBf16Once>;
          if (same && read_once(a.h, a.rows, a.cols) && read_once(a.dy, a.rows, a.cols) && read_once(a.dh, a.rows, a.cols))
            return launch(Once{}, Once{});
        }
        if (same) by_dtypes(a.h.dtype, a.dy.dtype, launch);
        else launch(std::integral_constant<int, kAnyDtype>{}, std::integral_constant<int, kAnyDtype>{});
      },
      [&] {
        const dim3 wide = grid(1, kGradBlocks / 2);
        deep = a.rows > kWideTurns * blocks;
        if (deep) hipLaunchKernelGGL(rmsnorm_grad_wide_kernel<double>, wide, dim3(kWide), 0, s, a);
        else hipLaunchKernelGGL(rmsnorm_grad_wide_kernel<float>, wide, dim3(kWide), 0, s, a);
      });
  if (!a.dw || blocks == 1) return hipGetLastError();
  auto join = [&](auto* part) {
    hipLaunchKernelGGL((rmsnorm_dw_kernel<std::remove_pointer_t<decltype(part)>>), dim3((a.cols + kDwCols - 1) / kDwCols), dim3(1024), 0,
                       s, part, blocks, a.cols, a.dw);
  };
  if (deep) join(static_cast<double*>(a.part));
  else join(static_cast<float*>(a.part));
  return hipGetLastError();
}

}  // namespace qmoe
