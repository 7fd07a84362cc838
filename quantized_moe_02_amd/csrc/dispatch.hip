// Tokens' rows into expert order (dispatch), back with weights (collect), and the
// gradient of the way back.
//
//   rows[slot(t, i)] = x[t];  y[t] = add[t] + sum_i w(t, i) rows[slot(t, i)]
//   drows[slot(t, i)] = w(t, i) dy[t],  dw(t, i) = dy[t] . rows[slot(t, i)]
//
// All of it moves bytes and is bound by HBM.  A workgroup goes by tokens, so that a
// token's row is read (written) once and its top_k rows are written (read) where
// inv_perm says; going by slots would read it top_k times.  Long rows: one token a
// workgroup, whose slots are then scalars; a lane has four rows in flight (eight in sums
// of fp32 take 76 registers, 6315 tokens of 11 x 517 40 us against 36; in the gradient
// of bf16 192, 4096 tokens of 8 x 6144 300 us for both calls against 283).  Few tokens of
// the gradient: a workgroup for each pick.  Sums are fp32, in the order of the picks; a
// dot product's lanes meet in a fixed order.
//
// Measured, averages, 8 rows a token, 6144 columns bf16: dispatch of 16384 tokens 333 us
// (1.81 GB, 5.4 TB/s); collect of 4096 103 (503 MB, 4.9 TB/s), its gradient 184 (856 MB,
// 4.7 TB/s); one token's collect 4.0 us, dispatch of 64 in E4M3 4.6.  8000 tokens of 8 x
// 1502: sums 45 us, with their gradient 142 (1504: 135).  Rows that end inside lines cost
// dispatch most, 8 x 2056 73 us against 58 for 2048: the line between two rows is written
// by two workgroups.
#include <algorithm>

#include "rows_device.h"

namespace qmoe {
namespace {

constexpr int kBlock = 256;
// Lanes that leave no CU idle (256 CUs of 512): with fewer the gradient takes a workgroup
// for each pick (sums and gradient of 2 tokens of 8 x 183 in a graph: 17 us with a
// workgroup for a token's picks one after the other, 8 so).
constexpr int64_t kGradFill = 1 << 17;

// The first n (0 < n < 16) of 16 bytes, as runs of eight, four, two and one.
__device__ __forceinline__ void copy_bytes(uint8_t* to, const uint8_t* from, int n) {
  for (int at = 0; at < n;) {
    const int rest = n - at;
    if (rest >= 8) __builtin_memcpy(to + at, from + at, 8), at += 8;
    else if (rest >= 4) __builtin_memcpy(to + at, from + at, 4), at += 4;
    else if (rest >= 2) __builtin_memcpy(to + at, from + at, 2), at += 2;
    else to[at] = from[at], at += 1;
  }
}

struct CopyArgs {
  const uint8_t *x, *x_scale;
  uint8_t *rows, *row_scale;
  int64_t x_pitch, row_pitch;   // bytes
  int row_bytes, scale_bytes;
  int chunks;                   // of 16 bytes a row
  const int32_t* inv;
  int T, K, slots;
};

// Rows as they are, then their scales: chunk `chunks` and the following ones.  A row's
// last chunk ends where the row ends (Span); of less than 16 bytes it goes in pieces.
template <bool LONG>
__global__ void __launch_bounds__(kBlock) dispatch_copy_kernel(CopyArgs a, RowMap m) {
  int t, c;
  locate<LONG>(m, t, c);
  if (t >= a.T) return;
  const int64_t pick = (int64_t)t * a.K;
  if (c < a.chunks && a.row_bytes >= 16) {
    const int at = min(c * 16, a.row_bytes - 16);
    uint4 v;
    __builtin_memcpy(&v, a.x + t * a.x_pitch + at, 16);
    for (int i = 0; i < a.K; ++i) {
      const int slot = a.inv[pick + i];
      if ((unsigned)slot < (unsigned)a.slots) __builtin_memcpy(a.rows + slot * a.row_pitch + at, &v, 16);
    }
    return;
  }
  const bool scale = c >= a.chunks;
  const int at = (scale ? c - a.chunks : c) * 16, bytes = scale ? a.scale_bytes : a.row_bytes;
  if (at >= bytes) return;
  const int64_t x_pitch = scale ? bytes : a.x_pitch, pitch = scale ? bytes : a.row_pitch;
  const uint8_t* from = (scale ? a.x_scale : a.x) + t * x_pitch + at;
  uint8_t* to = (scale ? a.row_scale : a.rows) + at;
  for (int i = 0; i < a.K; ++i) {
    const int slot = a.inv[pick + i];
    if ((unsigned)slot >= (unsigned)a.slots) continue;
    if (bytes - at >= 16) __builtin_memcpy(to + slot * pitch, from, 16);
    else if (bytes - at == 4) __builtin_memcpy(to + slot * pitch, from, 4);
    else copy_bytes(to + slot * pitch, from, bytes - at);
  }
}

// Rows from fp32 to bf16 or back.
template <int DT, bool LONG, bool TAIL>
__global__ void __launch_bounds__(kBlock) dispatch_cast_kernel(DispatchArgs a, RowMap m) {
  int t, unit;
  locate<LONG>(m, t, unit);
  const Span<TAIL> p(unit, a.cols);
  if (t >= a.T || p.n <= 0) return;
  Unit<DT> u;
  float v[kUnit];
  load_unit<TAIL>(u, a.x.p, DT, (int64_t)t * a.x.ld + p.c, p.n);
  unit_floats(u, DT, v);
  for (int i = 0; i < a.K; ++i) {
    const int slot = a.inv[(int64_t)t * a.K + i];
    if ((unsigned)slot >= (unsigned)a.slots) continue;
    store_unit<TAIL>(a.rows.p, DT == MOE_DT_BF16 ? MOE_DT_F32 : MOE_DT_BF16, (int64_t)slot * a.rows.ld + p.c, p.n, v);
  }
}

// Slots of picks [i, i + N) of a token, -1 for those that take no part.
template <int N>
__device__ __forceinline__ void slots_of(const int32_t* inv, int64_t pick, int n, int slots, int (&s)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = j < n ? inv[pick + j] : -1;
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = (unsigned)s[j] < (unsigned)slots ? s[j] : -1;
}

template <int DT, bool LONG, bool TAIL>
__global__ void __launch_bounds__(kBlock) collect_kernel(CollectArgs a, RowMap m) {
  constexpr int N = 4;          // rows in flight
  int t, unit;
  locate<LONG>(m, t, unit);
  const Span<TAIL> p(unit, a.cols);
  if (t >= a.T || p.n <= 0) return;
  float y[kUnit] = {};
  for (int i = 0; i < a.K; i += N) {
    const int64_t pick = (int64_t)t * a.K + i;
    int slot[N];
    slots_of(a.inv, pick, a.K - i, a.slots, slot);
    Unit<DT> u[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (slot[j] >= 0) load_unit<TAIL>(u[j], a.rows.p, kPlain<DT>, (int64_t)slot[j] * a.rows.ld + p.c, p.n);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (slot[j] < 0) continue;
      const float w = a.w ? a.w[pick + j] : 1.0f;
      float v[kUnit];
      unit_floats(u[j], kPlain<DT>, v);
#pragma unroll
      for (int l = 0; l < kUnit; ++l) y[l] = fmaf(w, v[l], y[l]);
    }
  }
  if (a.add.p) {
    Unit<kAnyDtype> u;
    float v[kUnit];
    load_unit<TAIL>(u, a.add.p, a.add.dtype, (int64_t)t * a.add.ld + p.c, p.n);
    unit_floats(u, a.add.dtype, v);
#pragma unroll
    for (int j = 0; j < kUnit; ++j) y[j] += v[j];
  }
  store_unit<TAIL>(a.y.p, a.y.dtype, (int64_t)t * a.y.ld + p.c, p.n, y);
}

// A token's picks [i, i + span) by G lanes that walk along its row (G == 0: by the
// whole workgroup), four picks at a time.
constexpr int kPicks = 4;
template <int DT, int G, bool TAIL>
__global__ void __launch_bounds__(kBlock) collect_grad_kernel(CollectGradArgs a, int span) {
  __shared__ float lds[G ? 1 : kBlock / kWave][kPicks];
  const int lanes = G ? G : blockDim.x;
  const int lane = G ? threadIdx.x % (G ? G : 1) : threadIdx.x;
  const int spans = (a.K + span - 1) / span;
  unsigned at = blockIdx.x;
  if constexpr (G == kWave) at = at * (kBlock / G) + __builtin_amdgcn_readfirstlane(threadIdx.x / G);
  else if constexpr (G != 0) at = at * (kBlock / G) + threadIdx.x / G;
  const int t = (int)(at / (unsigned)spans), begin = (int)(at - (unsigned)t * spans) * span;
  if (t >= a.T) return;
  const int end = min(begin + span, a.K), units = (a.cols + kUnit - 1) / kUnit;
  for (int i = begin; i < end; i += kPicks) {
    const int64_t pick = (int64_t)t * a.K + i;
    int slot[kPicks];
    float w[kPicks], dot[kPicks];
    slots_of(a.inv, pick, end - i, a.slots, slot);
#pragma unroll
    for (int j = 0; j < kPicks; ++j) {
      w[j] = a.w && i + j < end ? a.w[pick + j] : 1.0f;
      dot[j] = 0.0f;
    }
    for (int unit = lane; unit < units; unit += lanes) {
      const Span<TAIL> p(unit, a.cols);
      Unit<kAnyDtype> d;
      Unit<DT> r[kPicks];
      load_unit<TAIL>(d, a.dy.p, a.dy.dtype, (int64_t)t * a.dy.ld + p.c, p.n);
      if (a.dw) {
#pragma unroll
        for (int j = 0; j < kPicks; ++j)
          if (slot[j] >= 0) load_unit<TAIL>(r[j], a.rows.p, DT, (int64_t)slot[j] * a.rows.ld + p.c, p.n);
      }
      float dy[kUnit], v[kUnit];
      unit_floats(d, a.dy.dtype, dy);
#pragma unroll
      for (int j = 0; j < kPicks; ++j) {
        __builtin_amdgcn_sched_barrier(0);   // one pick after the other, for fewer registers
        if (slot[j] < 0) continue;
        if (a.dw) {
          unit_floats(r[j], DT, v);
          if (p.skip == 0) {
#pragma unroll
            for (int l = 0; l < kUnit; ++l) dot[j] = fmaf(dy[l], v[l], dot[j]);
          } else {
#pragma unroll
            for (int l = 0; l < kUnit; ++l) dot[j] = l >= p.skip ? fmaf(dy[l], v[l], dot[j]) : dot[j];
          }
        }
        if (a.drows.p) {
#pragma unroll
          for (int l = 0; l < kUnit; ++l) v[l] = w[j] * dy[l];
          store_unit<TAIL>(a.drows.p, DT, (int64_t)slot[j] * a.drows.ld + p.c, p.n, v);
        }
      }
    }
    if (!a.dw) continue;
#pragma unroll
    for (int j = 0; j < kPicks; ++j) {
      dot[j] = lanes_reduce<(G ? G : kWave)>(dot[j], [](float x, float y) { return x + y; });
      if constexpr (G != 0) {
        if (lane == 0 && i + j < end) a.dw[pick + j] = dot[j];
      } else if ((threadIdx.x & 63) == 0) {
        lds[threadIdx.x >> 6][j] = dot[j];
      }
    }
    if constexpr (G == 0) {
      __syncthreads();
      if (lane < kPicks && i + lane < end) {
        float sum = lds[0][lane];
        for (int v = 1; v < lanes / kWave; ++v) sum += lds[v][lane];
        a.dw[pick + lane] = sum;
      }
      __syncthreads();
    }
  }
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t s) {
  if (a.x.dtype != a.rows.dtype) {
    return by_rows<false>(row_map((a.cols + kUnit - 1) / kUnit, ragged_lines(a.rows.p, a.rows.ld * element(a.rows.dtype))), a.T,
                   a.cols < kUnit, [&](auto L, auto T, dim3 grid, dim3 block, const RowMap& m) {
      constexpr bool l = decltype(L)::value, t = decltype(T)::value;
      if (a.x.dtype == MOE_DT_F32) hipLaunchKernelGGL((dispatch_cast_kernel<MOE_DT_F32, l, t>), grid, block, 0, s, a, m);
      else hipLaunchKernelGGL((dispatch_cast_kernel<MOE_DT_BF16, l, t>), grid, block, 0, s, a, m);
    });
  }
  CopyArgs c{};
  c.x = static_cast<const uint8_t*>(a.x.p);
  c.rows = static_cast<uint8_t*>(a.rows.p);
  c.x_scale = a.x_scale;
  c.row_scale = a.row_scale;
  c.scale_bytes = a.scale_bytes;
  if (a.x.dtype == MOE_DT_MXFP4) {
    c.row_bytes = (a.cols + kMxBlock - 1) / kMxBlock * (kMxBlock / 2);
    c.x_pitch = c.row_pitch = c.row_bytes;
  } else {
    const int size = a.x.dtype == MOE_DT_F32 ? 4 : a.x.dtype == MOE_DT_BF16 ? 2 : 1;
    c.row_bytes = a.cols * size;
    c.x_pitch = a.x.ld * size;
    c.row_pitch = a.rows.ld * size;
  }
  c.chunks = (c.row_bytes + 15) / 16;
  c.inv = a.inv;
  c.T = a.T;
  c.K = a.K;
  c.slots = a.slots;
  return by_rows<false>(row_map(c.chunks + (c.scale_bytes + 15) / 16, ragged_lines(c.rows, c.row_pitch)), a.T, false,
                 [&](auto L, auto, dim3 grid, dim3 block, const RowMap& m) {
    hipLaunchKernelGGL((dispatch_copy_kernel<decltype(L)::value>), grid, block, 0, s, c, m);
  });
}

hipError_t launch_collect(const CollectArgs& a, hipStream_t s) {
  const bool tail = a.cols < kUnit || (a.y.p == a.add.p && a.cols % kUnit != 0);
  // large bf16 rows past the caches, also those that end inside lines (read_once; the same
  // rows again and again, 4096 tokens of 8 x 6144: 81 us against 92, 8000 of 8 x 1502: 45
  // against 50).  Right after the product that writes them, both in all: 2048 x 8 x 6144 120
  // against 124, 8000 x 8 x 2048 153 against 165, 1100 x 8 x 6144 the same, 4096 x 8 x 6144
  // 711 - 718 against 707; after a copy 223 against 239.  Rows of 200 MB that nothing wrote
  // or read in between are slower so (41 against 34).  The gradient reads them as the rest:
  // 276 us for both calls either way.
  const bool once = !tail && a.rows.dtype == MOE_DT_BF16 && (int64_t)a.T * a.K * a.cols * 2 >= kOnceBytes;
  return by_rows<true>(row_map((a.cols + kUnit - 1) / kUnit, false), a.T, tail,
                       [&](auto L, auto T, dim3 grid, dim3 block, const RowMap& m) {
    constexpr bool l = decltype(L)::value, t = decltype(T)::value;
    if constexpr (!t) {
      if (once) {
        hipLaunchKernelGGL((collect_kernel<kBf16Once, l, t>), grid, block, 0, s, a, m);
        return;
      }
    }
    if (a.rows.dtype == MOE_DT_F32) hipLaunchKernelGGL((collect_kernel<MOE_DT_F32, l, t>), grid, block, 0, s, a, m);
    else hipLaunchKernelGGL((collect_kernel<MOE_DT_BF16, l, t>), grid, block, 0, s, a, m);
  });
}

hipError_t launch_collect_grad(const CollectGradArgs& a, hipStream_t s) {
  using std::integral_constant;
  const int chunks = (a.cols + kUnit - 1) / kUnit;
  auto launch = [&](auto D, auto G, auto T) {
    constexpr int g = decltype(G)::value;
    int threads = kBlock, per = g ? kBlock / (g ? g : 1) : 1;
    if constexpr (g == 0) threads = row_map(chunks, false).threads;
    // few tokens: a workgroup for each pick
    const int span = (int64_t)a.T * (g ? g : threads) >= kGradFill ? a.K : 1;
    const int64_t groups = (int64_t)a.T * ((a.K + span - 1) / span);
    hipLaunchKernelGGL((collect_grad_kernel<decltype(D)::value, g, decltype(T)::value>), dim3((unsigned)((groups + per - 1) / per)),
                       dim3(threads), 0, s, a, span);
  };
  auto by_lanes = [&](auto D) {
    // over the rows themselves a row's last lane must not read what the lane before it wrote
    const bool tail = a.cols < kUnit || (a.rows.p == a.drows.p && a.cols % kUnit != 0);
    auto lanes = [&](auto T) {
      if (chunks <= 8) launch(D, integral_constant<int, 8>{}, T);
      else if (chunks <= 16) launch(D, integral_constant<int, 16>{}, T);
      else if (chunks <= 64) launch(D, integral_constant<int, 64>{}, T);
      else launch(D, integral_constant<int, 0>{}, T);
    };
    if (tail) lanes(std::true_type{});
    else lanes(std::false_type{});
  };
  if (a.rows.dtype == MOE_DT_F32) by_lanes(integral_constant<int, MOE_DT_F32>{});
  else by_lanes(integral_constant<int, MOE_DT_BF16>{});
  return hipGetLastError();
}

}  // namespace qmoe
