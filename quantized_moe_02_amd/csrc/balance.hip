// Balance loss of the router, its per-expert counts and its gradient.
//
// A token's shares are p = y / sum y with y = exp(l) (softmax) or y =
// sigmoid(l).  Both only depend on l up to a factor of y: the softmax takes
// the row's largest logit out, and so does the sigmoid where every logit is
// below -64, where sigmoid(l) = exp(l) to the last bit and could underflow
// throughout.  Its slope d log y / dl is 1 or sigmoid(-l).
//
// A lane holds four experts of a token, so a token takes the 4 to 64 lanes that
// its experts fill (LPT) and a wave several small tokens; sums and maxima over
// a token cross lanes within them.  Everything is one pass over the logits,
// bound by HBM: four rows per lane are requested at a time.
//
// Forward: the tokens are cut into chunks, one workgroup each; it counts the
// picks and sums the shares of each sequence that its chunk touches and writes
// them to slot chunk + sequence (both ascend along the tokens, so the slots of
// different pairs differ).  A second launch adds a sequence's partials in
// order, 32 experts per workgroup, a third one the loss (a workgroup that finds
// itself the last to finish would have to publish its part device-wide first,
// which took 14 us for 384 workgroups).  No atomics on floats: the same bits
// every time.  Sums within a chunk are fp32, across chunks and for the loss
// float64.
//
// Shares come from the hardware's exp and reciprocal: an exponential's argument is
// rounded at its own magnitude, so a share is off by up to (4 max|l| + 40) 2^-24 of
// itself.
//
// Measured, averages, 131072 tokens of 256 fp32 logits in 48 sequences: 33 us for the
// shares (4.2 TB/s read), 6 + 5 us for the sums, 55 us for the gradient (5 TB/s
// read and written): bound by HBM.  bf16 logits: 37 us for the shares and 48 for the
// gradient, half the bytes, so bound by the exponentials and sums beside them.  37
// tokens of 16 experts: 4.2 and 3.9 us, one launch each, bound by latency.  262144
// tokens of 256 experts in 4096 sequences: 121 us for the loss and 132 for the gradient
// (48 sequences: 70 and 131), in 65536: 1120 and 230, the sequences of a chunk and the
// parts of the loss coming one after the other; 65535 empty sequences between two
// tokens of one chunk are read one by one, 14 ms.
#include <algorithm>

#include "operators_internal.h"
#include "qmoe_device.h"

namespace qmoe {
namespace {

constexpr int kMaxE = 256;
constexpr int kMaxChunk = 256;   // MOE_MAX_TOKENS / 1024
constexpr int kRows = 4;         // rows in flight per lane
constexpr int kSliceE = 32;      // experts per workgroup of the second launch
constexpr int kSlices = 8;       // shares of a sequence's chunks in it

template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  v += dppf<kDppXor1>(v);
  v += dppf<kDppXor2>(v);
  if constexpr (LPT >= 8) v += dppf<kDppHalfMirror>(v);
  if constexpr (LPT >= 16) v += dppf<kDppMirror>(v);
  if constexpr (LPT >= 32) v = swap16_sum(v);
  if constexpr (LPT >= 64) v = swap32_sum(v);
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dppf<kDppXor1>(v));
  v = fmaxf(v, dppf<kDppXor2>(v));
  if constexpr (LPT >= 8) v = fmaxf(v, dppf<kDppHalfMirror>(v));
  if constexpr (LPT >= 16) v = fmaxf(v, dppf<kDppMirror>(v));
  if constexpr (LPT >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LPT >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}

// Offset of sequence s, clamped to the tokens.
__device__ __forceinline__ int seq_at(const BalanceArgs& a, int s) {
  return a.seq ? min(max(a.seq[s], 0), a.T) : (s == 0 ? 0 : a.T);
}

// First sequence that ends after token t (S if none).
__device__ __forceinline__ int seq_of(const BalanceArgs& a, int t) {
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (seq_at(a, m + 1) > t) hi = m;
    else lo = m + 1;
  }
  return lo;
}

// Logits of token t at experts e .. e + 3, -inf past E.  VEC: E % 4 == 0.
template <bool BF16, bool VEC>
__device__ __forceinline__ float4 load_row(const BalanceArgs& a, int t, int e) {
  const float none = -INFINITY;
  const int64_t i = (int64_t)t * a.E + e;
  float4 v = make_float4(none, none, none, none);
  if constexpr (VEC) {
    if (e < a.E) {
      if constexpr (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + i);
        v = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
      } else {
        v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + i);
      }
    }
  } else {
    auto at = [&](int j) {
      if (e + j >= a.E) return none;
      if constexpr (BF16) return bf16_lo(static_cast<const uint16_t*>(a.logits)[i + j]);
      return static_cast<const float*>(a.logits)[i + j];
    };
    v = make_float4(at(0), at(1), at(2), at(3));
  }
  return v;
}

// Shares of the token whose logits the LPT lanes of a group hold; with SLOPE
// also d log y / dl.
template <int LPT, bool SIGMOID, bool SLOPE>
__device__ __forceinline__ void shares(const float4& l4, float (&p)[4], float (&d)[4]) {
  const float l[4] = {l4.x, l4.y, l4.z, l4.w};
  const float top = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
  if constexpr (SIGMOID) {
    // lanes of groups with a logit above -64
    uint64_t high = __ballot(top > -64.0f);
    if constexpr (LPT < 64) {
      const int g0 = (int)(threadIdx.x & 63) & ~(LPT - 1);
      high = (high >> g0) & ((1ull << LPT) - 1);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = __expf(-fabsf(l[j]));
      const float r = __builtin_amdgcn_rcpf(1.0f + x);
      p[j] = l[j] >= 0.0f ? r : x * r;
      if constexpr (SLOPE) d[j] = l[j] >= 0.0f ? x * r : r;
    }
    if (__any(high == 0)) {
      const float m = group_max<LPT>(top);
      if (high == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = __expf(l[j] - m);
      }
    }
  } else {
    const float m = group_max<LPT>(top);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p[j] = __expf(l[j] - m);
      if constexpr (SLOPE) d[j] = 1.0f;
    }
  }
  const float z = 1.0f / group_sum<LPT>((p[0] + p[1]) + (p[2] + p[3]));
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] *= z;
}

// Sum of v over the workgroup's 256 threads, to every thread.
__device__ __forceinline__ double block_sum(double v, double* buf) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  return (buf[0] + buf[1]) + (buf[2] + buf[3]);
}

// ONE: a single chunk; the workgroup goes through every sequence and writes
// the results themselves.
template <int LPT, bool SIGMOID, bool BF16, bool VEC, bool ONE>
__global__ void __launch_bounds__(256) balance_partial_kernel(BalanceArgs a, int chunk) {
  constexpr int TPW = 64 / LPT;   // tokens per wave
  __shared__ __attribute__((aligned(16))) float sp[4 * TPW][LPT * 4];
  __shared__ int sc[kMaxE], sn, sk;
  __shared__ uint8_t routed[kMaxChunk];
  __shared__ double buf[4];
  double loss = 0.0;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int group = wv * TPW + lane / LPT, e0 = (lane % LPT) * 4;
  const int t0 = blockIdx.x * chunk, t1 = min(a.T, t0 + chunk);
  for (int s = ONE ? 0 : seq_of(a, t0); s < a.S; ++s) {
    const int lo = max(t0, seq_at(a, s)), hi = min(t1, seq_at(a, s + 1));
    if constexpr (ONE) {
      if (lo >= hi) {   // no tokens
        if (tid < a.E) a.counts[(int64_t)s * a.E + tid] = 0;
        if (tid == 0) a.tokens[s] = 0;
        continue;
      }
    } else {
      if (lo >= t1) break;
      if (lo >= hi) continue;
    }
    sc[tid] = 0;
    routed[tid] = 0;
    if (tid == 0) sn = sk = 0;
    __syncthreads();
    const int picks = (hi - lo) * a.K;
    for (int i = tid; i < picks; i += 256) {
      const int id = a.ids[(int64_t)lo * a.K + i];
      if (id >= 0 && id < a.E) {
        atomicAdd(&sc[id], 1);
        routed[i / a.K] = 1;
      }
    }
    __syncthreads();
    {
      const uint64_t on = __ballot(tid < hi - lo && routed[tid]);
      int k = tid < a.E ? sc[tid] : 0;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) k += __shfl_xor(k, o, 64);
      if (lane == 0) {
        atomicAdd(&sn, __popcll(on));
        atomicAdd(&sk, k);
      }
    }
    float acc[4] = {};
    for (int b = lo; b < hi; b += 4 * TPW * kRows) {
      float4 l[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) l[u] = load_row<BF16, VEC>(a, min(b + u * 4 * TPW + group, hi - 1), e0);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int t = b + u * 4 * TPW + group;
        float p[4], d[4];
        shares<LPT, SIGMOID, false>(l[u], p, d);
        const bool on = t < hi && routed[min(t, hi - 1) - lo];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += on ? p[j] : 0.0f;
      }
    }
    *reinterpret_cast<float4*>(&sp[group][e0]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    float t = 0.0f;
    if (tid < a.E) {
#pragma unroll
      for (int i = 0; i < 4 * TPW; ++i) t += sp[i][tid];
    }
    if constexpr (ONE) {
      if (tid < a.E) a.counts[(int64_t)s * a.E + tid] = sc[tid];
      if (tid == 0) a.tokens[s] = sn;
      const double v = block_sum(tid < a.E ? (double)t * sc[tid] : 0.0, buf);
      if (sn > 0) loss += v * a.E / ((double)sn * sk);
    } else {
      const int64_t slot = (int64_t)blockIdx.x + s;
      if (tid < a.E) {
        a.part_p[slot * a.E + tid] = t;
        a.part_c[slot * a.E + tid] = sc[tid];
      }
      if (tid == 0) {
        a.part_n[slot] = sn;
        a.part_k[slot] = sk;
      }
    }
    __syncthreads();
  }
  if constexpr (ONE) {
    if (tid == 0) *a.loss = (float)(loss * a.coef / a.S);
  }
}

// One workgroup: 32 experts of one sequence, eight threads per expert, each a
// range of the chunks.
__global__ void __launch_bounds__(256) balance_reduce_kernel(BalanceArgs a, int chunk, int slices) {
  __shared__ double rp[kSlices][kSliceE];
  __shared__ int rc[kSlices][kSliceE], rn[256], rk[256];
  const int s = blockIdx.x / slices, part = blockIdx.x - s * slices;
  const int tid = threadIdx.x, x = tid % kSliceE, y = tid / kSliceE;
  const int e = part * kSliceE + x;
  const int lo = seq_at(a, s), hi = seq_at(a, s + 1);
  const int c0 = lo / chunk, nc = hi > lo ? (hi - 1) / chunk - c0 + 1 : 0;
  double p = 0.0;
  int c = 0, n = 0, picks = 0;
  const int64_t first = (int64_t)c0 + s;
  if (e < a.E) {
    const int per = (nc + kSlices - 1) / kSlices;
    const int k1 = min(nc, (y + 1) * per);
#pragma unroll 8
    for (int k = y * per; k < k1; ++k) {
      p += (double)a.part_p[(first + k) * a.E + e];
      c += a.part_c[(first + k) * a.E + e];
    }
  }
  for (int k = tid; k < nc; k += 256) {
    n += a.part_n[first + k];
    picks += a.part_k[first + k];
  }
  rp[y][x] = p;
  rc[y][x] = c;
  rn[tid] = n;
  rk[tid] = picks;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) {
      rn[tid] += rn[tid + o];
      rk[tid] += rk[tid + o];
    }
    __syncthreads();
  }
  if (y == 0) {
#pragma unroll
    for (int i = 1; i < kSlices; ++i) {
      p += rp[i][x];
      c += rc[i][x];
    }
    if (e < a.E) a.counts[(int64_t)s * a.E + e] = c;
    rp[0][x] = p * c;
  }
  __syncthreads();
  if (tid == 0) {
    double t = 0.0;
    for (int i = 0; i < kSliceE; ++i) t += rp[0][i];
    if (part == 0) a.tokens[s] = rn[0];
    // these experts' part of sum f P
    t = rn[0] > 0 ? t * a.E / ((double)rn[0] * rk[0]) : 0.0;
    a.seq_loss[blockIdx.x] = t;
  }
}

// One workgroup: the loss from its n parts.
__global__ void __launch_bounds__(256) balance_loss_kernel(BalanceArgs a, int n) {
  __shared__ double buf[4];
  double t = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += 256) t += a.seq_loss[i];
  t = block_sum(t, buf);
  if (threadIdx.x == 0) *a.loss = (float)(t * a.coef / a.S);
}

// A wave takes `per` consecutive tokens (a multiple of TPW * kRows).
template <int LPT, bool SIGMOID, bool BF16, bool VEC>
__global__ void __launch_bounds__(256) balance_grad_kernel(BalanceArgs a, int per) {
  constexpr int TPW = 64 / LPT;
  const int lane = threadIdx.x & 63, group = lane / LPT, e0 = (lane % LPT) * 4;
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t w0 = (int64_t)wave * per;
  if (w0 >= a.T) return;
  const int t0 = (int)w0, t1 = min(a.T, t0 + per);
  const double up = a.dloss ? (double)*a.dloss : 1.0;
  float f[4] = {}, scale = 0.0f;
  int s = -1, s_end = -1;   // the sequence that f and scale belong to
  for (int b = t0; b < t1; b += TPW * kRows) {
    float4 l[kRows];
    bool on[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int t = min(b + u * TPW + group, t1 - 1);
      l[u] = load_row<BF16, VEC>(a, t, e0);
      bool any = false;
      for (int i = lane % LPT; i < a.K; i += LPT) {
        const int id = a.ids[(int64_t)t * a.K + i];
        any |= id >= 0 && id < a.E;
      }
      on[u] = any;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int t = min(b + u * TPW + group, t1 - 1);
      uint64_t hit = __ballot(on[u]);
      if constexpr (LPT < 64) hit = (hit >> (lane & ~(LPT - 1))) & ((1ull << LPT) - 1);
      if (__any(t >= s_end)) {
        if (t >= s_end) {
          s = seq_of(a, t);
          s_end = s < a.S ? seq_at(a, s + 1) : a.T;
        }
        float c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = e0 + j < a.E && s < a.S ? (float)a.counts[(int64_t)s * a.E + e0 + j] : 0.0f;
        // a sequence holds at most 2^22 picks: the sum is exact in fp32
        const float picks = group_sum<LPT>((c[0] + c[1]) + (c[2] + c[3]));
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = (float)a.E * c[j] / picks;
        scale = s < a.S ? (float)((double)a.coef * up / ((double)a.S * a.tokens[s])) : 0.0f;
      }
      float p[4], d[4], g[4];
      shares<LPT, SIGMOID, true>(l[u], p, d);
      const float dot = group_sum<LPT>((f[0] * p[0] + f[1] * p[1]) + (f[2] * p[2] + f[3] * p[3]));
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = hit != 0 && s < a.S ? scale * p[j] * (f[j] - dot) * d[j] : 0.0f;
      if (b + u * TPW + group < t1) {
        const int64_t i = (int64_t)t * a.E + e0;
        if constexpr (VEC) {
          if (e0 < a.E) {
            if constexpr (BF16) {
              typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
              *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(a.dlogits) + i) = bf16x4{(__bf16)g[0], (__bf16)g[1], (__bf16)g[2], (__bf16)g[3]};
            } else {
              *reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + i) = make_float4(g[0], g[1], g[2], g[3]);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (e0 + j < a.E) {
              if constexpr (BF16) static_cast<__bf16*>(a.dlogits)[i + j] = (__bf16)g[j];
              else static_cast<float*>(a.dlogits)[i + j] = g[j];
            }
          }
        }
      }
    }
  }
}

// Calls f(LPT, SIGMOID, BF16, VEC) as integral constants.
template <class F>
void dispatch(const BalanceArgs& a, F&& f) {
  auto with = [&](auto L) {
    auto types = [&](auto S) {
      const bool vec = a.E % 4 == 0;
      if (a.bf16 && vec) f(L, S, std::true_type{}, std::true_type{});
      else if (a.bf16) f(L, S, std::true_type{}, std::false_type{});
      else if (vec) f(L, S, std::false_type{}, std::true_type{});
      else f(L, S, std::false_type{}, std::false_type{});
    };
    if (a.sigmoid) types(std::true_type{});
    else types(std::false_type{});
  };
  if (a.E <= 16) with(std::integral_constant<int, 4>{});
  else if (a.E <= 32) with(std::integral_constant<int, 8>{});
  else if (a.E <= 64) with(std::integral_constant<int, 16>{});
  else if (a.E <= 128) with(std::integral_constant<int, 32>{});
  else with(std::integral_constant<int, 64>{});
}

}  // namespace

// Tokens per chunk: at most 1024 chunks where that leaves 32 tokens or more; down
// to 2 where sequences are short, since a workgroup takes its chunk's sequences
// one after the other (206 tokens in 39 sequences, loss and gradient: 22 us, with
// 32 tokens 38).
int balance_chunk(int T, int S) {
  return std::min(kMaxChunk, std::max((T + 1023) / 1024, std::min(32, std::max(2, T / S / 4))));
}
// Chunks that T tokens or fewer make at most: 1024 of 32 tokens or more; of c < 32
// tokens, which t < 4 S (c + 1) tokens come in, at most 4 S (c + 1) / c <= 6 S, and
// no more than half of 32768.
int balance_max_chunks(int T, int S) {
  return std::min((T + 1) / 2, std::max(1024, std::min(16384, 6 * S)));
}
int balance_slices(int E) { return (E + kSliceE - 1) / kSliceE; }

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  // few tokens of few sequences: one workgroup ends before two more launches (loss
  // and gradient of 37 tokens, 4 sequences: 17 us against 21; 100 tokens, 4
  // sequences: 23 against 20)
  if (a.T <= 128 && a.S <= 4 && a.T * a.S <= 256) {
    dispatch(a, [&](auto L, auto S, auto B, auto V) {
      hipLaunchKernelGGL((balance_partial_kernel<decltype(L)::value, decltype(S)::value, decltype(B)::value, decltype(V)::value, true>),
                         dim3(1), dim3(256), 0, s, a, kMaxChunk);
    });
    return hipGetLastError();
  }
  const int chunk = balance_chunk(a.T, a.S), slices = balance_slices(a.E);
  hipError_t e;
  if (a.T > 0) {
    dispatch(a, [&](auto L, auto S, auto B, auto V) {
      hipLaunchKernelGGL((balance_partial_kernel<decltype(L)::value, decltype(S)::value, decltype(B)::value, decltype(V)::value, false>),
                         dim3((a.T + chunk - 1) / chunk), dim3(256), 0, s, a, chunk);
    });
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL(balance_reduce_kernel, dim3((unsigned)a.S * slices), dim3(256), 0, s, a, chunk, slices);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(256), 0, s, a, a.S * slices);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceArgs& a, hipStream_t s) {
  dispatch(a, [&](auto L, auto S, auto B, auto V) {
    constexpr int step = 64 / decltype(L)::value * kRows;
    // eight waves per SIMD where there are tokens for them
    const int per = std::max(1, (a.T + 8191) / 8192 + step - 1) / step * step;
    const int waves = (a.T + per - 1) / per;
    hipLaunchKernelGGL((balance_grad_kernel<decltype(L)::value, decltype(S)::value, decltype(B)::value, decltype(V)::value>),
                       dim3((waves + 3) / 4), dim3(256), 0, s, a, per);
  });
  return hipGetLastError();
}

}  // namespace qmoe
