// Balance loss of the router, its per-expert counts and its gradient.
//
// With a = l (softmax) or log sigmoid(l) (sigmoid), a token's shares are
// p = softmax(a) either way: sigmoid(l) / sum sigmoid(l) = exp(a) / sum
// exp(a), so subtracting the row's largest a keeps both from overflowing and
// from 0 / 0 where every sigmoid underflows.  da/dl = 1 or sigmoid(-l).
//
// Forward: the tokens are cut into chunks; a workgroup sums the shares and
// counts the picks of each sequence that its chunk touches and writes the
// partial sums to slot chunk + sequence (both ascend along the tokens, so the
// slots of different pairs differ).  A second launch, one workgroup per
// sequence, adds a sequence's partials in order; the last workgroup to finish
// adds the sequences' losses.  No atomics on floats: the same bits every time.
// Sums within a chunk are fp32, across chunks and for the loss float64.
#include "operators_internal.h"
#include "qmoe_device.h"

namespace qmoe {
namespace {

constexpr int kMaxE = 256;
constexpr int kPer = kMaxE / kWave;   // experts per lane: lane + 64 j

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

__device__ __forceinline__ float load_logit(const BalanceArgs& a, int64_t i) {
  return a.bf16 ? __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.logits)[i] << 16)
                : static_cast<const float*>(a.logits)[i];
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

// Lane i < K: pick i of token t (-1 beyond); the token is routed if any lane has one.
__device__ __forceinline__ int load_pick(const BalanceArgs& a, int t, int lane) {
  const int id = lane < a.K ? a.ids[(int64_t)t * a.K + lane] : -1;
  return id >= 0 && id < a.E ? id : -1;
}

// The token's shares at experts lane + 64 j (0 past E), and d of its logits.
__device__ __forceinline__ void shares(const BalanceArgs& a, int t, int lane, float (&p)[kPer], float (&d)[kPer]) {
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane + 64 * j;
    p[j] = -INFINITY;
    d[j] = 1.0f;
    if (e < a.E) {
      const float l = load_logit(a, (int64_t)t * a.E + e);
      p[j] = l;
      if (a.sigmoid) {
        const float x = expf(-fabsf(l));
        p[j] = fminf(l, 0.0f) - log1pf(x);
        d[j] = (l > 0.0f ? x : 1.0f) / (1.0f + x);
        if (l != l) p[j] = l;   // fminf drops the NaN
      }
    }
    m = fmaxf(m, p[j]);
  }
  m = wave_max(m);
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    p[j] = lane + 64 * j < a.E ? expf(p[j] - m) : 0.0f;
    z += p[j];
  }
  z = wave_sum(z);
#pragma unroll
  for (int j = 0; j < kPer; ++j) p[j] /= z;
}

__global__ void __launch_bounds__(256) balance_partial_kernel(BalanceArgs a, int chunk) {
  __shared__ float sp[4][kMaxE];
  __shared__ int sc[kMaxE], sn;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  const int t0 = blockIdx.x * chunk, t1 = min(a.T, t0 + chunk);
  if (t0 >= t1) return;
  for (int s = seq_of(a, t0); s < a.S; ++s) {
    const int lo = max(t0, seq_at(a, s)), hi = min(t1, seq_at(a, s + 1));
    if (lo >= t1) break;
    if (lo >= hi) continue;
    __syncthreads();
    sc[threadIdx.x] = 0;
    if (threadIdx.x == 0) sn = 0;
    __syncthreads();
    float acc[kPer] = {};
    int n = 0;
    for (int t = lo + wv; t < hi; t += 4) {
      const int id = load_pick(a, t, lane);
      if (!__any(id >= 0)) continue;
      ++n;
      if (id >= 0) atomicAdd(&sc[id], 1);
      float p[kPer], d[kPer];
      shares(a, t, lane, p, d);
#pragma unroll
      for (int j = 0; j < kPer; ++j) acc[j] += p[j];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) sp[wv][lane + 64 * j] = acc[j];
    if (lane == 0) atomicAdd(&sn, n);
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    const int e = threadIdx.x;
    if (e < a.E) {
      a.part_p[slot * a.E + e] = (sp[0][e] + sp[1][e]) + (sp[2][e] + sp[3][e]);
      a.part_c[slot * a.E + e] = sc[e];
    }
    if (e == 0) a.part_n[slot] = sn;
  }
}

__global__ void __launch_bounds__(256) balance_reduce_kernel(BalanceArgs a, int chunk) {
  __shared__ double red[256];
  __shared__ int redi[256];
  __shared__ bool last;
  const int s = blockIdx.x, e = threadIdx.x;
  const int lo = seq_at(a, s), hi = seq_at(a, s + 1);
  double p = 0.0;
  int c = 0, n = 0;
  if (hi > lo) {
    const int c0 = lo / chunk, c1 = (hi - 1) / chunk;
    for (int k = c0; k <= c1; ++k) {
      const int64_t slot = (int64_t)k + s;
      if (e < a.E) {
        p += (double)a.part_p[slot * a.E + e];
        c += a.part_c[slot * a.E + e];
      }
      n += a.part_n[slot];
    }
  }
  if (e < a.E) a.counts[(int64_t)s * a.E + e] = c;
  if (e == 0) a.tokens[s] = n;
  red[e] = p * c;
  redi[e] = c;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (e < o) {
      red[e] += red[e + o];
      redi[e] += redi[e + o];
    }
    __syncthreads();
  }
  if (e == 0) {
    const double l = n > 0 ? red[0] * a.E / ((double)redi[0] * n) : 0.0;
    __hip_atomic_store(&a.seq_loss[s], l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.S - 1;
  }
  __syncthreads();
  if (!last) return;
  double t = 0.0;
  for (int i = e; i < a.S; i += 256) t += __hip_atomic_load(&a.seq_loss[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  red[e] = t;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (e < o) red[e] += red[e + o];
    __syncthreads();
  }
  if (e == 0) *a.loss = (float)(red[0] * a.coef / a.S);
}

// One wave per token.
__global__ void __launch_bounds__(256) balance_grad_kernel(BalanceArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int s = seq_of(a, t);
  float g[kPer] = {};
  if (__any(load_pick(a, t, lane) >= 0) && s < a.S) {
    float p[kPer], d[kPer], f[kPer];
    shares(a, t, lane, p, d);
    int c[kPer], tot = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = lane + 64 * j;
      c[j] = e < a.E ? a.counts[(int64_t)s * a.E + e] : 0;
      tot += c[j];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) tot += __shfl_xor(tot, o, 64);
    const float scale = (float)((double)a.coef * (a.dloss ? (double)*a.dloss : 1.0) / ((double)a.S * a.tokens[s]));
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      f[j] = (float)a.E * (float)c[j] / (float)tot;
      dot += f[j] * p[j];
    }
    dot = wave_sum(dot);
#pragma unroll
    for (int j = 0; j < kPer; ++j) g[j] = scale * p[j] * (f[j] - dot) * d[j];
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane + 64 * j;
    if (e < a.E) {
      if (a.bf16) static_cast<__bf16*>(a.dlogits)[(int64_t)t * a.E + e] = (__bf16)g[j];
      else static_cast<float*>(a.dlogits)[(int64_t)t * a.E + e] = g[j];
    }
  }
}

}  // namespace

// At least 64 tokens a chunk, and at most 1024 chunks.
int balance_chunk(int T) { return T <= 65536 ? 64 : (T + 1023) / 1024; }

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  const int chunk = balance_chunk(a.T);
  const int nc = (a.T + chunk - 1) / chunk;
  // at least one workgroup: it clears the ticket
  hipLaunchKernelGGL(balance_partial_kernel, dim3(nc > 0 ? nc : 1), dim3(256), 0, s, a, chunk);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_reduce_kernel, dim3(a.S), dim3(256), 0, s, a, chunk);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(balance_grad_kernel, dim3((a.T + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qmoe
