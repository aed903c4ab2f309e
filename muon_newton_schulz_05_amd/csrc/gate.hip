// gate.hip -- a router's gate (the largest logits of each token and their softmax weights), its balance loss
// with the counts of every expert, and both gradients.
//
// A token's logits lie in the registers of L lanes, V consecutive ones in each (L V >= experts), so that a wave
// holds 64 / L tokens and a reduction over experts is log2 L steps between lanes.
//
//  - gate: the choice takes `top` rounds of a maximum over keys, integers in the order of the values (ties: the lower
//    index first).  weights w_j = e^(z_j - m) / sum, the sum over all experts or, normalised, over the chosen.
//    Normalised, dz_j = w_j (dw_j - sum_i w_i dw_i) at the chosen; otherwise that with p_e in place of w for
//    every expert.
//  - balance loss E sum_e f_e P_e with f_e = c_e / (T top) and P_e = mean_t p_te: each wave adds up its tokens'
//    probabilities in registers, workgroups leave partial sums, the join adds them in order.  c_e are integer
//    counts, exact in any order, so LDS atomics may make them.  dz_te = dloss E / T p_te (f_e - sum_i p_ti f_i).
//
// What bounds them.  gate: per choice a maximum in the lane, log2 L steps between lanes and the taking out of the key, which
// every lane repeats whether it held the choice or not.  balance loss: at most 256 workgroups of 16 waves, half of what the card
// holds, with one exponential a logit between their loads, and a join by one workgroup; the gradient makes the softmax anew.  In
// us: gate 16384 x 64, top 8, bf16 5.9, its gradient 4.9; 65536 x 256 33 and 15 (over all experts 24), float32 41 and
// 20; balance loss of 65536 x 256, bf16, 17 and 8.5 for the join (512 KiB of sums), its gradient 23 (2.9 TB/s); 64 x 64 4 each.
//
// A masked token takes no part in anything, whatever its logits hold.  Logits of -inf are experts that cannot be
// chosen: their probability is zero, and a row of nothing else has no choice and no probabilities.
#include <algorithm>
#include <type_traits>

#include "act.h"
#include "gate.h"
#include "group.h"
#include "raw.h"

namespace muon {
namespace {

// e^x for x <= 0 to about 2^-22 of itself: the product's rounding, which the hardware's exp2 would turn into |x| 2^-24,
// is carried.  Below -200 it is zero; NaN stays NaN.
__device__ __forceinline__ float exp_f(float x) {
  x = x < -200.f ? -200.f : x;
  constexpr float kLog2e = 1.44269504f, kRest = 1.92596299e-8f;  // log2(e) and what float32 leaves of it
  const float t = x * kLog2e, lo = fmaf(x, kRest, fmaf(x, kLog2e, -t));
  return __builtin_amdgcn_exp2f(t) * fmaf(lo, 0.693147181f, 1.f);
}

constexpr float kInf = __builtin_huge_valf();

// Integers in the order of the values: NaN first, -inf and what is not there (0) never chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 is 0
  if (v != v) return 0xffffffffu;
  if (v == -kInf) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {  // any NaN for NaN
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The next choice of a token: the largest of its keys, the lowest expert among equals, which leaves the keys.  A bfloat16
// value's key has 16 bits, which leaves room for the expert: one maximum then finds both.  A
// float32 value takes a second reduction, of the experts that have it.
template <typename T> struct Choice;
template <> struct Choice<uint16_t> {
  static __device__ __forceinline__ uint32_t key(float v, int e) {
    const uint32_t k = order_key(v);
    return k ? (k & 0xffff0000u) | (uint32_t)(kGateMaxExperts - 1 - e) : 0u;
  }
  template <int L, int V>
  static __device__ __forceinline__ bool next(uint32_t (&key)[V], int, float& v, int& e) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    best = group_max<L>(best);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = key[i] == best ? 0u : key[i];
    e = kGateMaxExperts - 1 - (int)(best & (kGateMaxExperts - 1));
    // The low bits that a negative value's key would have are ones.
    v = key_value(best & 0x80000000u ? best & 0xffff0000u : best | 0xffffu);
    if (best >= 0xffff0000u) v = __builtin_nanf("");
    return best != 0u;
  }
};
template <> struct Choice<float> {
  static __device__ __forceinline__ uint32_t key(float v, int) { return order_key(v); }
  template <int L, int V>
  static __device__ __forceinline__ bool next(uint32_t (&key)[V], int first, float& v, int& e) {
    uint32_t best = key[0], at = ~0u;
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    best = group_max<L>(best);
#pragma unroll
    for (int i = 0; i < V; ++i) at = min(at, key[i] == best ? (uint32_t)(first + i) : ~0u);
    at = group_min<L>(at);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = (uint32_t)(first + i) == at ? 0u : key[i];
    e = (int)at;
    v = key_value(best);
    return best != 0u;
  }
};

// The tokens of a wave: lane l of L holds experts l V .. l V + V - 1.
template <typename T, int L, int V>
struct Row {
  int l, n;  // lane of the token; its experts
  __device__ __forceinline__ Row(int experts) {
    l = threadIdx.x & (L - 1);
    n = min(max(experts - l * V, 0), V);
  }
  // The lane's logits as they lie in memory, and as values: -inf where there is no expert, or no token.
  __device__ __forceinline__ void fetch(const T* row, bool in, Raw<T> (&raw)[V / 8]) const {
#pragma unroll
    for (int c = 0; c < V; c += 8) raw[c / 8].load(row + l * V + c, in ? min(n - c, 8) : 0);
  }
  __device__ __forceinline__ void values(const Raw<T> (&raw)[V / 8], bool in, float (&z)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = in && i < n ? raw[i / 8].at(i % 8) : -kInf;
  }
  __device__ __forceinline__ void load(const T* row, bool in, float (&z)[V]) const {
    Raw<T> raw[V / 8];
    fetch(row, in, raw);
    values(raw, in, z);
  }
  __device__ __forceinline__ void store(T* row, bool in, const float (&z)[V]) const {
#pragma unroll
    for (int c = 0; c < V; c += 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = z[c + i];
      store8(row + l * V + c, in ? min(n - c, 8) : 0, v);
    }
  }
  // z to probabilities; all zero where every logit is -inf.  (The largest value leaves NaN out, which comes back in
  // through its own exponential and the sum.)
  __device__ __forceinline__ void softmax(float (&z)[V]) const {
    float m = z[0], sum = 0.f;
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, z[i]);
    m = group_max<L>(m);
    m = m == -kInf ? 0.f : m;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      z[i] = exp_f(z[i] - m);
      sum += z[i];
    }
    sum = group_sum<L>(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] *= inv;
  }
};

// The tokens of one workgroup, from `first` on.
template <typename T, int L, int V>
__device__ __forceinline__ void gate_tokens(const GateArgs& a, int64_t first) {
  const Row<T, L, V> r(a.experts);
  const int64_t t = first + threadIdx.x / L;
  const bool in = t < a.tokens, on = in && (!a.mask || a.mask[t]);
  float z[V];
  r.load(static_cast<const T*>(a.logits) + t * a.ldz, on, z);
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = Choice<T>::key(z[i], r.l * V + i);
  // Rank j's choice stays in lane j mod L, slot j / L.
  float val[V], peak = 0.f;
  int id[V];
#pragma unroll
  for (int s = 0; s < V; ++s) {
    val[s] = 0.f;
    id[s] = -1;
    for (int q = 0; q < L; ++q) {
      if (s * L + q >= a.top) break;  // uniform
      float v;
      int at;
      const bool found = Choice<T>::template next<L, V>(key, r.l * V, v, at);
      if (s == 0 && q == 0) peak = v;
      if (q == r.l && found) {
        val[s] = v;
        id[s] = at;
      }
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int s = 0; s < V; ++s) {
    val[s] = id[s] >= 0 ? exp_f(val[s] - peak) : 0.f;
    sum += val[s];
  }
  if (!a.normalize) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += z[i] == -kInf ? 0.f : exp_f(z[i] - peak);
  }
  const float inv = 1.f / group_sum<L>(sum);
#pragma unroll
  for (int s = 0; s < V; ++s) {
    const int j = s * L + r.l;
    if (in && j < a.top) {
      a.weights[t * a.top + j] = id[s] >= 0 ? val[s] * inv : 0.f;
      a.ids[t * a.top + j] = id[s];
    }
  }
}

template <typename T, int L, int V>
__global__ __launch_bounds__(256) void k_gate(GateArgs a) {
  for (int64_t first = (int64_t)blockIdx.x * (256 / L); first < a.tokens; first += (int64_t)gridDim.x * (256 / L))
    gate_tokens<T, L, V>(a, first);
}

template <typename T, int L, int V>
__device__ __forceinline__ void gate_grad_tokens(const GateArgs& a, int64_t first) {
  // The chosen experts' part, laid out by expert: a token's row is its own lanes' alone.
  __shared__ float rows[256 / L][L * V];
  const Row<T, L, V> r(a.experts);
  const int sub = threadIdx.x / L;
  const int64_t t = first + sub;
  const bool in = t < a.tokens, on = in && (!a.mask || a.mask[t]);
#pragma unroll
  for (int i = 0; i < V; ++i) rows[sub][r.l * V + i] = 0.f;
  wave_fence();
  int id[V];
  float g[V], mean = 0.f, w[V];
#pragma unroll
  for (int s = 0; s < V; ++s) {
    const int j = s * L + r.l;
    const bool have = on && j < a.top;
    id[s] = have ? a.ids[t * a.top + j] : -1;
    if (id[s] >= a.experts) id[s] = -1;
    w[s] = id[s] >= 0 ? a.weights[t * a.top + j] : 0.f;
    g[s] = id[s] >= 0 ? a.dweights[t * a.top + j] : 0.f;
    mean += w[s] * g[s];
  }
  mean = group_sum<L>(mean);
#pragma unroll
  for (int s = 0; s < V; ++s)
    if (id[s] >= 0) rows[sub][id[s]] = a.normalize ? w[s] * (g[s] - mean) : w[s] * g[s];
  wave_fence();
  float d[V] = {};
  if (!a.normalize) {
    r.load(static_cast<const T*>(a.logits) + t * a.ldz, on, d);
    r.softmax(d);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) d[i] = rows[sub][r.l * V + i] - d[i] * mean;
  r.store(static_cast<T*>(a.dlogits) + t * a.experts, in, d);
  wave_fence();
}

template <typename T, int L, int V>
__global__ __launch_bounds__(256) void k_gate_grad(GateArgs a) {
  for (int64_t first = (int64_t)blockIdx.x * (256 / L); first < a.tokens; first += (int64_t)gridDim.x * (256 / L))
    gate_grad_tokens<T, L, V>(a, first);
}

__device__ __forceinline__ int expert_at(const BalanceArgs& a, int64_t i) {
  const int64_t v = a.ids64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
  return v >= 0 && v < a.experts ? (int)v : -1;
}

// The join of n blocks' sums: a thread adds one expert's over one of `parts` stretches of blocks.
__device__ void finish_balance(const BalanceArgs& a, int n, double* sums, int* counts, double* waves) {
  const int tid = threadIdx.x, parts = 1024 / a.experts;
  const int e = tid % a.experts, part = tid / a.experts;
  const int per = (n + parts - 1) / parts, b0 = min(n, part * per), b1 = part < parts ? min(n, b0 + per) : b0;
  double p = 0.0;
  int c = 0;
#pragma unroll 32
  for (int b = b0; b < b1; ++b) {
    p += (double)a.part[(int64_t)b * a.experts + e];
    c += a.part_counts[(int64_t)b * (a.experts + 1) + e];
  }
  sums[tid] = p;
  counts[tid] = c;
  int64_t tokens = 0;
  for (int b = tid; b < n; b += 1024) tokens += a.part_counts[(int64_t)b * (a.experts + 1) + a.experts];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) tokens += __shfl_xor(tokens, off, 64);
  if ((tid & 63) == 0) waves[tid >> 6] = (double)tokens;
  __syncthreads();
  double all = 0.0;
  for (int w = 0; w < 16; ++w) all += waves[w];
  __syncthreads();
  double term = 0.0;
  if (tid < a.experts) {
    p = 0.0;
    c = 0;
    for (int q = 0; q < parts; ++q) {
      p += sums[q * a.experts + tid];
      c += counts[q * a.experts + tid];
    }
    const double share = all > 0.0 ? (double)c / (all * a.top) : 0.0;
    a.counts[tid] = c;
    a.shares[tid] = (float)share;
    term = all > 0.0 ? share * p / all : 0.0;
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) term += __shfl_xor(term, off, 64);
  if ((tid & 63) == 0) waves[tid >> 6] = term;
  __syncthreads();
  if (tid != 0) return;
  term = 0.0;
  for (int w = 0; w < 16; ++w) term += waves[w];
  *a.loss = (float)(term * a.experts);
  a.shares[a.experts] = all > 0.0 ? (float)(a.experts / all) : 0.f;
}

__global__ __launch_bounds__(1024) void k_balance_join(BalanceArgs a, int blocks) {
  __shared__ double sums[1024], waves[16];
  __shared__ int counts[1024];
  finish_balance(a, blocks, sums, counts, waves);
}

// A workgroup's tokens are one stretch of them.
template <typename T, int L, int V>
__global__ __launch_bounds__(1024) void k_balance(BalanceArgs a, int64_t stretch) {
  __shared__ float sums[16][L * V];
  __shared__ int counts[kGateMaxExperts + 1];
  const int tid = threadIdx.x;
  for (int i = tid; i <= a.experts; i += 1024) counts[i] = 0;
  __syncthreads();
  const Row<T, L, V> r(a.experts);
  const int64_t t0 = blockIdx.x * stretch, t1 = min(a.tokens, t0 + stretch);
  float p[V] = {};
  int seen = 0;
  // The next token's logits are in flight while this one's are worked on; those of a masked one are read and not used.
  Raw<T> next[V / 8];
  bool next_on = false;
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    next_on = t < t1 && (!a.mask || a.mask[t]);
    r.fetch(static_cast<const T*>(a.logits) + t * a.ldz, t < t1, next);
  };
  fetch(t0 + tid / L);
  for (int64_t base = t0; base < t1; base += 1024 / L) {
    float z[V];
    const bool on = next_on;
    Raw<T> now[V / 8];
#pragma unroll
    for (int c = 0; c < V / 8; ++c) now[c] = next[c];
    fetch(base + 1024 / L + tid / L);
    r.values(now, on, z);
    r.softmax(z);
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] += z[i];
    seen += on && r.l == 0;
  }
  for (int64_t i = t0 * a.top + tid; i < t1 * a.top; i += 1024) {
    const int e = !a.mask || a.mask[i / a.top] ? expert_at(a, i) : -1;
    if (e >= 0) atomicAdd(&counts[e], 1);
  }
  if (seen) atomicAdd(&counts[a.experts], seen);
  // The wave's tokens, then the waves in order.
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int off = L; off < 64; off <<= 1) p[i] += __shfl_xor(p[i], off, 64);
    if ((tid & 63) < L) sums[tid >> 6][r.l * V + i] = p[i];
  }
  __syncthreads();
  for (int e = tid; e < a.experts; e += 1024) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[w][e];
    a.part[(int64_t)blockIdx.x * a.experts + e] = s;
  }
  for (int e = tid; e <= a.experts; e += 1024) a.part_counts[(int64_t)blockIdx.x * (a.experts + 1) + e] = counts[e];
}

template <typename T, int L, int V>
__global__ __launch_bounds__(256) void k_balance_grad(BalanceArgs a) {
  const Row<T, L, V> r(a.experts);
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = i < r.n ? a.shares[r.l * V + i] : 0.f;
  const float scale = *a.dloss * a.shares[a.experts];
  const int64_t step = (int64_t)gridDim.x * (256 / L);
  Raw<T> next[V / 8];
  bool next_on = false;
  auto fetch = [&](int64_t t) __attribute__((always_inline)) {
    next_on = t < a.tokens && (!a.mask || a.mask[t]);
    r.fetch(static_cast<const T*>(a.logits) + t * a.ldz, t < a.tokens, next);
  };
  fetch((int64_t)blockIdx.x * (256 / L) + threadIdx.x / L);
  for (int64_t base = (int64_t)blockIdx.x * (256 / L); base < a.tokens; base += step) {
    const int64_t t = base + threadIdx.x / L;
    const bool in = t < a.tokens, on = next_on;
    float z[V], mean = 0.f;
    Raw<T> now[V / 8];
#pragma unroll
    for (int c = 0; c < V / 8; ++c) now[c] = next[c];
    fetch(t + step);
    r.values(now, on, z);
    r.softmax(z);
#pragma unroll
    for (int i = 0; i < V; ++i) mean += z[i] * f[i];
    mean = group_sum<L>(mean);
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = on ? scale * (z[i] * (f[i] - mean)) : 0.f;
    r.store(static_cast<T*>(a.dlogits) + t * a.experts, in, z);
  }
}

// f(lanes of a token, its logits a lane).
template <typename F>
void by_experts(int experts, F&& f) {
  const std::integral_constant<int, 8> v8{};
  if (experts <= 8) return f(std::integral_constant<int, 1>{}, v8);
  if (experts <= 16) return f(std::integral_constant<int, 2>{}, v8);
  if (experts <= 32) return f(std::integral_constant<int, 4>{}, v8);
  if (experts <= 64) return f(std::integral_constant<int, 8>{}, v8);
  if (experts <= 128) return f(std::integral_constant<int, 16>{}, v8);
  if (experts <= 256) return f(std::integral_constant<int, 32>{}, v8);
  if (experts <= 512) return f(std::integral_constant<int, 64>{}, v8);
  return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}
int lanes_of(int experts) {
  int l = 1;
  while (l < 64 && l * 8 < experts) l *= 2;
  return l;
}

template <typename T>
hipError_t gate(const GateArgs& a, bool grad, hipStream_t s) {
  // A launch holds fewer than 2^32 threads.
  const int64_t per = 256 / lanes_of(a.experts);
  const unsigned blocks = (unsigned)std::min<int64_t>((a.tokens + per - 1) / per, 1 << 22);
  by_experts(a.experts, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    if (grad) hipLaunchKernelGGL((k_gate_grad<T, L, V>), dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_gate<T, L, V>), dim3(blocks), dim3(256), 0, s, a);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t balance(const BalanceArgs& a, hipStream_t s) {
  const int blocks = balance_blocks(a.tokens, a.experts);
  const int64_t stretch = blocks ? (a.tokens + blocks - 1) / blocks : 0;
  if (blocks > 0) {
    by_experts(a.experts, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      hipLaunchKernelGGL((k_balance<T, L, V>), dim3(blocks), dim3(1024), 0, s, a, stretch);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(1024), 0, s, a, blocks);
  return hipGetLastError();
}

template <typename T>
hipError_t balance_grad(const BalanceArgs& a, hipStream_t s) {
  const int64_t per = 256 / lanes_of(a.experts);
  const unsigned blocks = (unsigned)std::min<int64_t>((a.tokens + per - 1) / per, 2048);
  by_experts(a.experts, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    hipLaunchKernelGGL((k_balance_grad<T, L, V>), dim3(blocks), dim3(256), 0, s, a);
  });
  return hipGetLastError();
}

}  // namespace

int balance_blocks(int64_t tokens, int experts) {
  const int64_t per = 1024 / lanes_of(experts);
  return (int)std::min<int64_t>((tokens + per - 1) / per, 256);
}

hipError_t launch_gate(const GateArgs& a, int dtype, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  return dtype == MUON_BF16 ? gate<uint16_t>(a, false, s) : gate<float>(a, false, s);
}
hipError_t launch_gate_grad(const GateArgs& a, int dtype, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  return dtype == MUON_BF16 ? gate<uint16_t>(a, true, s) : gate<float>(a, true, s);
}
hipError_t launch_balance(const BalanceArgs& a, int dtype, hipStream_t s) {
  return dtype == MUON_BF16 ? balance<uint16_t>(a, s) : balance<float>(a, s);
}
hipError_t launch_balance_grad(const BalanceArgs& a, int dtype, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  return dtype == MUON_BF16 ? balance_grad<uint16_t>(a, s) : balance_grad<float>(a, s);
}

}  // namespace muon
