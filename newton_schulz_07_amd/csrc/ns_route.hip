// ns_route.hip - routing of tokens to experts, and its gradient.
//
//   s = softmax or sigmoid of a token's logits
//   key = s + bias, or the logit itself where there is no bias
//   groups: a group's rank is the sum of its group_best largest s + bias (s
//   without a bias); only the experts of the top_groups best groups stay
//   ids = the top_k largest keys (equal ones: the lower index first)
//   weights = scale s[ids] / (sum s[ids] + 1e-20), or scale s[ids]
//
// A NaN key counts as -inf, so ids are always distinct experts; a NaN logit
// still makes the weights it enters NaN.  A row whose logits are all -inf has
// scores of zero.
//
// Keys that pass through exp are compared in 64 bits: in 32, sums s + bias of
// different experts meet often enough that the choice would hang on the
// rounding of exp.  Logits are compared as they are.
#include "ns_device.h"
#include "ns_sublayer.h"

namespace ns {
namespace {

template <typename T> __device__ __forceinline__ float logit(const T* row, int e) { return (float)row[e]; }

template <typename F>
__device__ __forceinline__ F wave_max(F v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const F u = __shfl_xor(v, o, 64);
    v = u > v ? u : v;
  }
  return v;
}
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The best of the lanes' candidates: the larger key, equal ones by index.
template <typename F>
__device__ __forceinline__ void wave_best(F& key, int& idx) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const F k = __shfl_xor(key, o, 64);
    const int i = __shfl_xor(idx, o, 64);
    if (k > key || (k == key && i < idx)) {
      key = k;
      idx = i;
    }
  }
}

constexpr int kNone = 0x7fffffff;

// LDS bytes of the counts and their prefix, up to the next 8 bytes
__host__ __device__ inline size_t route_lds_ints(int experts) { return ((size_t)(2 * experts + 1) * 4 + 7) / 8 * 8; }

// The choice of one token by one wave: lane j < top_k returns expert *id and
// its weight *w.  Lane l holds experts l + 64 v.  F: the keys' type (double
// where they are s + bias or groups are ranked by s).
template <typename T, int V, typename F>
__device__ __forceinline__ void choose(const RouteArgs& g, const T* row, double* gkeys, int* id, float* w) {
  constexpr bool WIDE = sizeof(F) == 8;
  const int lane = threadIdx.x & 63, E = g.experts;
  float l[V];
  F s[V], key[V];
  bool all_low = true;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    l[v] = e < E ? logit(row, e) : -INFINITY;
  }
  // scores (in F)
  F top = (F)0, total = (F)1;
  if (g.score == NS_SCORE_SOFTMAX) {
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) m = l[v] > m ? l[v] : m;
    m = wave_max(m);
    all_low = m == -INFINITY;
    top = (F)m;
    F t = (F)0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (WIDE) s[v] = exp((double)l[v] - top);
      else s[v] = expf(l[v] - top);
      // past the last expert: exp(-inf) is zero unless every logit is -inf or one is +inf
      if (lane + 64 * v >= E) s[v] = (F)0;
      t += s[v];
    }
    if constexpr (WIDE) total = wave_sum64(t);
    else total = wave_sum(t);
    if (all_low) {  // a NaN among -inf stays NaN
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = (F)0;
      bool nan = false;
#pragma unroll
      for (int v = 0; v < V; ++v) nan |= l[v] != l[v];
      total = __any(nan) ? (F)NAN : (F)1;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = s[v] / total;
  } else if (WIDE) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = (F)(1.0 / (1.0 + exp(-(double)l[v])));
  }
  const bool has_bias = g.bias != nullptr;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    key[v] = has_bias ? s[v] + (F)(e < E ? g.bias[e] : 0.0f) : (F)l[v];
    if (!(key[v] == key[v])) key[v] = (F)-INFINITY;
  }
  uint32_t open = 0;  // this lane's experts that may still be chosen
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane + 64 * v < E) open |= 1u << v;

  if constexpr (WIDE) {
    if (g.groups > 1) {
      // every lane < groups ranks one group
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane + 64 * v;
        if (e < E) {
          double r = has_bias ? key[v] : s[v];
          gkeys[e] = r == r ? r : -INFINITY;
        }
      }
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's LDS writes are done
      __builtin_amdgcn_wave_barrier();
      const int gs = E / g.groups;
      double a = -INFINITY, b = -INFINITY;
      if (lane < g.groups)
        for (int i = 0; i < gs; ++i) {
          const double r = gkeys[lane * gs + i];
          b = r > a ? a : (r > b ? r : b);
          a = r > a ? r : a;
        }
      double rank = g.group_best > 1 && gs > 1 ? a + b : a;
      if (!(rank == rank)) rank = -INFINITY;
      uint64_t kept = 0;
      bool taken = lane >= g.groups;
      for (int j = 0; j < g.top_groups; ++j) {
        double k = taken ? -INFINITY : rank;
        int i = taken ? kNone : lane;
        wave_best(k, i);
        if (lane == i) taken = true;
        kept |= 1ull << (i & 63);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = lane + 64 * v;
        if (e < E && !((kept >> (e / gs)) & 1)) open &= ~(1u << v);
      }
    }
  }

  int mine = 0;
  for (int j = 0; j < g.top_k; ++j) {
    F k = (F)-INFINITY;
    int i = kNone;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if ((open >> v) & 1) {
        if (i == kNone || key[v] > k) {  // v ascends: equal keys keep the lower index
          k = key[v];
          i = lane + 64 * v;
        }
      }
    wave_best(k, i);
    if ((i & 63) == lane) open &= ~(1u << (i >> 6));
    if (lane == j) mine = i;
  }
  // the chosen experts' scores
  F sc = (F)0;
  if (lane < g.top_k) {
    const float x = logit(row, mine);
    if (g.score == NS_SCORE_SOFTMAX) {
      if constexpr (WIDE) sc = (all_low ? (F)0 : (F)exp((double)x - top)) / total;
      else sc = (all_low ? (F)0 : (F)expf(x - top)) / total;
    } else {
      if constexpr (WIDE) sc = 1.0 / (1.0 + exp(-(double)x));
      else sc = 1.0f / (1.0f + expf(-x));
    }
  }
  F out = sc;
  if (g.renormalize) {
    F sum;
    if constexpr (WIDE) sum = wave_sum64(sc);
    else sum = wave_sum(sc);
    out = sc / (sum + (F)1e-20);
  }
  *id = mine;
  *w = (float)(out * (F)g.scale);
}

// Lanes of the wave whose expert is the same as this lane's (`bits` bits of
// it), of those that are `live`.
__device__ __forceinline__ uint64_t same_expert(int e, int bits, bool live) {
  uint64_t m = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((e >> b) & 1);
    m &= ((e >> b) & 1) ? set : ~set;
  }
  return m;
}

// Exclusive prefix of counts[0 .. n) into out[0 .. n], by the first wave.
__device__ __forceinline__ void prefix_by_wave0(const int* counts, int* out, int n) {
  if (threadIdx.x < 64) {
    int carry = 0;
    for (int e0 = 0; e0 < n; e0 += 64) {
      const int e = e0 + (int)threadIdx.x;
      const int c = e < n ? counts[e] : 0;
      int p = c;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(p, o, 64);
        if ((int)threadIdx.x >= o) p += u;
      }
      if (e < n) out[e] = carry + p - c;
      carry += __shfl(p, 63, 64);
    }
    if (threadIdx.x == 0) out[n] = carry;
  }
}

__device__ __forceinline__ int bits_of(int n) { return 32 - __clz(n); }  // bits of the values 0 .. n

// The slots of up to 64 waves x 64 choices that `blockDim.x` threads hold,
// one each: base[e] + the choices of the same expert before this one.  cnt:
// [waves][experts] in LDS.  Ends with base[e] moved past them.
__device__ __forceinline__ int place(int e, bool live, int experts, int* base, uint16_t* cnt) {
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < waves * experts; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const uint64_t m = same_expert(e, bits_of(experts - 1), live);
  const int before = __popcll(m & ((1ull << lane) - 1));
  if (live && before == 0) cnt[wave * experts + e] = (uint16_t)__popcll(m);
  __syncthreads();
  int slot = 0;
  if (live) {
    slot = base[e] + before;
    for (int w = 0; w < wave; ++w) slot += cnt[w * experts + e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < experts; i += blockDim.x) {
    int s = 0;
    for (int w = 0; w < waves; ++w) s += cnt[w * experts + i];
    base[i] += s;
  }
  __syncthreads();
  return slot;
}

// A wave to a token.  One block: it walks all the tokens and makes the plan
// too.  More: block b takes 16 tokens and leaves its experts' counts in
// hist[b].
template <typename T, int V, typename F>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(const RouteArgs g) {
  constexpr bool WIDE = sizeof(F) == 8;
  extern __shared__ char smem[];
  int* hist = reinterpret_cast<int*>(smem);  // [experts]
  int* base = hist + g.experts;              // [experts + 1], one block only
  // the waves' keys while they choose (groups only), then the plan's counts
  double* gkeys = reinterpret_cast<double*>(smem + route_lds_ints(g.experts));
  uint16_t* cnt = reinterpret_cast<uint16_t*>(gkeys);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const bool plan = g.offsets != nullptr, single = gridDim.x == 1;
  for (int e = threadIdx.x; e < g.experts; e += kRouteWaves * 64) hist[e] = 0;
  __syncthreads();
  const int t1 = single ? g.tokens : min(g.tokens, (int)(blockIdx.x + 1) * kRouteWaves);
  for (int t = blockIdx.x * kRouteWaves + wave; t < t1; t += kRouteWaves) {
    int id;
    float w;
    choose<T, V, F>(g, reinterpret_cast<const T*>(g.logits) + (long long)t * g.ld, gkeys + (WIDE ? wave * g.experts : 0),
                    &id, &w);
    if (lane < g.top_k) {
      g.ids[(long long)t * g.top_k + lane] = id;
      g.weights[(long long)t * g.top_k + lane] = w;
      if (plan) atomicAdd(&hist[id], 1);
    }
  }
  if (!plan) return;
  __syncthreads();
  if (!single) {
    for (int e = threadIdx.x; e < g.experts; e += kRouteWaves * 64) g.hist[(size_t)blockIdx.x * g.experts + e] = hist[e];
    return;
  }
  prefix_by_wave0(hist, base, g.experts);
  __syncthreads();
  for (int e = threadIdx.x; e <= g.experts; e += kRouteWaves * 64) g.offsets[e] = base[e];
  __threadfence_block();
  __syncthreads();
  const int n = g.tokens * g.top_k;
  for (int p0 = 0; p0 < n; p0 += kRouteWaves * 64) {
    const int p = p0 + (int)threadIdx.x;
    const bool live = p < n;
    const int e = live ? g.ids[p] : 0;
    const int slot = place(e, live, g.experts, base, cnt);
    if (live) {
      g.slots[p] = slot;
      g.rows[slot] = p / g.top_k;
    }
  }
}

// hist[b][e] -> the choices of e in blocks before b; hist[blocks][e] -> all
// of them.  16 experts to a block, 64 runs of blocks each.
constexpr int kHistExperts = 16, kHistRuns = 64;
__global__ __launch_bounds__(kHistExperts* kHistRuns) void route_scan_kernel(int* hist, int blocks, int experts) {
  __shared__ int sum[kHistRuns][kHistExperts];
  const int x = threadIdx.x % kHistExperts, run = threadIdx.x / kHistExperts, e = blockIdx.x * kHistExperts + x;
  const int per = (blocks + kHistRuns - 1) / kHistRuns;
  const int b0 = min(blocks, run * per), b1 = min(blocks, b0 + per);
  int s = 0;
  if (e < experts)
    for (int b = b0; b < b1; ++b) s += hist[(size_t)b * experts + e];
  sum[run][x] = s;
  __syncthreads();
  int before = 0;
  for (int r = 0; r < run; ++r) before += sum[r][x];
  if (e >= experts) return;
  for (int b = b0; b < b1; ++b) {
    const int c = hist[(size_t)b * experts + e];
    hist[(size_t)b * experts + e] = before;
    before += c;
  }
  if (run == kHistRuns - 1) hist[(size_t)blocks * experts + e] = before;
}

// Slots and rows of a block's tokens, from where hist puts them.
__global__ __launch_bounds__(1024) void route_place_kernel(const RouteArgs g) {
  extern __shared__ char smem[];
  int* base = reinterpret_cast<int*>(smem);  // [experts + 1]
  uint16_t* cnt = reinterpret_cast<uint16_t*>(base + g.experts + 1);
  const int blocks = gridDim.x;
  prefix_by_wave0(g.hist + (size_t)blocks * g.experts, base, g.experts);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= g.experts; e += blockDim.x) g.offsets[e] = base[e];
  __syncthreads();
  for (int e = threadIdx.x; e < g.experts; e += blockDim.x) base[e] += g.hist[(size_t)blockIdx.x * g.experts + e];
  __syncthreads();
  const int n = g.tokens * g.top_k;  // fits: checked on the host
  const int p = (int)blockIdx.x * kRouteWaves * g.top_k + (int)threadIdx.x;
  const bool live = threadIdx.x < kRouteWaves * g.top_k && p < n;
  const int e = live ? g.ids[p] : 0;
  const int slot = place(e, live, g.experts, base, cnt);
  if (live) {
    g.slots[p] = slot;
    g.rows[slot] = p / g.top_k;
  }
}

// dlogits of one token by one wave.  With p_j = s_j / (sum + 1e-20), or s_j:
//   ds_j = scale (dw_j - sum_i dw_i p_i) / (sum + 1e-20), or scale dw_j
//   sigmoid: dl_e = ds_e s_e (1 - s_e);  softmax: dl_e = s_e (ds_e - sum_j ds_j s_j)
template <typename T, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteGradArgs g) {
  extern __shared__ float ds_of[];  // [4 waves][experts]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, E = g.experts;
  const int t = blockIdx.x * 4 + wave;
  if (t >= g.tokens) return;
  float* ds = ds_of + (size_t)wave * E;
  for (int e = lane; e < E; e += 64) ds[e] = 0.0f;
  const T* row = reinterpret_cast<const T*>(g.logits) + (long long)t * g.ld;
  T* out = reinterpret_cast<T*>(g.dlogits) + (long long)t * E;
  float s[V];
  float top = 0.0f, inv = 1.0f;
  bool all_low = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    s[v] = e < E ? logit(row, e) : -INFINITY;
  }
  if (g.score == NS_SCORE_SOFTMAX) {
    top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) top = s[v] > top ? s[v] : top;
    top = wave_max(top);
    float sum = 0.0f;
    bool nan = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      nan |= s[v] != s[v];
      s[v] = lane + 64 * v < E ? expf(s[v] - top) : 0.0f;
      sum += s[v];
    }
    sum = wave_sum(sum);
    all_low = top == -INFINITY;
    inv = all_low ? (__any(nan) ? NAN : 0.0f) : 1.0f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = all_low ? inv : s[v] * inv;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = 1.0f / (1.0f + expf(-s[v]));
  }
  float sj = 0.0f, dw = 0.0f;
  int id = -1;
  if (lane < g.top_k) {
    id = g.ids[(long long)t * g.top_k + lane];
    if ((unsigned)id >= (unsigned)E) id = -1;
  }
  if (id >= 0) {
    dw = g.dweights[(long long)t * g.top_k + lane] * g.scale;
    const float x = logit(row, id);
    sj = g.score == NS_SCORE_SOFTMAX ? (all_low ? inv : expf(x - top) * inv) : 1.0f / (1.0f + expf(-x));
  }
  float d = dw;
  if (g.renormalize) {
    const float sum = wave_sum(sj) + 1e-20f;
    d = (dw - wave_sum(dw * (sj / sum))) / sum;
  }
  const float mean = wave_sum(id >= 0 ? d * sj : 0.0f);
  if (id >= 0) ds[id] = d;
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane + 64 * v;
    if (e < E) out[e] = (T)(g.score == NS_SCORE_SOFTMAX ? s[v] * (ds[e] - mean) : ds[e] * s[v] * (1.0f - s[v]));
  }
}

template <typename T, int V>
void launch_v(const RouteArgs& g, hipStream_t st) {
  const int blocks = route_blocks(g.tokens);
  const bool wide = g.bias != nullptr || g.groups > 1;
  // the keys in 64 bits outweigh the counts in 16 (at most 136 KiB, at 1024 experts)
  const size_t lds = route_lds_ints(g.experts) + (g.groups > 1  ? (size_t)kRouteWaves * g.experts * 8
                                                  : blocks == 1 ? (size_t)kRouteWaves * g.experts * 2
                                                                : 0);
  if (wide) {
    dispatch_lds(route_kernel<T, V, double>, dim3(blocks), dim3(kRouteWaves * 64), lds, st, g);
  } else {
    dispatch_lds(route_kernel<T, V, float>, dim3(blocks), dim3(kRouteWaves * 64), lds, st, g);
  }
}

template <typename T>
void launch_t(const RouteArgs& g, hipStream_t st) {
  if (g.experts <= 64) launch_v<T, 1>(g, st);
  else if (g.experts <= 128) launch_v<T, 2>(g, st);
  else if (g.experts <= 256) launch_v<T, 4>(g, st);
  else if (g.experts <= 512) launch_v<T, 8>(g, st);
  else launch_v<T, 16>(g, st);
}

template <typename T>
void launch_grad(const RouteGradArgs& g, hipStream_t st) {
  const dim3 grid((g.tokens + 3) / 4), block(256);
  const size_t lds = (size_t)4 * g.experts * 4;
  if (g.experts <= 64) dispatch_lds(route_backward_kernel<T, 1>, grid, block, lds, st, g);
  else if (g.experts <= 128) dispatch_lds(route_backward_kernel<T, 2>, grid, block, lds, st, g);
  else if (g.experts <= 256) dispatch_lds(route_backward_kernel<T, 4>, grid, block, lds, st, g);
  else if (g.experts <= 512) dispatch_lds(route_backward_kernel<T, 8>, grid, block, lds, st, g);
  else dispatch_lds(route_backward_kernel<T, 16>, grid, block, lds, st, g);
}

}  // namespace

hipError_t launch_route(int dtype, const RouteArgs& g, hipStream_t st) {
  if (dtype == 1) launch_t<bf16>(g, st);
  else launch_t<float>(g, st);
  if (hipError_t e = hipGetLastError()) return e;
  const int blocks = route_blocks(g.tokens);
  if (g.offsets == nullptr || blocks == 1) return hipSuccess;
  dispatch(route_scan_kernel, dim3((g.experts + kHistExperts - 1) / kHistExperts), dim3(kHistExperts * kHistRuns), st,
           g.hist, blocks, g.experts);
  if (hipError_t e = hipGetLastError()) return e;
  const int threads = (kRouteWaves * g.top_k + 63) / 64 * 64;
  const size_t lds = (size_t)(g.experts + 1) * 4 + (size_t)(threads / 64) * g.experts * 2;
  dispatch_lds(route_place_kernel, dim3(blocks), dim3(threads), lds, st, g);
  return hipGetLastError();
}

hipError_t launch_route_backward(int dtype, const RouteGradArgs& g, hipStream_t st) {
  if (dtype == 1) launch_grad<bf16>(g, st);
  else launch_grad<float>(g, st);
  return hipGetLastError();
}

}  // namespace ns
