// ns_route.hip - routing of tokens to experts, and its gradient.
//
//   s = softmax or sigmoid of a token's logits
//   key = s + bias, or -inf for a logit of -inf; where there is no bias the
//   logit itself
//   groups: a group's rank is the sum of its group_best largest keys (s
//   without a bias), to which -inf adds nothing (-inf for a group of nothing
//   else); only the experts of the top_groups best groups stay
//   ids = the top_k largest keys (equal ones: the lower index first)
//   weights = scale s[ids] / (sum s[ids] + 1e-20), or scale s[ids]
//
// A NaN key counts as -inf, so ids are always distinct experts; a NaN logit
// still makes the weights it enters NaN.  A row whose logits are all -inf has
// scores of zero.
//
// Keys that pass through exp count in 64 bits: in 32, sums s + bias of
// different experts meet often enough that the choice would hang on the
// rounding of exp.  A token is first chosen for in fp32, with keys that hold
// their index in their last bits; where two keys (or two groups' ranks) that
// decide stand closer than that can tell apart, it is chosen for again in 64
// bits.  Logits without a bias are compared as they are.  Weights are made in
// fp32, from scores within a few steps (6e-8 of themselves off in a batch,
// against 3e-8 if everything but the last rounding is in 64 bits): the experts'
// outputs that they weigh are bf16 or fp32 sums.  Tokens that are chosen for
// again have theirs in 64 bits, as a by-product.
//
// Bound by instructions and, in small calls, by latency: the logits of 16384
// tokens and 128 experts are 8 MB (1.8 us of HBM).  16384 x 128 fp32, sigmoid
// with bias, 4 of 8 groups, top 8: 17 us and 7 us for the plan (with a wave to
// each token 34 us; with every key in 64 bits as well 65 us).  8192 x 128 softmax, top 8: 6
// and 7 us, its gradient 6 us.  One token: 4.3 us, of which a launch is 2.5.
// Batches of 513 to 1024 experts spill 70 registers, but for bf16 logits
// without a bias or groups (8192 x 1024, sigmoid: 12 us bf16, 18 fp32, with a
// bias 28 and 30).
#include <algorithm>
#include <type_traits>

#include "ns_device.h"
#include "ns_lanes.h"
#include "ns_sublayer.h"

namespace ns {
namespace {

template <typename T> __device__ __forceinline__ float logit(const T* row, int e) { return (float)row[e]; }

// Elements e0 .. e0 + V - 1 of a row of E; the last one again past its end.
// vec: E and the row's address are such that they come as whole vectors (or
// all lie past the end).  Element by element, lanes V apart keep the address
// unit busy for 8 times as long.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, bool vec, float (&l)[V]) {
  if (vec) {
    struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Some {
      T e[V];
    };
    const Some x = *reinterpret_cast<const Some*>(row + (e0 < E ? e0 : E - V));
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = (float)x.e[v];
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = logit(row, min(e0 + v, E - 1));
}
// whether rows of E elements, ld apart from an address p, come as vectors
template <typename T, int V> inline bool whole_vectors(const void* p, long long ld, int E) {
  const size_t unit = V * sizeof(T) < 16 ? V * sizeof(T) : 16;
  return E % V == 0 && ld * sizeof(T) % unit == 0 && reinterpret_cast<uintptr_t>(p) % unit == 0;
}

// A token takes L lanes of a wave, 16 (a DPP row, so that what its lanes tell
// each other stays off the LDS) or 64, of V experts each; lane l of them
// holds experts l V .. l V + V - 1.  16 lanes: four tokens share a wave's
// instructions, which is what bounds a long batch.
__device__ __forceinline__ float inverse(float v) { return __builtin_amdgcn_rcpf(v); }  // within a step of 1 / v
__device__ __forceinline__ double inverse(double v) { return 1.0 / v; }
// exp(v) within 2 steps, 0 below 2^-126: 2^(v log2 e), with what the product's
// rounding leaves out
__device__ __forceinline__ float exp_of(float v) {
  const float t = v * 0x1.715476p+0f;
  const float r = fmaf(v, 0x1.4ae0cp-26f, fmaf(v, 0x1.715476p+0f, -t));  // log2 e = 0x1.715476p+0 + 0x1.4ae0cp-26
  const float e = __builtin_amdgcn_exp2f(t);
  return e * (fabsf(t) < 256.0f ? fmaf(r, 0x1.62e43p-1f, 1.0f) : 1.0f);
}
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

constexpr int kNone = 0x7fffffff;

// Scores of a token's logits l (-inf past the last expert), in F.
template <int L, int V, typename F>
__device__ __forceinline__ void scores(const float (&l)[V], int score, F (&s)[V]) {
  if (score == NS_SCORE_SIGMOID) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = inverse((F)1 + exp_of(-(F)l[v]));
    return;
  }
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    m = larger(m, l[v]);
    nan |= l[v] != l[v];
  }
  m = lanes_max<L>(m);
  nan = lanes_min<L>(nan ? 0 : 1) == 0;
  F t = (F)0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // a row of -inf alone has scores of zero; past the last expert l - m may
    // be NaN (m = -inf or +inf), where the row is one of zeros or of NaNs
    s[v] = l[v] == -INFINITY ? (F)0 : exp_of((F)l[v] - (F)m);
    t += s[v];
  }
  t = lanes_sum<L>(t);
  if (m == -INFINITY) t = (F)1;
  if (nan) t = (F)NAN;
  t = inverse(t);
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = s[v] * t;
}

// Packed keys: a fp32 value as an integer of the same order (-0 as 0), its
// last bits replaced by an index that counts down, so that one integer
// maximum finds the largest value and, of values that agree but for those
// bits, the lower index.  -inf and NaN come after everything else, kClosed
// after those.
constexpr int kClosed = (int)0x80000000, kLeast = (int)0x80400000;
template <int LOW> __device__ __forceinline__ int packed(float v, int index) {
  const int b = __float_as_int(v + 0.0f);
  const int i = v > -INFINITY ? b ^ ((b >> 31) & 0x7fffffff) : kLeast;
  return (i & ~LOW) | (LOW - index);
}
template <int LOW> __device__ __forceinline__ float value_of(int key) {  // at most LOW steps below; NaN for -inf
  const int i = key & ~LOW;
  return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}
// Whether the values of two packed keys are in order for certain, each off by
// less than `off` / 2 and two steps before they were packed.
template <int LOW> __device__ __forceinline__ bool apart(int above, int below, float off) {
  const float x = value_of<LOW>(above), y = value_of<LOW>(below);
  return x - y > off + (LOW + 4) * 0x1p-23f * fmaxf(fabsf(x), fabsf(y));
}

// The same of an expert's neighbours in the order of their keys: s + bias, or
// logits, which are exact but for the bits that the index took (-inf has
// none: it goes by the index alone).  Nothing after the last expert.
template <int LOW> __device__ __forceinline__ bool in_order(int above, int below, bool has_bias, float off) {
  if (below == kClosed || (below & ~LOW) == (kLeast & ~LOW)) return true;
  return has_bias ? apart<LOW>(above, below, off) : ((above ^ below) & ~LOW) != 0;
}
// The token's lane before this one; `first` in its first.
template <int L> __device__ __forceinline__ int before(int v, int first) {
  if (L == 16) return __builtin_amdgcn_update_dpp(first, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  const int u = __shfl_up(v, 1, 64);
  return (threadIdx.x & 63) == 0 ? first : u;
}

// Adds to `place` how many of the row's 15 other lanes hold a larger key, or
// an equal one of a lower index.
template <int R> __device__ __forceinline__ void rank_among(double key, int index, int& place) {
  const double k = ror<R>(key);
  const int i = ror<R>(index);
  place += k > key || (k == key && i < index) ? 1 : 0;
  if constexpr (R > 1) rank_among<R - 1>(key, index, place);
}

// The choice of one token in fp32: its lanes write ids and weights to row
// `out` of g.ids and g.weights.  False, and nothing written, if a decision is
// too close.
//
// In units of 2^-24: exp is off by 2 of its value and by the distance to the
// largest logit (times the value at most 0.4 of the largest), the sum of a
// softmax by at most 24, its inverse by 2 and the product by 1, so a score is
// off by less than 32 = 2^-19 of the largest score, and a key by half a step
// more.
//
// WIDE: keys are s + bias, or groups are ranked.  Otherwise keys are logits,
// exact but for the packed bits, and the scores of the chosen ones alone are
// needed where they are renormalised (the sum is at least the largest's, so
// 1e-20 is nothing beside it).
template <typename T, int L, int V, bool WIDE>
__device__ __forceinline__ bool choose(const RouteArgs& g, const T* row, long long out, float* gkeys, int* hist) {
  constexpr int LOW = L * V - 1;
  const int ll = threadIdx.x & (L - 1), E = g.experts, e0 = ll * V;
  float l[V];
  int key[V];
  load_row<T, V>(row, e0, E, g.vec, l);
  const bool has_bias = WIDE && g.bias != nullptr, softmax = g.score == NS_SCORE_SOFTMAX;
  float shift[V];
  if (has_bias) load_row<float, V>(g.bias, e0, E, g.vec_bias, shift);
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? l[v] : -INFINITY;

  float top = 0.0f, times = 1.0f;  // softmax: a score is exp(l - top) times
  float off = 0.0f;                // twice a score's error
  bool nan = false;
  if (softmax) {
    top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      top = larger(top, l[v]);
      nan |= l[v] != l[v];
    }
    top = lanes_max<L>(top);
    nan = lanes_max<L>(nan ? 1 : 0) != 0;
  }
  bool sure = true;
  if constexpr (WIDE) {
    float s[V], most = 0.0f;
    if (softmax) {
      float t = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = l[v] == -INFINITY ? 0.0f : exp_of(l[v] - top);
        t += s[v];
      }
      t = lanes_sum<L>(t);
      times = nan ? NAN : top == -INFINITY ? 1.0f : inverse(t);
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] *= times;
      most = times;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = inverse(1.0f + exp_of(-l[v]));
        most = larger(most, s[v]);
      }
      most = lanes_max<L>(most);
    }
    off = most * 0x1p-18f;
    float r[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      r[v] = !has_bias ? s[v] : l[v] == -INFINITY ? -INFINITY : s[v] + shift[v];
      key[v] = packed<LOW>(has_bias ? r[v] : l[v], e0 + v);
    }
    if (g.groups > 1) {
      // lane i ranks groups i, i + L, ...; a group's keys stand an odd number
      // of words after the last one's (LDS banks)
      const int gs = E / g.groups, pitch = gs | 1;
      int grp = e0 / gs, in = e0 - grp * gs, of[V];  // the lane's experts' groups
#pragma unroll
      for (int v = 0; v < V; ++v) {
        of[v] = grp;
        if (e0 + v < E) gkeys[grp * pitch + in] = r[v] == r[v] ? r[v] : -INFINITY;
        if (++in == gs) {
          in = 0;
          ++grp;
        }
      }
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's LDS writes are done
      __builtin_amdgcn_wave_barrier();
      constexpr int GPL = kMaxGroups / L, GLOW = kMaxGroups - 1;
      int rank[GPL], ranked[GPL];
      float size[GPL];  // of the keys in a group's rank: each was rounded at its own
#pragma unroll
      for (int i = 0; i < GPL; ++i) {
        rank[i] = ranked[i] = kClosed;
        size[i] = 0.0f;
        if (i * L >= g.groups) continue;
        const int h = ll + i * L;
        float a = -INFINITY, b = -INFINITY;
        if (h < g.groups) {
          for (int j = 0; j < gs; j += 4) {  // four reads on their way at once
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = gkeys[h * pitch + min(j + u, gs - 1)];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              x[u] = j + u < gs ? x[u] : -INFINITY;
              b = __builtin_amdgcn_fmed3f(a, b, x[u]);  // b <= a: the second of the three
              a = x[u] > a ? x[u] : a;
            }
          }
          const bool two = g.group_best > 1 && gs > 1 && b > -INFINITY;
          rank[i] = ranked[i] = packed<GLOW>(two ? a + b : a, h);
          size[i] = two ? fabsf(a) + fabsf(b) : 0.0f;
        }
      }
      unsigned kept[2] = {0, 0};
      int last = 0, m = 0;
      for (int j = 0; j <= g.top_groups; ++j) {
        last = m;
        m = rank[0];
        if (g.groups > L)
#pragma unroll
          for (int i = 1; i < GPL; ++i) m = max(m, rank[i]);
        m = lanes_max<L>(m);
        if (j == g.top_groups) break;  // m: the best group that is left out
        rank[0] = rank[0] == m ? kClosed : rank[0];
        if (g.groups > L)
#pragma unroll
          for (int i = 1; i < GPL; ++i) rank[i] = rank[i] == m ? kClosed : rank[i];
        const int h = GLOW - (m & GLOW);
        kept[0] |= h < 32 ? 1u << h : 0u;
        kept[1] |= h < 32 ? 0u : 1u << (h - 32);
      }
      // A score's error enters a rank twice.  So does half a step of each key,
      // which is more than the rank's own where biases cancel: up to 2^-24 of
      // the two sizes, of either group.
      float blur = 2.0f * off;
      if (has_bias) {
        // (sizes are not negative: their bits are in their order)
        int most_of = ranked[0] == last || ranked[0] == m ? __float_as_int(size[0]) : 0;
        if (g.groups > L)
#pragma unroll
          for (int i = 1; i < GPL; ++i)
            if (ranked[i] == last || ranked[i] == m) most_of = max(most_of, __float_as_int(size[i]));
        blur += 0x1p-22f * __int_as_float(lanes_max<L>(most_of));
      }
      const bool least = (m & ~GLOW) == (kLeast & ~GLOW);  // nothing in the group: by its index
      sure = g.top_groups == g.groups || least || apart<GLOW>(last, m, blur);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = (of[v] < 32 ? kept[0] : kept[1]) >> (of[v] & 31) & 1 ? key[v] : kClosed;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = e0 + v < E ? key[v] : kClosed;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = e0 + v < E ? packed<LOW>(l[v], e0 + v) : kClosed;
    if (softmax && !g.renormalize) {
      float t = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) t += l[v] == -INFINITY ? 0.0f : exp_of(l[v] - top);
      times = top == -INFINITY ? 1.0f : inverse(lanes_sum<L>(t));
    }
  }
  // logits with nothing in the bits that were replaced (such as bf16's) are
  // told apart by the packed keys alone
  bool rounded = sizeof(T) == 4 && !has_bias;
  if (rounded) {
    int low = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) low |= l[v] > -INFINITY ? __float_as_int(l[v]) & LOW : 0;
    rounded = lanes_max<L>(low) != 0;
  }
  // Choice c L + j goes to lane j's mine[c], as its packed key.  Whether
  // neighbours are surely in order is looked at afterwards, all at once.
  constexpr int KC = kMaxTopK / L + 1;  // choices of a lane, and a round more
  int mine[KC];
  auto next = [&]() __attribute__((always_inline)) {  // the best key that is left
    int m = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = max(m, key[v]);
    m = lanes_max<L>(m);
    bool is[V];
#pragma unroll
    for (int v = 0; v < V; ++v) is[v] = key[v] == m;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = is[v] ? kClosed : key[v];
    return m;
  };
  const bool check = has_bias || rounded;
  const int rounds = min(g.top_k + (check ? 1 : 0), E);
  bool clear = true, edge = true;  // every pair in order; the last chosen and the first left out
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    mine[c] = kClosed;
    if (c * L >= rounds) continue;
    const int to = min(L, rounds - c * L);
    for (int j = 0; j < to; ++j) {
      const int m = next();
      mine[c] = ll == j ? m : mine[c];
    }
    if (check) {
      const int above = c == 0 ? before<L>(mine[c], mine[c]) : before<L>(mine[c], __shfl(mine[c > 0 ? c - 1 : 0], L - 1, L));
      const int first = c == 0 ? 1 : 0;
      const bool ok = in_order<LOW>(above, mine[c], has_bias, off);
      const bool in = ll >= first && ll < to;
      clear = clear && lanes_max<L>(in && !ok ? 1 : 0) == 0;
      if (c * L + to > g.top_k) edge = lanes_max<L>(in && ll == g.top_k - c * L && !ok ? 1 : 0) == 0;
    }
  }
  int n = rounds, last = kClosed;
  // Keys too close to tell: the candidates down to one that is surely past
  // the border get their keys in 64 bits, a lane each, and are ranked among
  // themselves; with more than 16 of them the whole token is chosen again.
  int place = ll;
  if (check && !clear) {
    if (g.top_k >= 16) return false;
    last = lanes_max<L>(ll == n - 1 ? mine[0] : kClosed);
    if (last == kClosed) {  // none is left out
      edge = true;
      --n;
    }
    while (!edge && n < 16 && n < E) {
      const int m = next();
      edge = m == kClosed || in_order<LOW>(last, m, has_bias, off);
      last = m;
      if (m == kClosed) break;
      mine[0] = ll == n ? m : mine[0];
      ++n;
    }
    if (n == E) edge = true;
    if (!edge || !sure) return false;
    double exact = -INFINITY;
    if (has_bias) {
      double sum = 1.0;
      if (softmax) {
        sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += l[v] == -INFINITY ? 0.0 : exp((double)l[v] - (double)top);
        sum = lanes_sum<L>(sum);
        if (top == -INFINITY && !nan) sum = 1.0;  // nothing but -inf: scores of zero
      }
      if (ll < n) {
        const double x = logit(row, LOW - (mine[0] & LOW));
        exact = softmax ? exp(x - (double)top) / sum : 1.0 / (1.0 + exp(-x));
        exact = x == -INFINITY ? -INFINITY : exact + (double)g.bias[LOW - (mine[0] & LOW)];
      }
    } else if (ll < n) {
      exact = logit(row, LOW - (mine[0] & LOW));
    }
    if (!(exact == exact)) exact = -INFINITY;
    const int index = ll < n ? LOW - (mine[0] & LOW) : kNone;
    place = 0;
    rank_among<15>(exact, index, place);
    if (ll >= n) place = L;
  }
  if (!sure) return false;

  // the chosen experts' scores, one lane each
  float sc[KC], total = 0.0f;
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    sc[c] = 0.0f;
    mine[c] = LOW - (mine[c] & LOW);
    if (c * L + place >= g.top_k) continue;
    const float x = logit(row, mine[c]);
    if (softmax) {
      sc[c] = x == -INFINITY ? 0.0f : exp_of(x - top);
      sc[c] *= nan ? NAN : times;
    } else {
      sc[c] = inverse(1.0f + exp_of(-x));
    }
    total += sc[c];
  }
  float by = g.scale;
  if (g.renormalize) by = g.scale / (lanes_sum<L>(total) + 1e-20f);
#pragma unroll
  for (int c = 0; c < KC; ++c)
    if (c * L + place < g.top_k) {
      g.ids[out + c * L + place] = mine[c];
      g.weights[out + c * L + place] = sc[c] * by;
      if (hist) atomicAdd(&hist[mine[c]], 1);
    }
  return true;
}

// The same in 64 bits, for the tokens that need it: a whole wave to a token.
template <typename T, int V>
__device__ __forceinline__ void choose_exactly(const RouteArgs& g, const T* row, long long out, double* gkeys, int* hist) {
  constexpr int L = 64;
  typedef double F;
  const int ll = threadIdx.x & (L - 1), E = g.experts, e0 = ll * V;
  float l[V];
  F s[V], key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? logit(row, e0 + v) : -INFINITY;
  scores<L, V, F>(l, g.score, s);
  const bool has_bias = g.bias != nullptr;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = has_bias ? s[v] + (F)(e0 + v < E ? g.bias[e0 + v] : 0.0f) : (F)l[v];
    if (!(key[v] == key[v]) || l[v] == -INFINITY) key[v] = (F)-INFINITY;
  }
  if (g.groups > 1) {
    // lane i ranks groups i, i + L, ...; a group's keys stand an odd number
    // of doubles after the last one's (LDS banks)
    const int gs = E / g.groups, pitch = gs | 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = e0 + v;
      const double r = has_bias ? key[v] : s[v];
      if (e < E) gkeys[e / gs * pitch + e % gs] = r == r ? r : -INFINITY;
    }
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's LDS writes are done
    __builtin_amdgcn_wave_barrier();
    constexpr int GPL = kMaxGroups / L;
    double rank[GPL];
#pragma unroll
    for (int i = 0; i < GPL; ++i) {
      const int grp = ll + i * L;
      double a = -INFINITY, b = -INFINITY;
      if (grp < g.groups)
        for (int j = 0; j < gs; ++j) {
          const double r = gkeys[grp * pitch + j];
          b = fmax(b, fmin(a, r));
          a = fmax(a, r);
        }
      rank[i] = g.group_best > 1 && gs > 1 && b > -INFINITY ? a + b : a;
      if (!(rank[i] == rank[i])) rank[i] = -INFINITY;
      if (grp >= g.groups) rank[i] = NAN;  // NaN: not to be chosen (any more)
    }
    uint64_t kept = 0;
    for (int j = 0; j < g.top_groups; ++j) {
      double m = rank[0];
#pragma unroll
      for (int i = 1; i < GPL; ++i) m = larger(m, rank[i]);
      m = lanes_max<L>(m);
      int best = kNone;
#pragma unroll
      for (int i = GPL - 1; i >= 0; --i) best = rank[i] == m ? ll + i * L : best;
      best = lanes_min<L>(best);
#pragma unroll
      for (int i = 0; i < GPL; ++i)
        if (best == ll + i * L) rank[i] = NAN;
      kept |= 1ull << (best & 63);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = e0 + v;
      if (e < E && !((kept >> (e / gs)) & 1)) key[v] = (F)NAN;
    }
  }
  int place[V];  // the choice that an expert is, or -1
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (e0 + v >= E) key[v] = (F)NAN;  // NaN: not to be chosen (any more)
    place[v] = -1;
  }
  for (int j = 0; j < g.top_k; ++j) {
    F m = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = larger(m, key[v]);
    m = lanes_max<L>(m);
    int best = kNone;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) best = key[v] == m ? e0 + v : best;
    best = lanes_min<L>(best);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (best == e0 + v) {
        key[v] = (F)NAN;
        place[v] = j;
      }
  }
  F total = (F)1;
  if (g.renormalize) {
    total = (F)0;
#pragma unroll
    for (int v = 0; v < V; ++v) total += place[v] >= 0 ? s[v] : (F)0;
    total = lanes_sum<L>(total) + (F)1e-20;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (place[v] >= 0) {
      g.ids[out + place[v]] = e0 + v;
      g.weights[out + place[v]] = (float)(s[v] / total * (F)g.scale);
      if (hist) atomicAdd(&hist[e0 + v], 1);
    }
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

// LDS bytes of the counts and their prefix, up to the next 8 bytes
__host__ __device__ inline size_t route_lds_ints(int experts) { return ((size_t)(2 * experts + 1) * 4 + 7) / 8 * 8; }

// LDS bytes of a wave's keys where groups are ranked: its tokens' in fp32, or
// one token's in 64 bits
__host__ __device__ inline size_t route_keys_bytes(int tokens_per_wave, int experts, int groups) {
  return groups > 1 ? (size_t)(experts + groups) * (tokens_per_wave > 2 ? tokens_per_wave * 4 : 8) / 8 * 8 : 0;
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

// Slots and rows of choices [p0, p1), in order, from base on.
__device__ __forceinline__ void place_tokens(const RouteArgs& g, int p0, int p1, int* base, uint16_t* cnt) {
  for (; p0 < p1; p0 += blockDim.x) {
    const int p = p0 + (int)threadIdx.x;
    const bool live = p < p1;
    const int e = live ? g.ids[p] : 0;
    const int slot = place(e, live, g.experts, base, cnt);
    if (live) {
      g.slots[p] = slot;
      // (counts that are another call's, such as those of two graphs that were
      // captured on one stream and run on two, lead to no write outside rows)
      if ((unsigned)slot < (unsigned)(g.tokens * g.top_k)) g.rows[slot] = p / g.top_k;
    }
  }
}

// 64 / L tokens to a wave.  One block: it walks all the tokens and makes the
// plan too.  More: a block takes kRouteWaves 64 / L tokens and leaves its
// experts' counts in hist[block].
template <typename T, int L, int V, bool WIDE, bool SINGLE>
__global__ __launch_bounds__((SINGLE ? route_single_waves(L * V) : kRouteWaves) * 64) void route_kernel(const RouteArgs g) {
  constexpr int TPW = 64 / L;
  extern __shared__ char smem[];
  int* hist = reinterpret_cast<int*>(smem);  // [experts]
  int* base = hist + g.experts;              // [experts + 1], one block only
  // the tokens' keys while they choose (groups only), then the plan's counts
  char* keys = smem + route_lds_ints(g.experts);
  uint16_t* cnt = reinterpret_cast<uint16_t*>(keys);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6, lane = threadIdx.x & 63;
  const bool plan = g.offsets != nullptr;
  if (plan) {
    for (int e = threadIdx.x; e < g.experts; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const int tb = waves * TPW, t1 = SINGLE ? g.tokens : min(g.tokens, (int)(blockIdx.x + 1) * tb);
  int t0 = blockIdx.x * tb + wave * TPW;
  do {
    const int t = t0 + lane / L;
    const T* logits = reinterpret_cast<const T*>(g.logits);
    char* mine = keys + (WIDE ? (size_t)wave * route_keys_bytes(TPW, g.experts, g.groups) : 0);
    bool sure = true;
    if (t < t1)
      sure = choose<T, L, V, WIDE>(g, logits + (long long)t * g.ld, (long long)t * g.top_k,
                                   reinterpret_cast<float*>(mine) + (WIDE ? lane / L * (g.experts + g.groups) : 0),
                                   plan ? hist : nullptr);
    if (WIDE || sizeof(T) == 4)  // (bf16 logits are told apart by their packed keys)
      for (uint64_t left = __ballot(!sure && lane % L == 0); left != 0; left &= left - 1) {
        const long long x = t0 + (__ffsll((unsigned long long)left) - 1) / L;
        choose_exactly<T, (L * V + 63) / 64>(g, logits + x * g.ld, x * g.top_k, reinterpret_cast<double*>(mine),
                                             plan ? hist : nullptr);
      }
    t0 += tb;
  } while (SINGLE && t0 < t1);
  if (!plan) return;
  __threadfence_block();
  __syncthreads();
  if (!SINGLE) {
    for (int e = threadIdx.x; e < g.hist_ld; e += blockDim.x)
      g.hist[(size_t)blockIdx.x * g.hist_ld + e] = e < g.experts ? hist[e] : 0;
    return;
  }
  prefix_by_wave0(hist, base, g.experts);
  __syncthreads();
  for (int e = threadIdx.x; e <= g.experts; e += blockDim.x) g.offsets[e] = base[e];
  place_tokens(g, 0, g.tokens * g.top_k, base, cnt);
}

// hist[b][e] -> the choices of e in blocks before b; hist[blocks][e] -> all
// of them.  Four experts to a thread, 256 runs of blocks each: a run to a
// lane, so that the runs are added up by shuffles.
constexpr int kHistLanes = 4, kHistRuns = 256;
__global__ __launch_bounds__(kHistLanes* kHistRuns) void route_scan_kernel(int* hist, int blocks, int ld) {
  __shared__ int4 sum[kHistLanes][kHistRuns / 64];
  const int x = threadIdx.x / kHistRuns, run = threadIdx.x % kHistRuns, lane = run & 63, w = run >> 6;
  const int e = (blockIdx.x * kHistLanes + x) * 4;
  const int per = (blocks + kHistRuns - 1) / kHistRuns;
  const int b0 = min(blocks, run * per), b1 = e < ld ? min(blocks, b0 + per) : b0;
  int4 s = make_int4(0, 0, 0, 0);
  for (int b = b0; b < b1; ++b) {
    const int4 c = *reinterpret_cast<const int4*>(hist + (size_t)b * ld + e);
    s = make_int4(s.x + c.x, s.y + c.y, s.z + c.z, s.w + c.w);
  }
  int4 p = s;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int4 u = make_int4(__shfl_up(p.x, o, 64), __shfl_up(p.y, o, 64), __shfl_up(p.z, o, 64), __shfl_up(p.w, o, 64));
    if (lane >= o) p = make_int4(p.x + u.x, p.y + u.y, p.z + u.z, p.w + u.w);
  }
  if (lane == 63) sum[x][w] = p;
  __syncthreads();
  int4 at = make_int4(p.x - s.x, p.y - s.y, p.z - s.z, p.w - s.w);
  for (int v = 0; v < w; ++v) at = make_int4(at.x + sum[x][v].x, at.y + sum[x][v].y, at.z + sum[x][v].z, at.w + sum[x][v].w);
  for (int b = b0; b < b1; ++b) {
    int4* h = reinterpret_cast<int4*>(hist + (size_t)b * ld + e);
    const int4 c = *h;
    *h = at;
    at = make_int4(at.x + c.x, at.y + c.y, at.z + c.z, at.w + c.w);
  }
  if (run == kHistRuns - 1 && e < ld) *reinterpret_cast<int4*>(hist + (size_t)blocks * ld + e) = at;
}

// Slots and rows of a block's tokens, bound by latency (7 us for 16384 tokens
// of 8 choices: the counts, their prefix, then the choices).  SCANNED: from where route_scan_kernel
// has put them; otherwise each block adds up the counts of all blocks itself.
template <bool SCANNED>
__global__ __launch_bounds__(1024) void route_place_kernel(const RouteArgs g, int block_tokens) {
  extern __shared__ char smem[];
  int* base = reinterpret_cast<int*>(smem);  // [experts + 1]
  uint16_t* cnt = reinterpret_cast<uint16_t*>(base + g.experts + 1);
  if (SCANNED) {
    prefix_by_wave0(g.hist + (size_t)gridDim.x * g.hist_ld, base, g.experts);
    __syncthreads();
    if (blockIdx.x == 0)
      for (int e = threadIdx.x; e <= g.experts; e += blockDim.x) g.offsets[e] = base[e];
    __syncthreads();
    for (int e = threadIdx.x; e < g.experts; e += blockDim.x) base[e] += g.hist[(size_t)blockIdx.x * g.hist_ld + e];
  } else {
    // four experts to a thread, as many runs of blocks as there are threads
    // left; cnt's place holds the sums of all blocks and of those before
    int *all = reinterpret_cast<int*>(smem + route_lds_ints(g.experts)), *before = all + g.hist_ld;
    for (int e = threadIdx.x; e < 2 * g.hist_ld; e += blockDim.x) all[e] = 0;
    __syncthreads();
    const int quads = g.hist_ld / 4, runs = blockDim.x / quads, q = threadIdx.x % quads, run = threadIdx.x / quads;
    int4 a = make_int4(0, 0, 0, 0), b = a;
    if (run < runs)
#pragma unroll 4
      for (int i = run; i < (int)gridDim.x; i += runs) {
        const int4 c = *reinterpret_cast<const int4*>(g.hist + (size_t)i * g.hist_ld + 4 * q);
        a = make_int4(a.x + c.x, a.y + c.y, a.z + c.z, a.w + c.w);
        if (i < (int)blockIdx.x) b = make_int4(b.x + c.x, b.y + c.y, b.z + c.z, b.w + c.w);
      }
    if (run < runs) {  // sums of integers: any order gives the same
      atomicAdd(&all[4 * q], a.x); atomicAdd(&all[4 * q + 1], a.y);
      atomicAdd(&all[4 * q + 2], a.z); atomicAdd(&all[4 * q + 3], a.w);
      atomicAdd(&before[4 * q], b.x); atomicAdd(&before[4 * q + 1], b.y);
      atomicAdd(&before[4 * q + 2], b.z); atomicAdd(&before[4 * q + 3], b.w);
    }
    __syncthreads();
    prefix_by_wave0(all, base, g.experts);
    __syncthreads();
    if (blockIdx.x == 0)
      for (int e = threadIdx.x; e <= g.experts; e += blockDim.x) g.offsets[e] = base[e];
    __syncthreads();
    for (int e = threadIdx.x; e < g.experts; e += blockDim.x) base[e] += before[e];
    __syncthreads();
  }
  const int t0 = blockIdx.x * block_tokens, t1 = min(g.tokens, t0 + block_tokens);
  place_tokens(g, t0 * g.top_k, t1 * g.top_k, base, cnt);
}

// dlogits of a token by one wave.  With p_j = s_j / (sum + 1e-20), or s_j:
//   ds_j = scale (dw_j - sum_i dw_i p_i) / (sum + 1e-20), or scale dw_j
//   sigmoid: dl_e = ds_e s_e (1 - s_e);  softmax: dl_e = s_e (ds_e - sum_j ds_j s_j)
// A sigmoid and its complement both come from e = exp(-|l|), as 1 / (1 + e) and
// e / (1 + e): of a large logit, which is what is chosen, 1 - s has no bits left.
// dw is spread over the experts in LDS; the ids of a token are distinct.  A
// wave to each token at any length (16384 x 256 fp32, softmax: 11 us, with 16
// lanes 16.3; sigmoid 10).  HBM would take 7 us for these 34 MB; what takes the
// rest is not measured.
template <typename T, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteGradArgs g) {
  constexpr int L = 64;
  extern __shared__ float spread[];  // [tokens of the block][experts]
  const int ll = threadIdx.x & (L - 1), E = g.experts, e0 = ll * V;
  const int t = blockIdx.x * (256 / L) + threadIdx.x / L;
  if (t >= g.tokens) return;
  float* dw_of = spread + (size_t)(threadIdx.x / L) * E;
  int* chosen = reinterpret_cast<int*>(spread + (size_t)(256 / L) * E) + (size_t)(threadIdx.x / L) * E;
  for (int e = ll; e < E; e += L) chosen[e] = 0;
  const T* row = reinterpret_cast<const T*>(g.logits) + (long long)t * g.ld;
  float l[V], s[V], d[V];
  load_row<T, V>(row, e0, E, g.vec, l);
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? l[v] : -INFINITY;
  for (int j = ll; j < g.top_k; j += L) {
    const int id = g.ids[(long long)t * g.top_k + j];
    if ((unsigned)id < (unsigned)E) {
      dw_of[id] = g.dweights[(long long)t * g.top_k + j] * g.scale;
      chosen[id] = 1;
    }
  }
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave's LDS writes are done
  __builtin_amdgcn_wave_barrier();
  float rest[V];  // sigmoid: 1 - s
  if (g.score == NS_SCORE_SIGMOID) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float e = exp_of(-fabsf(l[v])), r = inverse(1.0f + e);
      s[v] = l[v] < 0.0f ? e * r : r;
      rest[v] = l[v] < 0.0f ? r : e * r;
    }
  } else {
    scores<L, V, float>(l, g.score, s);
  }
  bool on[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    on[v] = e0 + v < E && chosen[e0 + v] != 0;
    d[v] = on[v] ? dw_of[e0 + v] : 0.0f;
  }
  if (g.renormalize) {
    float sum = 0.0f, mean = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) sum += on[v] ? s[v] : 0.0f;
    sum = lanes_sum<L>(sum) + 1e-20f;
#pragma unroll
    for (int v = 0; v < V; ++v) mean += on[v] ? d[v] * s[v] : 0.0f;
    const float by = 1.0f / sum;
    mean = lanes_sum<L>(mean) * by;
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = on[v] ? (d[v] - mean) * by : 0.0f;
  }
  float mean = 0.0f;
  if (g.score == NS_SCORE_SOFTMAX) {
#pragma unroll
    for (int v = 0; v < V; ++v) mean += on[v] ? d[v] * s[v] : 0.0f;
    mean = lanes_sum<L>(mean);
  }
  T* out = reinterpret_cast<T*>(g.dlogits) + (long long)t * E + e0;
  struct alignas(V * sizeof(T) < 16 ? V * sizeof(T) : 16) Some {
    T e[V];
  } x;
#pragma unroll
  for (int v = 0; v < V; ++v)
    x.e[v] = (T)(g.score == NS_SCORE_SOFTMAX ? s[v] * (d[v] - mean) : d[v] * s[v] * rest[v]);
  if (g.vec_out) {
    if (e0 < E) *reinterpret_cast<Some*>(out) = x;
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (e0 + v < E) out[v] = x.e[v];
}

template <typename T, int L, int V>
void launch_v(RouteArgs g, hipStream_t st) {
  g.vec = whole_vectors<T, V>(g.logits, g.ld, g.experts);
  g.vec_bias = whole_vectors<float, V>(g.bias, 0, g.experts);
  const RouteShape r = route_shape(g.tokens, g.experts);
  const bool wide = g.bias != nullptr || g.groups > 1, single = r.blocks == 1;
  const size_t keys = r.waves * route_keys_bytes(r.tokens_per_wave, g.experts, g.groups);
  const size_t cnt = single ? (size_t)r.waves * g.experts * 2 : 0;
  const size_t lds = route_lds_ints(g.experts) + (keys > cnt ? keys : cnt);  // at most 144 KiB, with 1024 experts in groups
  const dim3 grid(r.blocks), block(r.waves * 64);
  if (!single) {
    if (wide) dispatch_lds(route_kernel<T, L, V, true, false>, grid, block, lds, st, g);
    else dispatch_lds(route_kernel<T, L, V, false, false>, grid, block, lds, st, g);
  } else if constexpr (L == 64) {  // (few tokens: a wave to each)
    if (wide) dispatch_lds(route_kernel<T, L, V, true, true>, grid, block, lds, st, g);
    else dispatch_lds(route_kernel<T, L, V, false, true>, grid, block, lds, st, g);
  }
}

template <typename T, int V>
void launch_grad_v(RouteGradArgs g, hipStream_t st) {
  g.vec = whole_vectors<T, V>(g.logits, g.ld, g.experts);
  g.vec_out = whole_vectors<T, V>(g.dlogits, g.experts, g.experts);
  constexpr int tb = 4;
  dispatch_lds(route_backward_kernel<T, V>, dim3((g.tokens + tb - 1) / tb), dim3(256), (size_t)tb * g.experts * 8, st,
               g);
}

// Calls f with the experts of a lane, of L lanes.
template <int L, typename F>
void for_width(int experts, F f) {
  if (experts <= L) f(std::integral_constant<int, 1>());
  else if (experts <= 2 * L) f(std::integral_constant<int, 2>());
  else if (experts <= 4 * L) f(std::integral_constant<int, 4>());
  else if (experts <= 8 * L) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_route(int dtype, const RouteArgs& g, hipStream_t st) {
  const RouteShape r = route_shape(g.tokens, g.experts);
  auto lanes = [&](auto l) {
    for_width<l.value>(g.experts, [&](auto v) {
      if (dtype == 1) launch_v<bf16, l.value, v.value>(g, st);
      else launch_v<float, l.value, v.value>(g, st);
    });
  };
  if (r.tokens_per_wave == 4) lanes(std::integral_constant<int, 16>());
  else lanes(std::integral_constant<int, 64>());
  if (hipError_t e = hipGetLastError()) return e;
  if (g.offsets == nullptr || r.blocks == 1) return hipSuccess;
  const int block_tokens = r.waves * r.tokens_per_wave;
  const bool scan = r.blocks > kRouteUnscannedBlocks;
  const int threads = scan ? std::min(1024, (block_tokens * g.top_k + 63) / 64 * 64) : 1024;
  const size_t cnt = (size_t)(threads / 64) * g.experts * 2, sums = scan ? 0 : (size_t)2 * g.hist_ld * 4 + (g.experts * 4 + 8);
  const size_t lds = (size_t)(g.experts + 1) * 4 + std::max(cnt, sums);
  if (scan) {
    dispatch(route_scan_kernel, dim3((g.hist_ld + 4 * kHistLanes - 1) / (4 * kHistLanes)), dim3(kHistLanes * kHistRuns),
             st, g.hist, r.blocks, g.hist_ld);
    if (hipError_t e = hipGetLastError()) return e;
    dispatch_lds(route_place_kernel<true>, dim3(r.blocks), dim3(threads), lds, st, g, block_tokens);
  } else {
    dispatch_lds(route_place_kernel<false>, dim3(r.blocks), dim3(threads), lds, st, g, block_tokens);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(int dtype, const RouteGradArgs& g, hipStream_t st) {
  for_width<64>(g.experts, [&](auto v) {
    if (dtype == 1) launch_grad_v<bf16, v.value>(g, st);
    else launch_grad_v<float, v.value>(g, st);
  });
  return hipGetLastError();
}

}  // namespace ns
