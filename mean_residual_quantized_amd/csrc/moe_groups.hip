// Routing by softmax or sigmoid scores, with a bias for balance and groups of
// experts, for gfx950, and its gradient.
//
//   s_e = sigmoid(l_e) or softmax(l)_e;  c_e = s_e + b_e, by which experts are chosen
//   a group's score: the sum of its one or two largest c_e; the best groups stay
//   the topk largest c_e of theirs are chosen; w = scale s_e (/ the chosen ones' sum)
//
// The choice is by c_e in fp64 (equal ones: the lowest index first).  It is
// made from fp32 scores, their lowest bits given to the expert's place, and
// where two of those lie closer than their errors allow to tell, and are not of
// the same logit and bias, the wavefront's tokens are chosen again in fp64.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "launch.hpp"
#include "moe_lanes.hpp"

namespace averis {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// The lane's V logits: experts g V .. g V + V - 1 of the token's G lanes.  Lanes
// and places then order as the experts do, and a group of experts is a run of
// lanes wherever its size is a multiple of V.
template <typename T, int V>
__device__ __forceinline__ void load_run(const T* row, int first, int experts, float* l) {
  if (first + V <= experts) {
#pragma unroll
    for (int v = 0; v < V; v += Elem<T>::kPer)
      Elem<T>::unpack(*reinterpret_cast<const piece_t*>(row + first + v), l + v);
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    l[v] = first + v < experts ? Elem<T>::f32(row[first + v]) : kMasked;
}

// Sum over G neighbouring lanes in fp64, and the largest
template <int G>
__device__ __forceinline__ double group_sum64(double v) {
#pragma unroll
  for (int d = 1; d < G; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// The two largest of two ordered pairs
template <typename K>
__device__ __forceinline__ void merge2(K& a1, K& a2, K b1, K b2) {
  const K lo = a1 < b1 ? a1 : b1;
  a1 = a1 < b1 ? b1 : a1;
  a2 = a2 < b2 ? b2 : a2;
  a2 = a2 < lo ? lo : a2;
}

// V values into descending order (odd-even merge sort)
template <int V>
__device__ __forceinline__ void sort_down(uint32_t* s) {
#pragma unroll
  for (int p = 1; p < V; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t a = s[i + j], b = s[i + j + k];
            s[i + j] = a > b ? a : b;
            s[i + j + k] = a > b ? b : a;
          }
}

// what a lane of a token's G may keep in LDS, for it and for its neighbours
template <int G, int V>
struct RouteShare {
  static constexpr int kTokens = 256 / G;
  static constexpr int kGroups = G * V < kMaxGroups ? G * V : kMaxGroups;
  static constexpr int kSlots = G * V < kMaxTopk ? G * V : kMaxTopk;
  double group[kTokens][kGroups];    // scores (fp32 ones in their place)
  uint32_t key[kTokens][kSlots];     // chosen
  int32_t id[kTokens][kSlots];
};

// one wavefront's LDS accesses are in order
__device__ __forceinline__ void lds_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// Scores of the lane's logits in fp64: 0 where an expert is closed (softmax;
// sigmoid gives that itself).
template <int G, int V>
__device__ __forceinline__ void scores64(const float* l, int score, double* s) {
  if (score == kScoreSigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = 1.0 / (1.0 + exp(-(double)l[v]));
    return;
  }
  float top = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) top = __builtin_fmaxf(top, l[v]);
  top = group_fmax<G>(top);
  if (top == kMasked) top = 0.0f;
  double total = 0.0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = exp((double)l[v] - (double)top);
    total += s[v];
  }
  total = group_sum64<G>(total);
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = total == 0.0 ? 0.0 : s[v] / total;
}

// orders as c does: NaN above +inf, -0 as +0; closed (-inf) below all
__device__ __forceinline__ double rank64(double c) { return c != c ? __builtin_inf() : c; }

// The choice in fp64, for every token of the wavefront.  Its ids go to sh.id.
// NaN scores count as +inf here and by NaN's own mark above it.
template <int G, int V>
__device__ __forceinline__ void choose64(const float* l, const RouteGroups& a, int g, int tok,
                                      RouteShare<G, V>& sh) {
  double c[V];
  const bool limited = a.topk_groups < a.groups;
  const bool by_logit = !a.bias && !(limited && a.group_top == 2);
  bool nan[V];
  if (by_logit) {
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = l[v];
  } else {
    scores64<G, V>(l, a.score, c);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = g * V + v;
      if (a.bias) c[v] += e < a.experts ? (double)a.bias[e] : 0.0;
      if (l[v] == kMasked) c[v] = (double)kMasked;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    nan[v] = c[v] != c[v];
    c[v] = rank64(c[v]);
  }
  const double closed = -__builtin_inf();
  if (limited) {
    for (int j = 0; j < a.groups; ++j) {
      double t1 = closed, t2 = closed;
      bool n = false;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = g * V + v;
        const bool in = e >= j * a.gsize && e < (j + 1) * a.gsize;
        merge2(t1, t2, in ? c[v] : closed, closed);
        n |= in && nan[v];
      }
#pragma unroll
      for (int d = 1; d < G; d <<= 1) merge2(t1, t2, __shfl_xor(t1, d, 64), __shfl_xor(t2, d, 64));
      const uint64_t any = __ballot(n) >> ((threadIdx.x & 63) & ~(G - 1));
      double s = t1;
      if (t1 != closed && a.group_top == 2 && t2 != closed) s = t1 + t2;
      // a group with a NaN is above every other
      if (G == 64 ? any != 0 : (any & ((1ull << (G & 63)) - 1)) != 0) s = __builtin_nan("");
      if (g == 0) sh.group[tok][j] = s;
    }
    lds_order();
    // (by the lane: the groups of its experts)
    int last = -1;
    bool stays = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = g * V + v < a.experts ? g * V + v : a.experts - 1, mine = e / a.gsize;
      if (mine != last) {
        const double s = sh.group[tok][mine];
        int rank = 0;
        for (int j = 0; j < a.groups; ++j) {
          const double o = sh.group[tok][j];
          const bool above = s != s ? o != o && j < mine : o != o || o > s || (o == s && j < mine);
          rank += above ? 1 : 0;
        }
        stays = rank < a.topk_groups && !(s == closed);
        last = mine;
      }
      if (!stays) {
        c[v] = closed;
        nan[v] = false;
      }
    }
  }
  for (int r = 0; r < a.topk; ++r) {
    double best = closed;
    int at = 0x7FFFFFFF;
    bool n = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool up = c[v] != closed && ((nan[v] && !n) || (nan[v] == n && c[v] > best) || at == 0x7FFFFFFF);
      best = up ? c[v] : best;
      at = up ? g * V + v : at;
      n = up ? nan[v] : n;
    }
#pragma unroll
    for (int d = 1; d < G; d <<= 1) {
      const double ob = __shfl_xor(best, d, 64);
      const int oa = __shfl_xor(at, d, 64);
      const bool on = __shfl_xor((int)n, d, 64) != 0;
      const bool up = oa != 0x7FFFFFFF &&
                      (at == 0x7FFFFFFF || (on && !n) ||
                       (on == n && (ob > best || (ob == best && oa < at))));
      best = up ? ob : best;
      at = up ? oa : at;
      n = up ? on : n;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (g * V + v == at) c[v] = closed;
    if (g == 0) sh.id[tok][r] = at == 0x7FFFFFFF ? -1 : at;
  }
  lds_order();
}

// sigmoid(x) e^-min(most, 0): with most the largest logit that it is summed
// with, no sum of these is 0 where that of the scores would be
__device__ __forceinline__ float sigmoid_over(float x, float most) {
  if (x > 0.0f) return 1.0f / (1.0f + expf(-x));
  return expf(x - __builtin_fminf(most, 0.0f)) / (1.0f + expf(x));
}

// G lanes share a token, V of its experts each.  Each lane sorts its keys
// once; a round then compares the lanes' first keys alone, and the lane that
// has the largest moves on to its next.
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void k_route_groups(const T* __restrict__ logits, RouteGroups a) {
  __shared__ RouteShare<G, V> sh;
  constexpr uint32_t kPlace = V - 1;   // the key's bits for the place: V - 1 - v
  constexpr int KO = (kMaxTopk < G * V ? kMaxTopk : G * V) > G ? (kMaxTopk < G * V ? kMaxTopk : G * V) / G : 1;
  const int lane = threadIdx.x & 63, g = threadIdx.x % G, tok = threadIdx.x / G;
  const int base = lane & ~(G - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + tok;
  const bool live = t < a.tokens;   // the others repeat the last token, unstored
  const T* row = logits + (live ? t : a.tokens - 1) * a.ld;
  float l[V];
  load_run<T, V>(row, g * V, a.experts, l);
  const bool limited = a.topk_groups < a.groups;
  // Without a bias the logits order as the scores do (but sums of two do not).
  const bool by_logit = !a.bias && !(limited && a.group_top == 2);

  float top = 0.0f, total = 1.0f;   // softmax
  if (a.score == kScoreSoftmax && !(by_logit && a.renorm)) {
    top = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = __builtin_fmaxf(top, l[v]);
    top = group_fmax<G>(top);
    if (top == kMasked) top = 0.0f;
    float part = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) part += __builtin_amdgcn_exp2f((l[v] - top) * kLog2e);
    total = group_sum<G>(part);
    if (total == 0.0f) total = 1.0f;
  }
  uint32_t s[V];
  {
    const float inv = 1.0f / total;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float c = l[v];
      if (!by_logit) {
        c = a.score == kScoreSigmoid
                ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l[v]))
                : __builtin_amdgcn_exp2f((l[v] - top) * kLog2e) * inv;
        if (a.bias) c += g * V + v < a.experts ? a.bias[g * V + v] : 0.0f;
      }
      uint32_t k = f32_ordered(c + 0.0f);
      if (c != c) k = 0xFFFFFFFFu;
      k = (k & ~kPlace) | (kPlace - v);
      s[v] = l[v] == kMasked || c == kMasked ? 0u : k;
    }
  }
  // a key's value, and whether one lies so near below another that their order is open
  auto value = [](uint32_t k) __attribute__((always_inline)) { return f32_from_ordered(k & ~kPlace); };
  // Errors: a score's is at most 2^-20 (exp2 and the reciprocal 1 ulp each, the exponent |l| 2^-24, the
  // sum of a softmax 2^-20), without a bias 2^-16 of it; a key's cut bits 2^-19 of the value.
  const float rel = a.bias ? 0x1p-17f : 0x1p-15f, abs_ = a.bias ? 0x1p-18f : 0.0f;
  auto near = [&](uint32_t hi, uint32_t lo) __attribute__((always_inline)) {
    if (hi == 0u || lo == 0u) return false;
    if (by_logit) return sizeof(T) == 4 && (hi & ~kPlace) == (lo & ~kPlace);
    const float x = value(hi), y = value(lo);
    return x - y <= rel * __builtin_fabsf(x) + abs_;
  };
  bool open = false;   // the order is open
  if (!limited) {
    sort_down<V>(s);
  } else {
    const int p = a.group_lanes;   // lanes to a group; 0: groups end inside a lane's run
    // a group's score from its two largest keys, as an ordered key: 0 closed
    auto score_key = [&](uint32_t k1, uint32_t k2) __attribute__((always_inline)) {
      if (k1 == 0u) return 0u;
      float x = value(k1);
      if (a.group_top == 2 && k2 != 0u) x += value(k2);
      return x != x ? 0xFFFFFFFFu : f32_ordered(x + 0.0f);
    };
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;   // the last group that stays, the first that does not
    float mag = 0.0f;
    auto magnitude = [&](uint32_t k1, uint32_t k2) __attribute__((always_inline)) {
      const float x = k1 ? __builtin_fabsf(value(k1)) + (k2 ? __builtin_fabsf(value(k2)) : 0.0f) : 0.0f;
      mag = __builtin_fmaxf(mag, x);
    };
    if (p > 0) {
      sort_down<V>(s);
      uint32_t k1 = s[0], k2 = s[1];
      if (p > 1) merge2(k1, k2, partner<1>(k1), partner<1>(k2));
      if (p > 2) merge2(k1, k2, partner<2>(k1), partner<2>(k2));
      if (p > 4) merge2(k1, k2, partner<4>(k1), partner<4>(k2));
      if (p > 8) merge2(k1, k2, partner<8>(k1), partner<8>(k2));
      if (p > 16) merge2(k1, k2, partner<16>(k1), partner<16>(k2));
      const uint32_t mine = score_key(k1, k2);
      magnitude(k1, k2);
      const int at = g / p;
      int rank = 0;
      for (int j = 0; j < a.groups; ++j) {
        const uint32_t o = (uint32_t)__shfl((int)mine, base + j * p, 64);
        rank += o > mine || (o == mine && j < at) ? 1 : 0;
      }
      // (lanes past the last expert have closed groups)
      const bool stays = rank < a.topk_groups && mine != 0u;
      if (stays) lo = mine;
      else hi = mine;
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] = stays ? s[v] : 0u;
    } else {
      uint32_t* score = reinterpret_cast<uint32_t*>(sh.group[tok]);
      for (int j = 0; j < a.groups; ++j) {
        uint32_t k1 = 0u, k2 = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = g * V + v;
          merge2(k1, k2, e >= j * a.gsize && e < (j + 1) * a.gsize ? s[v] : 0u, 0u);
        }
#pragma unroll
        for (int d = 1; d < G; d <<= 1)
          merge2(k1, k2, (uint32_t)__shfl_xor((int)k1, d, 64), (uint32_t)__shfl_xor((int)k2, d, 64));
        magnitude(k1, k2);
        if (g == 0) score[j] = score_key(k1, k2);
      }
      lds_order();
      int last = -1;
      bool stays = false;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = g * V + v < a.experts ? g * V + v : a.experts - 1;
        const int at = (int)(((uint64_t)(uint32_t)e * a.gsize_inv) >> 32);   // e / gsize
        if (at != last) {
          const uint32_t mine = score[at];
          int rank = 0;
          for (int j = 0; j < a.groups; ++j) {
            const uint32_t o = score[j];
            rank += o > mine || (o == mine && j < at) ? 1 : 0;
          }
          stays = rank < a.topk_groups && mine != 0u;
          if (stays) lo = lo < mine ? lo : mine;
          else hi = hi > mine ? hi : mine;
          last = at;
        }
        s[v] = stays ? s[v] : 0u;
      }
      sort_down<V>(s);
    }
    lo = group_min<G>(lo);
    hi = group_max<G>(hi);
    mag = group_fmax<G>(mag);
    if (lo != 0xFFFFFFFFu && hi != 0u) {
      if (by_logit) {
        open = sizeof(T) == 4 && lo == hi;   // (fp32: the cut bits decide)
      } else {
        const float x = f32_from_ordered(lo), y = f32_from_ordered(hi);
        open = x - y <= 2.0f * (rel * mag + abs_);
      }
    }
  }

  for (int r = 0; r < a.topk; ++r) {
    const uint32_t head = s[0] & ~kPlace;
    const uint32_t best = group_max<G>(head);
    uint64_t has = __ballot(head == best) >> base;
    if constexpr (G < 64) has &= (1ull << (G & 63)) - 1;
    // equal keys: the lowest expert is the lowest lane's
    if (g == __builtin_ctzll(has)) {
      sh.key[tok][r] = s[0];
      sh.id[tok][r] = best == 0u ? -1 : g * V + (int)(kPlace - (s[0] & kPlace));
#pragma unroll
      for (int v = 0; v + 1 < V; ++v) s[v] = s[v + 1];
      s[V - 1] = 0u;
    }
  }
  lds_order();

  // Is the order of the chosen open, or the last one's to what was left?  Two
  // of the same logit and bias are not: the lowest index has come first.
  auto bias_of = [&](int e) { return a.bias ? a.bias[e] : 0.0f; };
  auto same = [&](int d, int e) {
    return Elem<T>::f32(row[d]) == Elem<T>::f32(row[e]) && bias_of(d) == bias_of(e);
  };
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    const int j = o * G + g;
    if (j + 1 < a.topk && near(sh.key[tok][j], sh.key[tok][j + 1]))
      open |= !same(sh.id[tok][j], sh.id[tok][j + 1]);
  }
  {
    const uint32_t last = sh.key[tok][a.topk - 1];
    if (near(last, s[0])) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (near(last, s[v]))
          open |= !same(sh.id[tok][a.topk - 1], g * V + (int)(kPlace - (s[v] & kPlace)));
    }
  }
  if (__builtin_expect(__ballot(open) != 0, 0)) choose64<G, V>(l, a, g, tok, sh);

  // the weights
  float x[KO];
  int id[KO];
  float most = kMasked;
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    const int j = o * G + g;
    id[o] = j < a.topk ? sh.id[tok][j] : -1;
    x[o] = id[o] >= 0 ? Elem<T>::f32(row[id[o]]) : kMasked;
    most = __builtin_fmaxf(most, x[o]);
  }
  if (a.renorm) {
    most = group_fmax<G>(most);
    if (most == kMasked) most = 0.0f;
  }
  float part = 0.0f;
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    x[o] = a.score == kScoreSigmoid ? sigmoid_over(x[o], a.renorm ? most : 0.0f)
           : a.renorm               ? expf(x[o] - most)
                                    : expf(x[o] - top) / total;
    x[o] = id[o] >= 0 ? x[o] : 0.0f;
    part += x[o];
  }
  float inv = a.scale;
  if (a.renorm) {
    const float sum = group_sum<G>(part);
    inv = sum == 0.0f ? 0.0f : a.scale / sum;
  }
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    const int j = o * G + g;
    if (live && j < a.topk) {
      a.ids[t * a.topk + j] = id[o];
      a.weights[t * a.topk + j] = id[o] < 0 ? 0.0f : x[o] * inv;
    }
  }
}

// With D_j = scale dw_j of the chosen, and m the weighted mean of D:
//   sigmoid:  dl_j = (D_j - m) w_j (1 - s_j), renormalised; D_j s_j (1 - s_j) else
//   softmax:  dl_j = (D_j - m) w_j over the chosen, renormalised; over all experts else
// The chosen few are scattered into the token's zeros in LDS, and whole rows
// written.
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void k_route_groups_grad(const T* logits, RouteGroupsGrad a,
                                                           T* dlogits) {
  __shared__ __attribute__((aligned(16))) float img[256 / G][G * V];
  constexpr int KM = kMaxTopk < G * V ? kMaxTopk : G * V, KO = KM > G ? KM / G : 1;
  const int g = threadIdx.x % G, tok = threadIdx.x / G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + tok;
  const bool live = t < a.tokens;
  const int64_t tr = live ? t : a.tokens - 1;
  const T* row = logits + tr * a.ld;
  const bool dense = a.score == kScoreSoftmax && !a.renorm;
  float x[KO], d[KO];
  int id[KO];
  float most = kMasked;
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    const int j = o * G + g;
    id[o] = -1;
    d[o] = 0.0f;
    if (j < a.topk) {
      id[o] = a.ids[tr * a.topk + j];
      d[o] = a.scale * a.dweights[tr * a.topk + j];
    }
    if ((uint32_t)id[o] >= (uint32_t)a.experts) id[o] = -1;
    x[o] = id[o] >= 0 ? Elem<T>::f32(row[id[o]]) : kMasked;
    most = __builtin_fmaxf(most, x[o]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) img[tok][g * V + v] = 0.0f;
  lds_order();
  if (!dense) {
    if (a.renorm) {
      most = group_fmax<G>(most);
      if (most == kMasked) most = 0.0f;
    }
    float part = 0.0f, dot = 0.0f, rest[KO];
#pragma unroll
    for (int o = 0; o < KO; ++o) {
      rest[o] = a.score == kScoreSigmoid ? sigmoid_over(-x[o], 0.0f) : 1.0f;   // 1 - s
      x[o] = a.score == kScoreSigmoid ? sigmoid_over(x[o], a.renorm ? most : 0.0f) : expf(x[o] - most);
      x[o] = id[o] >= 0 ? x[o] : 0.0f;
      d[o] = id[o] >= 0 ? d[o] : 0.0f;
      part += x[o];
      dot = __builtin_fmaf(x[o], d[o], dot);
    }
    float inv = 1.0f, mean = 0.0f;
    if (a.renorm) {
      const float sum = group_sum<G>(part);
      inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      mean = group_sum<G>(dot) * inv;
    }
#pragma unroll
    for (int o = 0; o < KO; ++o)
      if (id[o] >= 0) img[tok][id[o]] = (d[o] - mean) * (x[o] * inv) * rest[o];
    lds_order();
  }
  float f[V];
  if (dense) {
#pragma unroll
    for (int o = 0; o < KO; ++o)
      if (id[o] >= 0) img[tok][id[o]] = d[o];
    lds_order();
    float l[V];
    load_run<T, V>(row, g * V, a.experts, l);
    float top = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) top = __builtin_fmaxf(top, l[v]);
    top = group_fmax<G>(top);
    if (top == kMasked) top = 0.0f;
    float part = 0.0f, dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      f[v] = img[tok][g * V + v];
      l[v] = expf(l[v] - top);
      part += l[v];
      dot = __builtin_fmaf(l[v], f[v], dot);
    }
    const float sum = group_sum<G>(part), inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const float mean = group_sum<G>(dot) * inv;
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = l[v] * inv * (f[v] - mean);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = img[tok][g * V + v];
  }
  if (!live) return;
  T* out = dlogits + t * a.ldd;
  if (g * V + V <= a.experts) {
#pragma unroll
    for (int v = 0; v < V; v += Elem<T>::kPer)
      *reinterpret_cast<piece_t*>(out + g * V + v) = Elem<T>::pack(f + v);
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (g * V + v < a.experts) out[g * V + v] = Elem<T>::from(f[v]);
}

// Eight experts a lane (more than 512: sixteen).
#define AVERIS_GROUP_SHAPES(CALL) \
  if (experts <= 8) {             \
    CALL(1, 8);                   \
  } else if (experts <= 16) {     \
    CALL(2, 8);                   \
  } else if (experts <= 32) {     \
    CALL(4, 8);                   \
  } else if (experts <= 64) {     \
    CALL(8, 8);                   \
  } else if (experts <= 128) {    \
    CALL(16, 8);                  \
  } else if (experts <= 256) {    \
    CALL(32, 8);                  \
  } else if (experts <= 512) {    \
    CALL(64, 8);                  \
  } else {                        \
    CALL(64, 16);                 \
  }

template <typename T>
void groups_t(const T* l, const RouteGroups& a, hipStream_t st) {
  const int experts = a.experts;
#define AVERIS_ROUTE(G, V)                                                                       \
  in_launches(a.tokens, 256 / G, [&](int64_t t, int64_t n) {                                     \
    RouteGroups b = a;                                                                           \
    b.tokens = n;                                                                                \
    b.ids += t * a.topk;                                                                         \
    b.weights += t * a.topk;                                                                     \
    const int p = a.gsize / V;                                                                   \
    b.group_lanes = a.gsize % V == 0 && (p & (p - 1)) == 0 ? p : 0;                              \
    k_route_groups<T, G, V><<<dim3((unsigned)((n + 256 / G - 1) / (256 / G))), 256, 0, st>>>(    \
        l + t * a.ld, b);                                                                        \
  })
  AVERIS_GROUP_SHAPES(AVERIS_ROUTE)
#undef AVERIS_ROUTE
}

template <typename T>
void groups_grad_t(const T* l, const RouteGroupsGrad& a, T* dl, hipStream_t st) {
  const int experts = a.experts;
#define AVERIS_ROUTE(G, V)                                                                       \
  in_launches(a.tokens, 256 / G, [&](int64_t t, int64_t n) {                                     \
    RouteGroupsGrad b = a;                                                                       \
    b.tokens = n;                                                                                \
    b.ids += t * a.topk;                                                                         \
    b.dweights += t * a.topk;                                                                    \
    k_route_groups_grad<T, G, V><<<dim3((unsigned)((n + 256 / G - 1) / (256 / G))), 256, 0,      \
                                   st>>>(l + t * a.ld, b, dl + t * a.ldd);                       \
  })
  AVERIS_GROUP_SHAPES(AVERIS_ROUTE)
#undef AVERIS_ROUTE
}

}  // namespace

hipError_t launch_route_groups(const void* logits, bool bf16, const RouteGroups& a, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  if (bf16)
    groups_t(static_cast<const uint16_t*>(logits), a, st);
  else
    groups_t(static_cast<const float*>(logits), a, st);
  return hipGetLastError();
}

hipError_t launch_route_groups_grad(const void* logits, bool bf16, const RouteGroupsGrad& a,
                                    void* dlogits, hipStream_t st) {
  if (a.tokens == 0) return hipSuccess;
  if (bf16)
    groups_grad_t(static_cast<const uint16_t*>(logits), a, static_cast<uint16_t*>(dlogits), st);
  else
    groups_grad_t(static_cast<const float*>(logits), a, static_cast<float*>(dlogits), st);
  return hipGetLastError();
}

}  // namespace averis
