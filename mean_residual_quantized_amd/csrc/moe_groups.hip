// Routing by softmax or sigmoid scores, with a bias for balance and groups of
// experts, for gfx950, and its gradient.
//
//   s_e = sigmoid(l_e) or softmax(l)_e;  c_e = s_e + b_e, by which experts are chosen
//   a group's score: the sum of its one or two largest c_e; the best groups stay
//   the topk largest c_e of theirs are chosen; w = scale s_e (/ the chosen ones' sum)
//
// The choice is by c_e in fp64 (equal ones: the lowest index first).  It is
// made from fp32 scores, their lowest bits given to the expert's place, and
// where some of those lie closer than their errors allow to tell, and are not of
// the same logit and bias, the few are ranked by their fp64 values, or, where that
// does not settle it, the wavefront's tokens chosen again in fp64.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"
#include "moe_lanes.hpp"

namespace averis {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Logits first .. first + V - 1 of a row, of which `many` are there (the others closed)
template <typename T, int V>
__device__ __forceinline__ void load_run(const T* row, int first, int many, float* l) {
  if (many >= V) {
#pragma unroll
    for (int v = 0; v < V; v += Elem<T>::kPer)
      Elem<T>::unpack(*reinterpret_cast<const piece_t*>(row + first + v), l + v);
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    l[v] = v < many ? Elem<T>::f32(row[first + v]) : kMasked;
}

// the other lane's value, 64 bits of it
template <int D, typename K>
__device__ __forceinline__ K partner_of(K v) {
  if constexpr (sizeof(K) == 4) {
    return __builtin_bit_cast(K, partner<D>(__builtin_bit_cast(uint32_t, v)));
  } else {
    const u32x2_t w = __builtin_bit_cast(u32x2_t, v);
    return __builtin_bit_cast(K, u32x2_t{partner<D>(w[0]), partner<D>(w[1])});
  }
}
// f(D) for each step of a butterfly over G lanes
template <int G, int D = 1, typename F>
__device__ __forceinline__ void butterfly(F f) {
  if constexpr (D < G) {
    f(std::integral_constant<int, D>{});
    butterfly<G, 2 * D>(f);
  }
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

// What a token's lanes keep in LDS for one another: the two largest of each lane,
// then each group's score (G lanes hold at most G groups), and the chosen.
template <int G, int V>
struct alignas(16) RouteShare {
  static constexpr int kTokens = 256 / G;
  static constexpr int kGroups = G < 4 ? 4 : G;
  static constexpr int kSlots = G * V < kMaxTopk ? G * V : kMaxTopk;
  double pair[kTokens][G][2];          // (the fp32 keys in their place)
  double score[kTokens][kGroups];
  uint32_t edge[kTokens][2];           // scores of the last group that stays, of the first that does not
  uint32_t key[kTokens][kSlots + 1];   // (the next one behind them)
  int32_t id[kTokens][kSlots + 1];
};

// one wavefront's LDS accesses are in order
__device__ __forceinline__ void lds_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// the lane's experts: a run of `many` from `first` on, within its group
struct RouteLane {
  int group, first, many;
};
template <int V>
__device__ __forceinline__ RouteLane route_lane(const RouteGroups& a, int g) {
  RouteLane r;
  r.group = (int)(((uint64_t)(uint32_t)g * a.lanes_inv) >> 32);   // g / group_lanes
  const int place = (g - r.group * a.group_lanes) * V, left = a.gsize - place;
  r.first = r.group * a.gsize + place;
  r.many = r.group >= a.groups ? 0 : left < V ? left : V;
  return r;
}

// The choice in fp64, for every token of the wavefront; its ids go to sh.id.
template <typename T, int G, int V>
__device__ __forceinline__ void choose64(const T* row, const RouteGroups& a, int g, int tok,
                                         RouteShare<G, V>& sh) {
  const RouteLane at0 = route_lane<V>(a, g);
  const bool limited = a.topk_groups < a.groups;
  const bool by_logit = !a.bias && !(limited && a.group_top == 2);
  const double closed = -__builtin_inf();
  double c[V];
  uint32_t nan = 0;   // bit v: c[v] is NaN (and +inf in its place)
  {
    float l[V];
    load_run<T, V>(row, at0.first, at0.many, l);
    double top = 0.0, inv = 1.0;
    if (!by_logit && a.score == kScoreSoftmax) {
      float m = l[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = __builtin_fmaxf(m, l[v]);
      m = group_fmax<G>(m);
      top = m == kMasked ? 0.0 : (double)m;
      double total = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[v] = exp((double)l[v] - top);
        total += c[v];
      }
      butterfly<G>([&](auto d) { total += partner_of<decltype(d)::value>(total); });
      inv = total;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (by_logit) c[v] = l[v];
      else if (a.score == kScoreSigmoid) c[v] = 1.0 / (1.0 + exp(-(double)l[v]));
      else c[v] = inv == 0.0 ? 0.0 : c[v] / inv;
      if (a.bias && v < at0.many) c[v] += (double)a.bias[at0.first + v];
      if (l[v] == kMasked) c[v] = closed;
      if (c[v] != c[v]) {
        nan |= 1u << v;
        c[v] = __builtin_inf();
      }
    }
  }
  if (limited) {
    double t1 = closed, t2 = closed;
#pragma unroll
    for (int v = 0; v < V; ++v) merge2(t1, t2, c[v], closed);
    sh.pair[tok][g][0] = nan ? __builtin_nan("") : t1;
    sh.pair[tok][g][1] = t2;
    lds_order();
    if (g < a.groups) {
      double s1 = closed, s2 = closed;
      bool any = false;   // a group with a NaN is above every other
      for (int i = 0; i < a.group_lanes; ++i) {
        const double u = sh.pair[tok][g * a.group_lanes + i][0];
        any |= u != u;
        merge2(s1, s2, u, sh.pair[tok][g * a.group_lanes + i][1]);
      }
      if (a.group_top == 2 && s2 != closed) s1 += s2;
      sh.score[tok][g] = any ? __builtin_nan("") : s1;
    }
    lds_order();
    const int mine = at0.group < a.groups ? at0.group : 0;
    const double s = sh.score[tok][mine];
    int rank = 0;
    for (int j = 0; j < a.groups; ++j) {
      const double o = sh.score[tok][j];
      rank += s != s ? (o != o && j < mine) : (o != o || o > s || (o == s && j < mine));
    }
    if (rank >= a.topk_groups || s == closed) {
      nan = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = closed;
    }
  }
  constexpr int kNone = 0x7FFFFFFF;
  for (int r = 0; r < a.topk; ++r) {
    double best = closed;
    int at = kNone, n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int m = (nan >> v) & 1;
      const bool up = c[v] != closed && (at == kNone || m > n || (m == n && c[v] > best));
      best = up ? c[v] : best;
      at = up ? at0.first + v : at;
      n = up ? m : n;
    }
    butterfly<G>([&](auto d) {
      const double ob = partner_of<decltype(d)::value>(best);
      const int oa = partner_of<decltype(d)::value>(at), on = partner_of<decltype(d)::value>(n);
      const bool up = oa != kNone && (at == kNone || on > n || (on == n && (ob > best || (ob == best && oa < at))));
      best = up ? ob : best;
      at = up ? oa : at;
      n = up ? on : n;
    });
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at0.first + v == at) c[v] = closed;
    if (g == 0) sh.id[tok][r] = at == kNone ? -1 : at;
  }
  lds_order();
}

// sigmoid(x) e^-min(most, 0): with most the largest logit that it is summed
// with, no sum of these is 0 where that of the scores would be
__device__ __forceinline__ float sigmoid_over(float x, float most) {
  if (x > 0.0f) return 1.0f / (1.0f + expf(-x));
  return expf(x - __builtin_fminf(most, 0.0f)) / (1.0f + expf(x));
}

// G lanes share a token, V experts each of one group's (lanes and places order as
// the experts do).  Each lane sorts its keys once; a round then compares the
// lanes' first keys alone, and the lane that has the largest moves on to its
// next.  Bound by vector instructions (their pipes are busy for 30 of the first
// case's 36 us; 68 lane-instructions an expert), most of them the scores' and keys'
// (about ten and two slow ones an expert), the sort's (eight an expert) and the
// rounds' (about 40): 65521 tokens of 256 experts in 8 groups, top 8, fp32 36 us
// (67 MB, 1.9 TB/s; 69 with eight experts a lane and every near choice made again
// whole), 10007 of 160 in 8 groups bf16 8.4 us, 16 of 64 5.0 us (latency).
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void k_route_groups(const T* __restrict__ logits, RouteGroups a) {
  __shared__ RouteShare<G, V> sh;
  constexpr uint32_t kPlace = V - 1;        // the key's bits for the place: V - 1 - v
  constexpr uint32_t kOpen = 0x00800000u;   // keys of open experts are at least this
  constexpr int KM = kMaxTopk < G * V ? kMaxTopk : G * V, KO = KM > G ? KM / G : 1;
  const int lane = threadIdx.x & 63, g = threadIdx.x % G, tok = threadIdx.x / G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + tok;
  const bool live = t < a.tokens;   // the others repeat the last token, unstored
  const T* row = logits + (live ? t : a.tokens - 1) * a.ld;
  const RouteLane at0 = route_lane<V>(a, g);
  const bool limited = a.topk_groups < a.groups;
  // Without a bias the logits order as the scores do (but sums of two do not).
  const bool by_logit = !a.bias && !(limited && a.group_top == 2);

  uint32_t s[V];
  float top = 0.0f, total = 1.0f;   // softmax
  {
    float l[V], bias[V];
    load_run<T, V>(row, at0.first, at0.many, l);
    if (a.bias) load_run<float, V>(a.bias, at0.first, at0.many, bias);
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
    const float inv = 1.0f / total;
    float c[V];
    if (by_logit) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = l[v] + 0.0f;   // (-0 as 0)
    } else if (a.score == kScoreSigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l[v]));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = __builtin_amdgcn_exp2f((l[v] - top) * kLog2e) * inv;
    }
    if (a.bias) {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] += bias[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = l[v] == kMasked ? kMasked : c[v];   // (its key is below kOpen)
      uint32_t k = __float_as_uint(c[v]);
      k ^= (uint32_t)((int32_t)k >> 31) | 0x80000000u;
      k = c[v] != c[v] ? 0xFFFFFFFFu : k;
      s[v] = (k & ~kPlace) | (kPlace - v);
    }
  }
  // A key's value, and whether one lies so near below another that their order is open.
  // Errors: a score's is at most 2^-20 (exp2 and the reciprocal 1 ulp each, the exponent |l| 2^-24, the
  // sum of a softmax 2^-20), without a bias 2^-16 of it and 2^-126 (exp2 and the reciprocal give 0 below
  // the normal numbers); a key's cut bits 2^-18 of the value.
  auto value = [](uint32_t k, uint32_t cut) __attribute__((always_inline)) { return f32_from_ordered(k & ~cut); };
  const float rel = a.bias ? 0x1p-17f : 0x1p-15f, abs_ = a.bias ? 0x1p-18f : 0x1p-125f;
  auto near = [&](uint32_t hi, uint32_t lo) __attribute__((always_inline)) {
    if (hi < kOpen || lo < kOpen) return false;
    if (by_logit) return sizeof(T) == 4 && (hi & ~kPlace) == (lo & ~kPlace);
    const float x = value(hi, kPlace), y = value(lo, kPlace);
    return x - y <= rel * __builtin_fabsf(x) + abs_;
  };
  sort_down<V>(s);
  auto bias_of = [&](int e) { return a.bias ? a.bias[e] : 0.0f; };
  // of the same logit and bias: the lowest index has come first
  auto same = [&](int d, int e) {
    return Elem<T>::f32(row[d]) == Elem<T>::f32(row[e]) && bias_of(d) == bias_of(e);
  };
  auto exact = [&](int e) {   // (a softmax's sum is choose64's)
    if (e < 0) return -__builtin_inf();
    const double l = (double)Elem<T>::f32(row[e]);
    return by_logit ? l : 1.0 / (1.0 + exp(-l)) + (double)bias_of(e);
  };
  bool open = false, all = false;   // the order is open; nothing but choose64 settles it
  if (limited) {
    // a group's score as a key whose lowest six bits give equal ones an order; closed: 0
    constexpr uint32_t kCut = 63;
    uint32_t* pairs = reinterpret_cast<uint32_t*>(sh.pair[tok]);
    uint32_t* scores = reinterpret_cast<uint32_t*>(sh.score[tok]);
    *reinterpret_cast<u32x2_t*>(pairs + 4 * g) = u32x2_t{s[0], s[1]};
    if (g < 2) sh.edge[tok][g] = 0u;
    if constexpr (G == 1) sh.edge[tok][1] = 0u;
    lds_order();
    float size = 0.0f;   // |first| + |second|
    const int padded = (a.groups + 3) & ~3;
    for (int j = g; j < padded; j += G) {
      uint32_t k1 = 0u, k2 = 0u, score = 0u;
      if (j < a.groups) {
        for (int i = 0; i < a.group_lanes; ++i) {
          const u32x2_t o = *reinterpret_cast<const u32x2_t*>(pairs + 4 * (j * a.group_lanes + i));
          merge2(k1, k2, o[0], o[1]);
        }
      }
      if (k1 >= kOpen) {
        float x = value(k1, kPlace);
        size = __builtin_fabsf(x);
        if (a.group_top == 2 && k2 >= kOpen) {
          const float y = value(k2, kPlace);
          x += y;
          size += __builtin_fabsf(y);
        }
        score = ((x != x ? 0xFFFFFFFFu : f32_ordered(x + 0.0f)) & ~kCut) | (kCut - j);
      }
      scores[j] = score;
    }
    // With a bias the errors go by the largest parts of any group: one further from the edge, whose parts
    // cancel, may be known less well than the two beside it
    if (a.bias) size = group_fmax<G>(size);
    lds_order();
    const int group = at0.group < a.groups ? at0.group : 0;
    const uint32_t mine = scores[group];
    int rank = 0;
    for (int j = 0; j < padded; j += 4) {
      const u32x4_t o = *reinterpret_cast<const u32x4_t*>(scores + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) rank += o[i] > mine ? 1 : 0;
    }
    bool stays = rank < a.topk_groups && mine != 0u;
    if (at0.many > 0 && at0.first == at0.group * a.gsize && mine != 0u &&
        (rank == a.topk_groups - 1 || rank == a.topk_groups))
      sh.edge[tok][rank == a.topk_groups ? 1 : 0] = mine;
    lds_order();
    const uint32_t hi = sh.edge[tok][0], lo = sh.edge[tok][1];
    if (hi != 0u && lo != 0u) {
      if (by_logit) {
        open = sizeof(T) == 4 && (hi & ~kCut) == (lo & ~kCut);
      } else {
        const float x = value(hi, kCut), y = value(lo, kCut);
        // (not >, for two sums past fp32's range differ by NaN)
        open = !(x - y > 2.0f * (rel * (a.bias ? size : x) + abs_) + 0x1p-16f * __builtin_fabsf(x));
      }
    }
    if (__builtin_expect(__ballot(open) != 0, 0)) {
      // the groups' exact scores, of the two largest keys each
      all = open && !by_logit && a.score == kScoreSoftmax;
      uint32_t ref = 0u;               // the key of the last that counts
      int e1 = -1, e2 = -1, own = -1;   // own: the one whose value counts last
      if (g < a.groups) {
        uint32_t k1 = 0u, k2 = 0u;
        for (int i = 0; i < a.group_lanes; ++i) {
          const u32x2_t o = *reinterpret_cast<const u32x2_t*>(pairs + 4 * (g * a.group_lanes + i));
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t k = o[q];
            if (k < kOpen) continue;
            const int e = g * a.gsize + i * V + (int)(kPlace - (k & kPlace));
            if (k > k1) {
              k2 = k1, e2 = e1;
              k1 = k, e1 = e;
            } else if (k > k2) {
              k2 = k, e2 = e;
            }
          }
        }
        double x = exact(e1);
        const double y = exact(e2);
        if (a.group_top == 2) {
          own = x < y ? e1 : e2;
          if (e2 >= 0) x += y;
          ref = k2;
        } else {
          own = x < y ? e2 : e1;
          x = y > x ? y : x;
          ref = k1;
        }
        all |= open && x != x;
        sh.score[tok][g] = x;
      }
      // Whether another of the group's may be above that one: every key is looked at, for before one a
      // little larger there can be any number of equal ones, whose indexes are lower.  One that is the same
      // as `own` is not
      const int from = (lane & ~(G - 1)) + group;
      ref = (uint32_t)__shfl((int)ref, from, 64);
      e1 = __shfl(e1, from, 64);
      e2 = __shfl(e2, from, 64);
      own = __shfl(own, from, 64);
      if (open && near(ref, s[0])) {
        uint32_t places = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) places |= (near(ref, s[v]) ? 1u : 0u) << (kPlace - (s[v] & kPlace));
        // (in the experts' order, whole pieces a load: 65521 x 256 equal logits in 8 groups 70 us in fp32, 61
        // in bf16; key by key 155 and 149)
        float l[V], bias[V];
        load_run<T, V>(row, at0.first, at0.many, l);
        if (a.bias) load_run<float, V>(a.bias, at0.first, at0.many, bias);
        const float its = Elem<T>::f32(row[own]), its_bias = bias_of(own);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = at0.first + v;
          if ((places >> v & 1u) && e != e1 && e != e2) all |= !(l[v] == its && (!a.bias || bias[v] == its_bias));
        }
      }
      lds_order();
      if (open) {
        const double x = sh.score[tok][group];
        rank = 0;
        for (int j = 0; j < a.groups; ++j) {
          const double o = sh.score[tok][j];
          rank += o > x || (o == x && j < group) ? 1 : 0;
        }
        stays = rank < a.topk_groups && x != -__builtin_inf();
      }
      open = false;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = stays ? s[v] : 0u;
  }

  // the largest key left goes to slot r
  auto take = [&](int r) __attribute__((always_inline)) {
    const uint32_t head = s[0] & ~kPlace;
    const uint32_t best = group_max<G>(head);
    const uint64_t has = __ballot(head == best);
    // equal keys: the lowest expert is the lowest lane's
    int first;
    if constexpr (G == 64) {
      first = __builtin_ctzll(has);
    } else {
      const uint32_t half = (uint32_t)(lane & 32 ? has >> 32 : has);
      first = __builtin_ctz(G == 32 ? half : (half >> (lane & 31 & ~(G - 1))) & ((1u << (G & 31)) - 1u));
    }
    if (g == first) {
      sh.key[tok][r] = s[0];
      sh.id[tok][r] = s[0] < kOpen ? -1 : at0.first + (int)(kPlace - (s[0] & kPlace));
#pragma unroll
      for (int v = 0; v + 1 < V; ++v) s[v] = s[v + 1];
      s[V - 1] = 0u;
    }
  };
  for (int r = 0; r < a.topk; ++r) take(r);
  lds_order();

  // Is the order of the chosen open, or the last one's to what was left?
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    const int j = o * G + g;
    if (j + 1 < a.topk && near(sh.key[tok][j], sh.key[tok][j + 1]))
      open |= !same(sh.id[tok][j], sh.id[tok][j + 1]);
  }
  const uint32_t last = sh.key[tok][a.topk - 1];
  if (near(last, s[0])) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (near(last, s[v]))
        open |= !same(sh.id[tok][a.topk - 1], at0.first + (int)(kPlace - (s[v] & kPlace)));
  }
  // (a lane's own finding is its token's)
  open = group_max<G>(open ? 1u : 0u) != 0u;
  if (__builtin_expect(__ballot(open || all) != 0, 0)) {
    // Mostly two neighbours: the chosen and the next one are ranked by their exact
    // values.  Where that does not settle it (more behind the next one, a softmax's
    // sum, NaN), all of it again.
    take(a.topk);
    lds_order();
    all |= open && ((!by_logit && a.score == kScoreSoftmax) || near(last, s[0]));
    auto above = [](double c, int e, double d, int f) { return c > d || (c == d && (uint32_t)e < (uint32_t)f); };
    const int next = sh.id[tok][a.topk];
    const double cn = exact(next);
    double c[KO];
    int e[KO], rank[KO], below = 0;   // of the slots, that are above the next one
    all |= open && cn != cn;
#pragma unroll
    for (int o = 0; o < KO; ++o) {
      const int j = o * G + g;
      e[o] = j < a.topk ? sh.id[tok][j] : -1;
      c[o] = exact(e[o]);
      all |= open && c[o] != c[o];
      rank[o] = above(cn, next, c[o], e[o]) ? 1 : 0;
    }
#pragma unroll
    for (int o = 0; o < KO; ++o) {
#pragma unroll 1
      for (int i = 0; i < G; ++i) {
        const int src = (lane & ~(G - 1)) + i;
        const double d = __shfl(c[o], src, 64);
        const int f = __shfl(e[o], src, 64);
        below += above(d, f, cn, next) ? 1 : 0;
#pragma unroll
        for (int q = 0; q < KO; ++q) rank[q] += above(d, f, c[q], e[q]) ? 1 : 0;
      }
    }
    lds_order();
    if (open) {   // (the wavefront's other tokens are as they were)
#pragma unroll
      for (int o = 0; o < KO; ++o)
        if (o * G + g < a.topk) sh.id[tok][o * G + g] = -1;
      lds_order();
#pragma unroll
      for (int o = 0; o < KO; ++o)
        if (e[o] >= 0 && rank[o] < a.topk) sh.id[tok][rank[o]] = e[o];
      if (g == 0 && next >= 0 && below < a.topk) sh.id[tok][below] = next;
    }
    lds_order();
    if (__ballot(all) != 0) choose64<T, G, V>(row, a, g, tok, sh);
  }

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
  const float sum = a.renorm ? group_sum<G>(part) : 1.0f;
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    const int j = o * G + g;
    if (live && j < a.topk) {
      a.ids[t * a.topk + j] = id[o];
      a.weights[t * a.topk + j] = id[o] < 0 || sum == 0.0f ? 0.0f : x[o] / sum * a.scale;
    }
  }
}

// With D_j = scale dw_j of the chosen, and m the weighted mean of D:
//   sigmoid:  dl_j = (D_j - m) w_j (1 - s_j), renormalised; D_j s_j (1 - s_j) else
//   softmax:  dl_j = (D_j - m) w_j over the chosen, renormalised; over all experts else
// The chosen few are scattered into the token's zeros in LDS, and whole rows
// written.  Bound by memory: 65521 tokens of 256 experts fp32 18 us (67 MB written
// and 36 read, a line for each chosen logit).
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
    }
    float mean = 0.0f;
    if (a.renorm) {
      // divided, not multiplied by 1 / sum: one expert alone has the weight 1, and no gradient
      const float sum = group_sum<G>(part);
#pragma unroll
      for (int o = 0; o < KO; ++o) {
        x[o] = sum == 0.0f ? 0.0f : x[o] / sum;
        dot = __builtin_fmaf(x[o], d[o], dot);
      }
      mean = group_sum<G>(dot);
    }
#pragma unroll
    for (int o = 0; o < KO; ++o)
      if (id[o] >= 0) img[tok][id[o]] = (d[o] - mean) * x[o] * rest[o];
    lds_order();
  }
  float f[V];
  if (dense) {
#pragma unroll
    for (int o = 0; o < KO; ++o)
      if (id[o] >= 0) img[tok][id[o]] = d[o];
    lds_order();
    float l[V];
    load_run<T, V>(row, g * V, a.experts - g * V, l);
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

template <typename T, int G, int V>
void groups_gv(const T* l, const RouteGroups& a, hipStream_t st) {
  in_launches(a.tokens, 256 / G, [&](int64_t t, int64_t n) {
    RouteGroups b = a;
    b.tokens = n;
    b.ids += t * a.topk;
    b.weights += t * a.topk;
    k_route_groups<T, G, V><<<dim3((unsigned)((n + 256 / G - 1) / (256 / G))), 256, 0, st>>>(l + t * a.ld, b);
  });
}

// Lanes a token and experts a lane: sixteen, for a wavefront's rounds serve all its tokens (65521 x 256,
// without the second looks: eight experts on each of 32 lanes 48 us, sixteen on each of 16 29 us), eight
// where sixteen would need as many lanes.  A group takes whole lanes; with 32 experts a lane any division
// fits 64 lanes.
template <typename T>
void groups_t(const T* l, RouteGroups a, hipStream_t st) {
  if (a.topk_groups == a.groups) {   // no group matters
    a.groups = a.topk_groups = 1;
    a.gsize = a.experts;
  }
  auto lanes = [&](int v) {
    int need = a.groups * ((a.gsize + v - 1) / v), g = 1;
    while (g < need) g *= 2;
    return g;
  };
  auto shape = [&](int v) {
    a.group_lanes = (a.gsize + v - 1) / v;
    a.lanes_inv = (((uint64_t)1 << 32) + (uint64_t)a.group_lanes - 1) / (uint64_t)a.group_lanes;
  };
  const int g8 = lanes(8), g16 = lanes(16);
  if (g8 <= 4) {
    shape(8);
    if (g8 == 1) groups_gv<T, 1, 8>(l, a, st);
    else if (g8 == 2) groups_gv<T, 2, 8>(l, a, st);
    else groups_gv<T, 4, 8>(l, a, st);
  } else if (g8 <= 16 && g16 == g8) {   // sixteen a lane need as many: eight
    shape(8);
    if (g8 == 8) groups_gv<T, 8, 8>(l, a, st);
    else groups_gv<T, 16, 8>(l, a, st);
  } else if (g16 <= 64) {
    shape(16);
    if (g16 <= 4) groups_gv<T, 4, 16>(l, a, st);
    else if (g16 == 8) groups_gv<T, 8, 16>(l, a, st);
    else if (g16 == 16) groups_gv<T, 16, 16>(l, a, st);
    else if (g16 == 32) groups_gv<T, 32, 16>(l, a, st);
    else groups_gv<T, 64, 16>(l, a, st);
  } else {
    shape(32);
    groups_gv<T, 64, 32>(l, a, st);
  }
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
