// Mixture-of-experts routing and token exchange for gfx950: the router's
// top-k weights and their gradient, the stable order of the routed rows by
// expert (the segment offsets every grouped call takes), tokens to their
// experts' rows and back, and the gradients of both.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_common.hpp"
#include "launch.hpp"

namespace averis {
namespace {

// ---------------------------------------------------------------------------
// 16-byte pieces at element alignment: gfx950 loads and stores them at any
// address, so one path serves every stride and offset
// ---------------------------------------------------------------------------
typedef u32x4_t piece_t __attribute__((aligned(2)));

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {   // bf16 bits
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float f32(uint16_t v) { return bf16_lo(v); }
  static __device__ __forceinline__ uint16_t from(float v) { return (uint16_t)bf16x2_rne(v, 0.0f); }
  static __device__ __forceinline__ void unpack(u32x4_t p, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(p[i]);
      f[2 * i + 1] = bf16_hi(p[i]);
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    return u32x4_t{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                   bf16x2_rne(f[6], f[7])};
  }
};
template <>
struct Elem<float> {
  static constexpr int kPer = 4;
  static __device__ __forceinline__ float f32(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
  static __device__ __forceinline__ void unpack(u32x4_t p, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(p[i]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    return u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3])};
  }
};

// elements c .. c + kPer - 1 of a row of `cols` (those past the end are 0)
template <typename T>
__device__ __forceinline__ u32x4_t load_piece(const T* row, int64_t c, int64_t cols) {
  constexpr int P = Elem<T>::kPer;
  if (c + P <= cols) return *reinterpret_cast<const piece_t*>(row + c);
  // the row's last elements: all loads at once, those past the end of its last
  // element
  u32x4_t v = {0u, 0u, 0u, 0u};
  T e[P];
#pragma unroll
  for (int i = 0; i < P; ++i) e[i] = row[c + i < cols ? c + i : cols - 1];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (sizeof(T) == 2)
      v[i / 2] |= (c + i < cols ? (uint32_t)e[i] : 0u) << (16 * (i & 1));
    else
      v[i] = c + i < cols ? __float_as_uint(e[i]) : 0u;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store_piece(T* row, int64_t c, int64_t cols, u32x4_t v) {
  constexpr int P = Elem<T>::kPer;
  if (c + P <= cols) {
    *reinterpret_cast<piece_t*>(row + c) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (c + i < cols) {
      if constexpr (sizeof(T) == 2)
        row[c + i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
      else
        row[c + i] = __uint_as_float(v[i]);
    }
  }
}

// ---------------------------------------------------------------------------
// reductions over groups of G neighbouring lanes (butterflies: every lane of
// the group gets the result).  The mirrors pair the halves of 8 and 16 lanes
// once those halves agree.
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
  else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
  else if constexpr (D == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);
  else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);
  else return (uint32_t)__shfl_xor((int)v, D, 64);
}
template <int G, typename F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F op) {
  if constexpr (G > 1) v = op(v, partner<1>(v));
  if constexpr (G > 2) v = op(v, partner<2>(v));
  if constexpr (G > 4) v = op(v, partner<4>(v));
  if constexpr (G > 8) v = op(v, partner<8>(v));
  if constexpr (G > 16) v = op(v, partner<16>(v));
  if constexpr (G > 32) v = op(v, partner<32>(v));
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int G>
__device__ __forceinline__ float group_fmax(float v) {
  return __uint_as_float(group_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__builtin_fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}

// ---------------------------------------------------------------------------
// Router.  G lanes share a token; a lane has V of its logits in pieces of Q
// neighbours, dealt out lane by lane, so that a load of all the lanes takes
// neighbouring bytes.
// ---------------------------------------------------------------------------
constexpr float kMasked = -__builtin_inff();

template <typename T, int G, int V>
struct Deal {
  static constexpr int Q = V < Elem<T>::kPer ? V : Elem<T>::kPer;
  // expert of the lane's v-th logit
  static __device__ __forceinline__ int expert(int g, int v) { return (v / Q * G + g) * Q + v % Q; }
  // the lane's v of expert e, V or more if it is another lane's
  static __device__ __forceinline__ uint32_t place(int g, int e) {
    const uint32_t u = (uint32_t)e, v = u / (Q * G) * Q + u % Q;
    return u / Q % G == (uint32_t)g ? v : 0xFFFFu;
  }
};

template <typename T, int G, int V>
__device__ __forceinline__ void load_logits(const T* row, int g, int experts, float* l) {
  using D = Deal<T, G, V>;
  if constexpr (D::Q == Elem<T>::kPer) {
    if (D::expert(G - 1, V - 1) < experts) {
#pragma unroll
      for (int v = 0; v < V; v += D::Q)
        Elem<T>::unpack(*reinterpret_cast<const piece_t*>(row + D::expert(g, v)), l + v);
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = D::expert(g, v);
    l[v] = e < experts ? Elem<T>::f32(row[e]) : kMasked;
  }
}

// A logit's key orders as its value (NaN above +inf, -0 equal to +0); 0 stands
// for masked, absent and taken.  A bf16 value takes half of it, and the other
// half holds the expert, the lowest on top.
template <typename T>
__device__ __forceinline__ uint32_t logit_key(float l, uint32_t e) {
  uint32_t k = f32_ordered(l + 0.0f);
  if (l != l) k = 0xFFFFFFFFu;
  if constexpr (sizeof(T) == 2) k = (k & 0xFFFF0000u) | (0xFFFFu - e);
  return l == kMasked ? 0u : k;
}
template <typename T>
__device__ __forceinline__ float key_logit(uint32_t k) {
  if constexpr (sizeof(T) == 2) k = (k & 0x80000000u) ? k & 0xFFFF0000u : k | 0xFFFFu;
  return f32_from_ordered(k);
}

// Top-k by k rounds of a group maximum over the lane's V and the group.  bf16:
// the key names the expert.  fp32: the smallest expert that has the key; all
// that have it are taken out as they are found, and put back where there were
// several (the wavefront's count of them says so), against one search and one
// removal: 65521 tokens, 128 experts, top 6, 16.0 -> 15.0 us (33.5 MB, 2.2
// TB/s).  Bound by vector instructions at many tokens, by latency at few (16
// tokens 2.7 us).
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void k_route(const T* __restrict__ logits, int64_t tokens,
                                               int experts, int64_t ld, int topk, int renorm,
                                               int32_t* __restrict__ ids,
                                               float* __restrict__ weights) {
  constexpr int KO = kMaxTopk > G ? kMaxTopk / G : 1;
  using D = Deal<T, G, V>;
  const int g = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const bool live = t < tokens;   // the others repeat the last token, unstored
  const T* row = logits + (live ? t : tokens - 1) * ld;
  float l[V];
  load_logits<T, G, V>(row, g, experts, l);
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = logit_key<T>(l[v], (uint32_t)D::expert(g, v));
  float top = 0.0f;          // the largest logit
  float val[KO];
  int id[KO];
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    val[o] = kMasked;
    id[o] = -1;
    const int rounds = topk - o * G < G ? topk - o * G : G;
    for (int r = 0; r < rounds; ++r) {
      uint32_t best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
      best = group_max<G>(best);
      uint32_t at;
      if constexpr (sizeof(T) == 2) {
        at = 0xFFFFu - (best & 0xFFFFu);
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key[v] == best ? 0u : key[v];
      } else {
        const uint32_t pick = best != 0u ? best : 1u;   // (1 is no logit's key)
        at = 0xFFFFu;
        int hits = 0;   // of all the wavefront's tokens
#pragma unroll
        for (int v = V - 1; v >= 0; --v) {
          const bool hit = key[v] == pick;
          hits += __builtin_popcountll(__ballot(hit));
          at = hit ? (uint32_t)D::expert(g, v) : at;
          key[v] = hit ? 0u : key[v];
        }
        at = group_min<G>(at);
        if (hits != __builtin_popcountll(__ballot(best != 0u)) / G) {
          // equal logits: those behind the lowest expert go back
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (logit_key<T>(l[v], 0u) == pick && (uint32_t)D::expert(g, v) > at) key[v] = pick;
        }
      }
      const float x = key_logit<T>(best);
      if (o == 0 && r == 0 && best != 0u) top = x;
      if (r == g && best != 0u) {
        val[o] = x;
        id[o] = (int)at;
      }
    }
  }
  // softmax against the largest logit; masked ones give exp(-inf) = 0
  float part = 0.0f;
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    val[o] = expf(val[o] - top);
    if (renorm) part += val[o];
  }
  if (!renorm) {
#pragma unroll
    for (int v = 0; v < V; ++v) part += expf(l[v] - top);
  }
  float total = group_sum<G>(part);
  if (total == 0.0f) total = 1.0f;   // no open expert
#pragma unroll
  for (int o = 0; o < KO; ++o) {
    const int j = o * G + g;
    if (live && j < topk) {
      ids[t * topk + j] = id[o];
      // (without an expert 0, also where a NaN or an infinity makes the others' NaN)
      weights[t * topk + j] = id[o] < 0 ? 0.0f : val[o] / total;
    }
  }
}

// w = softmax over the chosen (renorm) or all logits.  With s_e = dweights of
// the slot that chose e (0 if none) and m = sum over the chosen of w s:
// dl_e = w_e (s_e - m), zero outside the chosen when renorm.  65521 tokens, 128
// experts fp32: 15.4 us (67 MB, 4.4 TB/s).  w is exp times the sum's reciprocal,
// a rounding more than the quotient of k_route (quotients here: 14.5 -> 15.9 us
// back to back, error 6.8e-8 -> 6.7e-8 of the norm).
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void k_route_grad(const T* logits, int64_t tokens,
                                                    int experts, int64_t ld, int topk, int renorm,
                                                    const int32_t* __restrict__ ids,
                                                    const float* __restrict__ dweights,
                                                    T* dlogits, int64_t ldd) {
  using D = Deal<T, G, V>;
  const int g = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const bool live = t < tokens;
  const int64_t tr = live ? t : tokens - 1;
  float l[V], s[V];
  load_logits<T, G, V>(logits + tr * ld, g, experts, l);
  uint32_t chosen = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = 0.0f;
  for (int j0 = 0; j0 < topk; j0 += 8) {   // eight slots' loads in flight
    int e[8];
    float d[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      e[u] = -1;
      d[u] = 0.0f;
      if (j0 + u < topk) {
        e[u] = ids[tr * topk + j0 + u];
        d[u] = dweights[tr * topk + j0 + u];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t mine = D::place(g, e[u]);
      if (j0 + u < topk && e[u] >= 0) {
        chosen |= mine < (uint32_t)V ? 1u << (mine & 31u) : 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = mine == (uint32_t)v ? d[u] : s[v];
      }
    }
  }
  float top = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) top = __builtin_fmaxf(top, l[v]);
  top = group_fmax<G>(top);
  if (top == kMasked) top = 0.0f;
  float total = 0.0f, mean = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool in = (chosen >> v) & 1u;
    l[v] = (in || !renorm) ? expf(l[v] - top) : 0.0f;
    total += l[v];
    if (in) mean = __builtin_fmaf(l[v], s[v], mean);
  }
  total = group_sum<G>(total);
  mean = group_sum<G>(mean);
  if (total == 0.0f) total = 1.0f;
  const float inv = 1.0f / total;
  mean *= inv;
  if (!live) return;
  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool in = (chosen >> v) & 1u;
    d[v] = (in || !renorm) ? l[v] * inv * (s[v] - mean) : 0.0f;
  }
  T* out = dlogits + t * ldd;
  if constexpr (D::Q == Elem<T>::kPer) {
    if (D::expert(G - 1, V - 1) < experts) {
#pragma unroll
      for (int v = 0; v < V; v += D::Q)
        *reinterpret_cast<piece_t*>(out + D::expert(g, v)) = Elem<T>::pack(d + v);
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (D::expert(g, v) < experts) out[D::expert(g, v)] = Elem<T>::from(d[v]);
}

// ---------------------------------------------------------------------------
// Stable counting sort of the slots by expert.  A slot without a valid expert
// goes to bucket `experts`, the tail.  Each wavefront owns a run of slots:
// its counts per bucket are turned into its first rows per bucket (buckets,
// then wavefronts, in order), then it ranks its slots 64 at a time by ballots
// over the bucket's bits.  No step depends on the order of atomics.  Bound by
// the latency of its launches: 32768 slots, 64 experts 8.7 us (0.4 MB), 393120
// slots, 128 experts 13.2 us.
// ---------------------------------------------------------------------------

__device__ __forceinline__ int bucket_of(int32_t id, int experts) {
  return (uint32_t)id < (uint32_t)experts ? id : experts;
}

// exclusive prefix sum over the block's threads; total: the whole sum.
// sh: one int per wavefront
template <int WAVES>
__device__ __forceinline__ int block_exclusive(int v, int* sh, int& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(incl, d, 64);
    if (lane >= d) incl += u;
  }
  if (lane == 63) sh[w] = incl;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    const int s = sh[i];
    if (i < w) before += s;
    total += s;
  }
  __syncthreads();
  return before + incl - v;
}

// the wavefront's slots (registers) and its counts, in cnt[wave][bucket]
template <int WAVES, int STEPS>
__device__ __forceinline__ void sort_count(const int32_t* ids, int64_t first, int64_t n,
                                           int experts, int* cnt, int* b) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nb = experts + 1;
  const int64_t s0 = first + (int64_t)w * (64 * STEPS);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t s = s0 + 64 * i + lane;
    b[i] = s < n ? bucket_of(ids[s], experts) : -1;
  }
  for (int i = threadIdx.x; i < WAVES * nb; i += 64 * WAVES) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    if (b[i] >= 0) atomicAdd(&cnt[w * nb + b[i]], 1);
  __syncthreads();
}

// rows of the wavefront's slots from its first rows in cnt[wave][bucket]
template <int STEPS>
__device__ __forceinline__ void sort_place(int64_t first, int64_t n, int experts, int* cnt,
                                           const int* b, int32_t* pos, int32_t* src) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nb = experts + 1;
  const int64_t s0 = first + (int64_t)w * (64 * STEPS);
  const uint64_t below = (1ull << lane) - 1ull;
  const int bits = 32 - __builtin_clz(experts);   // buckets 0 .. experts
  volatile int* row0 = cnt + w * nb;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    if (s0 + 64 * i >= n) break;
    const bool ok = b[i] >= 0;
    uint64_t same = __ballot(ok);
    for (int k = 0; k < bits; ++k) {
      const bool one = (b[i] >> k) & 1;
      const uint64_t m = __ballot(one);
      same &= one ? m : ~m;
    }
    if (ok) {
      const int rank = __builtin_popcountll(same & below);
      const int p = row0[b[i]];          // all lanes read before the leaders write:
      __builtin_amdgcn_wave_barrier();   // one wavefront's LDS accesses are in order
      if (rank == 0) row0[b[i]] = p + __builtin_popcountll(same);
      const int r = p + rank;
      const int64_t s = s0 + 64 * i + lane;
      pos[s] = b[i] < experts ? r : ~r;
      if (src) src[r] = (int32_t)s;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// One workgroup does everything up to 8192 slots (one / several workgroups, us,
// 64 experts: 128 slots 4.4 / 7.5, 4096 7.8 / 9.3, 8192 9.2 / 9.7).
constexpr int kSortWavesOne = 16, kSortStepsOne = 8;     // one workgroup for everything
constexpr int kSortWavesMany = 4, kSortStepsMany = 4;    // workgroups of a larger sort
constexpr int64_t kSortOne = (int64_t)kSortWavesOne * 64 * kSortStepsOne;       // 8192 slots
constexpr int64_t kSortChunk = (int64_t)kSortWavesMany * 64 * kSortStepsMany;   // 1024 slots

__global__ __launch_bounds__(64 * kSortWavesOne) void k_sort_one(
    const int32_t* __restrict__ ids, int n, int experts, int64_t* __restrict__ offsets,
    int32_t* __restrict__ pos, int32_t* __restrict__ src) {
  extern __shared__ int cnt[];   // [waves][experts + 1]
  __shared__ int sh[kSortWavesOne];
  int b[kSortStepsOne];
  const int nb = experts + 1;
  sort_count<kSortWavesOne, kSortStepsOne>(ids, 0, n, experts, cnt, b);
  // thread e: expert e (experts <= the block's threads); the tail after them
  const int e = threadIdx.x;
  int mine = 0;
  if (e < experts)
    for (int w = 0; w < kSortWavesOne; ++w) mine += cnt[w * nb + e];
  int kept;
  const int before = block_exclusive<kSortWavesOne>(mine, sh, kept);
  auto rows_of = [&](int bkt, int run) {
    for (int w = 0; w < kSortWavesOne; ++w) {
      const int c = cnt[w * nb + bkt];
      cnt[w * nb + bkt] = run;
      run += c;
    }
  };
  if (e < experts) {
    rows_of(e, before);
    offsets[e] = before;
  }
  if (e == 0) {
    rows_of(experts, kept);
    offsets[experts] = kept;
  }
  __syncthreads();
  sort_place<kSortStepsOne>(0, n, experts, cnt, b, pos, src);
}

// counts of a chunk -> hist[bucket][chunk]
__global__ __launch_bounds__(64 * kSortWavesMany) void k_sort_hist(
    const int32_t* __restrict__ ids, int64_t n, int experts, int chunks, int* __restrict__ hist) {
  extern __shared__ int cnt[];
  int b[kSortStepsMany];
  sort_count<kSortWavesMany, kSortStepsMany>(ids, (int64_t)blockIdx.x * kSortChunk, n, experts, cnt, b);
  const int nb = experts + 1;
  for (int e = threadIdx.x; e < nb; e += 64 * kSortWavesMany) {
    int c = 0;
    for (int w = 0; w < kSortWavesMany; ++w) c += cnt[w * nb + e];
    hist[(int64_t)e * chunks + blockIdx.x] = c;
  }
}

// many chunks: a bucket's counts -> the slots of it in the chunks before, and all of them in
// totals[bucket]: a wavefront a bucket, 64 chunks at a time, eight such loads in
// flight
__global__ __launch_bounds__(256) void k_sort_scan(int* __restrict__ hist, int experts, int chunks,
                                                   int* __restrict__ totals) {
  const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e > experts) return;
  int* row = hist + (int64_t)e * chunks;
  int run = 0;
  for (int c0 = 0; c0 < chunks; c0 += 64 * 8) {
    int v[8];   // all loads at once
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = c0 + 64 * u + lane;
      v[u] = c < chunks ? row[c] : 0;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (c0 + 64 * u >= chunks) break;
      const int c = c0 + 64 * u + lane;
      int incl = v[u];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int t = __shfl_up(incl, d, 64);
        if (lane >= d) incl += t;
      }
      if (c < chunks) row[c] = run + incl - v[u];
      run += __shfl(incl, 63, 64);
    }
  }
  if (lane == 0) totals[e] = run;
}

// each workgroup sums the buckets' totals for itself: the offsets.  hist and
// totals as k_sort_scan left them, or the counts and no totals
__global__ __launch_bounds__(64 * kSortWavesMany) void k_sort_place(
    const int32_t* __restrict__ ids, int64_t n, int experts, int chunks,
    const int* __restrict__ hist, const int* __restrict__ totals, int64_t* __restrict__ offsets,
    int32_t* __restrict__ pos, int32_t* __restrict__ src) {
  extern __shared__ int cnt[];
  __shared__ int sh[kSortWavesMany];
  constexpr int T = 64 * kSortWavesMany;
  int b[kSortStepsMany];
  const int64_t first = (int64_t)blockIdx.x * kSortChunk;
  sort_count<kSortWavesMany, kSortStepsMany>(ids, first, n, experts, cnt, b);
  const int nb = experts + 1;
  int before = 0;   // rows of the buckets of earlier rounds
  for (int e0 = 0; e0 < nb; e0 += T) {
    const int e = e0 + threadIdx.x;
    int all;
    // slots of the bucket: all, and in the chunks before
    int mine = 0, pre = 0;
    if (e < nb) {
      const int* row = hist + (int64_t)e * chunks;
      if (totals) {
        mine = totals[e];
        pre = row[blockIdx.x];
      } else {
        for (int c0 = 0; c0 < chunks; c0 += 16) {   // sixteen loads in flight
          int v[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) v[u] = c0 + u < chunks ? row[c0 + u] : 0;
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            pre += c0 + u < (int)blockIdx.x ? v[u] : 0;
            mine += v[u];
          }
        }
      }
    }
    const int start = before + block_exclusive<kSortWavesMany>(mine, sh, all);
    before += all;
    if (e >= nb) continue;
    if (blockIdx.x == 0) offsets[e] = start;   // offsets[experts]: the tail's first row
    int run = start + pre;
    for (int w = 0; w < kSortWavesMany; ++w) {
      const int c = cnt[w * nb + e];
      cnt[w * nb + e] = run;
      run += c;
    }
  }
  __syncthreads();
  sort_place<kSortStepsMany>(first, n, experts, cnt, b, pos, src);
}

__global__ void k_zero_offsets(int64_t* offsets, int count) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < count) offsets[i] = 0;
}

// ---------------------------------------------------------------------------
// Token exchange.  blockDim.x lanes (whole wavefronts) go along a token's
// columns in 16-byte pieces, blockDim.y tokens to a workgroup.  Rows outside
// the slots there are (those of all the call's launches), which only malformed
// positions name, are neither read nor written.  All four are bound by memory:
// a row is read or written once, whole, in lines; sums are fp32, rounded once.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// A token is read once and written to its k rows.  4096 tokens, top 8, 2048
// bf16: 26.3 us (151 MB, 5.7 TB/s).  Streaming stores made the rows 10 % sooner
// written, and what reads them next slower by more (4096 tokens and their fp8
// quantization 55.2 us, with streaming stores 57.3).
template <typename T>
__global__ __launch_bounds__(256) void k_dispatch(const T* __restrict__ x, int64_t tokens,
                                                  int64_t cols, int64_t ldx,
                                                  const int32_t* __restrict__ pos, int topk,
                                                  T* __restrict__ rows, int64_t ldr, int64_t slots) {
  constexpr int P = Elem<T>::kPer;
  const int64_t t = uniform64((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= tokens) return;
  const int32_t* pt = pos + t * topk;
  for (int64_t c = (int64_t)threadIdx.x * P; c < cols; c += (int64_t)blockDim.x * P) {
    const u32x4_t v = load_piece(x + t * ldx, c, cols);
    for (int j = 0; j < topk; ++j) {
      const int p = pt[j];
      const int64_t r = p < 0 ? ~p : p;
      if (r < slots) store_piece(rows + r * ldr, c, cols, p < 0 ? u32x4_t{0u, 0u, 0u, 0u} : v);
    }
  }
}

// y_t = sum_j w_tj rows[pos_tj], slots in order, fp32; eight rows in flight.
// 4096 tokens, top 8, 2048 bf16: 35.8 us (151 MB, 4.2 TB/s).
template <typename T, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_combine(const T* __restrict__ rows, int64_t tokens,
                                                 int64_t cols, int64_t ldr,
                                                 const int32_t* __restrict__ pos,
                                                 const float* __restrict__ weights, int topk,
                                                 T* __restrict__ y, int64_t ldy, int64_t slots) {
  constexpr int P = Elem<T>::kPer, U = 8;
  const int64_t t = uniform64((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= tokens) return;
  for (int64_t c = (int64_t)threadIdx.x * P; c < cols; c += (int64_t)blockDim.x * P) {
    float acc[P];
#pragma unroll
    for (int e = 0; e < P; ++e) acc[e] = 0.0f;
    for (int j0 = 0; j0 < topk; j0 += U) {
      u32x4_t v[U];
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = j0 + u < topk ? pos[t * topk + j0 + u] : -1;
        w[u] = 0.0f;
        v[u] = u32x4_t{0u, 0u, 0u, 0u};
        if (p >= 0 && p < slots) {
          v[u] = load_piece(rows + (int64_t)p * ldr, c, cols);
          w[u] = WEIGHTED ? weights[t * topk + j0 + u] : 1.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[P];
        Elem<T>::unpack(v[u], f);
#pragma unroll
        for (int e = 0; e < P; ++e)
          acc[e] = WEIGHTED ? __builtin_fmaf(w[u], f[e], acc[e]) : acc[e] + f[e];
      }
    }
    store_piece(y + t * ldy, c, cols, Elem<T>::pack(acc));
  }
}

// drows[pos_tj] = w_tj dy_t and dweights_tj = <dy_t, rows[pos_tj]>: one
// wavefront a slot, neighbouring slots share dy_t through the cache.  4096
// tokens, top 8, 2048 bf16: 50.9 us (285 MB, 5.6 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_combine_grad(const T* __restrict__ dy, int64_t here,
                                                      int64_t cols, int64_t ldy,
                                                      const T* rows, int64_t ldr,
                                                      const int32_t* __restrict__ pos,
                                                      const float* __restrict__ weights, int topk,
                                                      T* drows, int64_t lddr,
                                                      float* __restrict__ dweights, int64_t slots) {
  constexpr int P = Elem<T>::kPer;
  const int lane = threadIdx.x & 63;
  const uint32_t s = __builtin_amdgcn_readfirstlane(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (s >= (uint64_t)here) return;
  const int p = pos[s];
  const bool kept = p >= 0 && p < slots;
  const int64_t r = p < 0 ? ~p : p;
  const float w = kept ? weights[s] : 0.0f;
  const T* g = dy + (int64_t)(s / (uint32_t)topk) * ldy;
  float dot = 0.0f;
  for (int64_t c = (int64_t)lane * P; c < cols; c += 64 * P) {
    u32x4_t out = {0u, 0u, 0u, 0u};
    if (kept) {
      float a[P], b[P];
      Elem<T>::unpack(load_piece(g, c, cols), a);
      Elem<T>::unpack(load_piece(rows + r * ldr, c, cols), b);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        dot = __builtin_fmaf(a[e], b[e], dot);
        a[e] *= w;
      }
      out = Elem<T>::pack(a);
    }
    if (r < slots) store_piece(drows + r * lddr, c, cols, out);
  }
  dot = group_sum<64>(dot);
  if (lane == 0) dweights[s] = dot;
}

// As many wavefronts along a row as it has pieces for, four at most; the rest of
// the workgroup takes other tokens (us, dispatch and combine, top 8, bf16; by
// this rule / one wavefront a row / four): 16 tokens of 2048 columns 2.9 3.3 /
// 5.8 7.3 / 3.4 3.3; 4096 of 256 5.9 5.2 / 5.9 5.1 / 6.4 6.6; 4096 of 4096 57.4
// 49.0 / 63.8 54.3 / 57.1 51.4.
dim3 exchange_block(int64_t cols, int per) {
  const int64_t pieces = (cols + per - 1) / per;
  int x = 64;
  while (x < 256 && x < pieces) x *= 2;
  return dim3((unsigned)x, (unsigned)(256 / x));
}

}  // namespace

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Lanes per token and logits per lane by the number of experts: as few lanes as
// keep the logits in registers.  Twice the lanes (half the logits) is faster
// for few tokens and slower for many, half the lanes the other way round (us,
// half / these / twice the lanes, bf16, route and gradient): 4096 tokens of 64
// experts 4.4 4.7 / 3.6 3.8 / 3.3 3.6, of 256 5.8 6.6 / 4.3 5.0 / 4.0 4.3; 65536
// of 64 7.7 8.2 / 8.0 8.6 / 10.5 11.9, of 256 18.4 23.7 / 18.7 24.3 / 23.4 26.1.
#define AVERIS_ROUTE_SHAPES(CALL)      \
  if (experts <= 8) {                  \
    CALL(8, 1);                        \
  } else if (experts <= 32) {          \
    CALL(8, 4);                        \
  } else if (experts <= 64) {          \
    CALL(8, 8);                        \
  } else if (experts <= 128) {         \
    CALL(8, 16);                       \
  } else if (experts <= 256) {         \
    CALL(16, 16);                      \
  } else if (experts <= 512) {         \
    CALL(32, 16);                      \
  } else {                             \
    CALL(64, 16);                      \
  }

// A grid has fewer than 2^32 threads (workgroups of 256 here): f(first, many)
// for each launch of n tokens, `per` of them a workgroup.
template <typename F>
static void in_launches(int64_t n, int64_t per, F f) {
  const int64_t most = ((1 << 24) - 1) * per;
  for (int64_t i = 0; i < n; i += most) f(i, n - i < most ? n - i : most);
}

template <typename T>
static void route_t(const T* l, int64_t tokens, int experts, int64_t ld, int topk, bool renorm,
                    int32_t* ids, float* w, hipStream_t st) {
#define AVERIS_ROUTE(G, V)                                                                      \
  in_launches(tokens, 256 / G, [&](int64_t t, int64_t n) {                                      \
    k_route<T, G, V><<<dim3((unsigned)((n + 256 / G - 1) / (256 / G))), 256, 0, st>>>(           \
        l + t * ld, n, experts, ld, topk, renorm, ids + t * topk, w + t * topk);                \
  })
  AVERIS_ROUTE_SHAPES(AVERIS_ROUTE)
#undef AVERIS_ROUTE
}

template <typename T>
static void route_grad_t(const T* l, int64_t tokens, int experts, int64_t ld, int topk,
                         bool renorm, const int32_t* ids, const float* dw, T* dl, int64_t ldd,
                         hipStream_t st) {
#define AVERIS_ROUTE(G, V)                                                                      \
  in_launches(tokens, 256 / G, [&](int64_t t, int64_t n) {                                      \
    k_route_grad<T, G, V><<<dim3((unsigned)((n + 256 / G - 1) / (256 / G))), 256, 0, st>>>(      \
        l + t * ld, n, experts, ld, topk, renorm, ids + t * topk, dw + t * topk, dl + t * ldd,  \
        ldd);                                                                                   \
  })
  AVERIS_ROUTE_SHAPES(AVERIS_ROUTE)
#undef AVERIS_ROUTE
}

hipError_t launch_moe_route(const void* logits, bool bf16, int64_t tokens, int experts, int64_t ld,
                            int topk, bool renorm, int32_t* ids, float* weights, hipStream_t st) {
  if (tokens == 0) return hipSuccess;
  if (bf16)
    route_t(static_cast<const uint16_t*>(logits), tokens, experts, ld, topk, renorm, ids, weights,
            st);
  else
    route_t(static_cast<const float*>(logits), tokens, experts, ld, topk, renorm, ids, weights,
            st);
  return hipGetLastError();
}

hipError_t launch_moe_route_grad(const void* logits, bool bf16, int64_t tokens, int experts,
                                 int64_t ld, int topk, bool renorm, const int32_t* ids,
                                 const float* dweights, void* dlogits, int64_t ldd,
                                 hipStream_t st) {
  if (tokens == 0) return hipSuccess;
  if (bf16)
    route_grad_t(static_cast<const uint16_t*>(logits), tokens, experts, ld, topk, renorm, ids,
                 dweights, static_cast<uint16_t*>(dlogits), ldd, st);
  else
    route_grad_t(static_cast<const float*>(logits), tokens, experts, ld, topk, renorm, ids,
                 dweights, static_cast<float*>(dlogits), ldd, st);
  return hipGetLastError();
}

static int64_t sort_chunks(int64_t slots) { return (slots + kSortChunk - 1) / kSortChunk; }

size_t moe_sort_ws_bytes(int64_t slots, int experts) {
  if (slots <= kSortOne) return 0;
  // counts [bucket][chunk], totals [bucket]
  return (((size_t)sort_chunks(slots) + 1) * (size_t)(experts + 1) * 4 + 255) & ~(size_t)255;
}

hipError_t launch_moe_sort(const int32_t* ids, int64_t slots, int experts, int64_t* offsets,
                           int32_t* pos, int32_t* src, void* ws, hipStream_t st) {
  if (slots == 0) {
    k_zero_offsets<<<dim3((unsigned)((experts + 256) / 256)), 256, 0, st>>>(offsets, experts + 1);
    return hipGetLastError();
  }
  if (slots <= kSortOne) {
    const size_t lds = (size_t)kSortWavesOne * (experts + 1) * 4;
    const hipError_t e = lds_attr_once<&k_sort_one>(kSortWavesOne * (kMaxExperts + 1) * 4);
    if (e != hipSuccess) return e;
    k_sort_one<<<1, 64 * kSortWavesOne, lds, st>>>(ids, (int)slots, experts, offsets, pos, src);
    return hipGetLastError();
  }
  const int chunks = (int)sort_chunks(slots);
  const size_t lds = (size_t)kSortWavesMany * (experts + 1) * 4;
  int* hist = static_cast<int*>(ws);
  k_sort_hist<<<chunks, 64 * kSortWavesMany, lds, st>>>(ids, slots, experts, chunks, hist);
  int* totals = hist + (int64_t)(experts + 1) * chunks;
  // few counts: every workgroup reads its buckets' whole rows, a launch less
  // (scanned / unscanned, us, 64 experts: 16384 slots 9.6 / 8.0, 32768 9.7 /
  // 8.7, 65536 9.7 / 10.2; 256 experts: 8200 slots 10.8 / 9.3, 32768 11.4 /
  // 13.1; 8 experts: 65536 slots 9.1 / 8.5, 131072 9.7 / 10.4)
  if (chunks > 64 || chunks * (experts + 1) > 4096)
    k_sort_scan<<<dim3((unsigned)((experts + 4) / 4)), 256, 0, st>>>(hist, experts, chunks, totals);
  else
    totals = nullptr;
  k_sort_place<<<chunks, 64 * kSortWavesMany, lds, st>>>(ids, slots, experts, chunks, hist, totals,
                                                         offsets, pos, src);
  return hipGetLastError();
}

template <typename T>
static void dispatch_t(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const int32_t* pos,
                       int topk, void* rows, int64_t ldr, hipStream_t st) {
  const dim3 b = exchange_block(cols, Elem<T>::kPer);
  in_launches(tokens, b.y, [&](int64_t t, int64_t n) {
    k_dispatch<T><<<dim3((unsigned)((n + b.y - 1) / b.y)), b, 0, st>>>(
        static_cast<const T*>(x) + t * ldx, n, cols, ldx, pos + t * topk, topk,
        static_cast<T*>(rows), ldr, tokens * topk);
  });
}

hipError_t launch_moe_dispatch(const void* x, bool bf16, int64_t tokens, int64_t cols, int64_t ldx,
                               const int32_t* pos, int topk, void* rows, int64_t ldr,
                               hipStream_t st) {
  if (tokens == 0) return hipSuccess;
  if (bf16)
    dispatch_t<uint16_t>(x, tokens, cols, ldx, pos, topk, rows, ldr, st);
  else
    dispatch_t<float>(x, tokens, cols, ldx, pos, topk, rows, ldr, st);
  return hipGetLastError();
}

template <typename T>
static void combine_t(const void* rows, int64_t tokens, int64_t cols, int64_t ldr,
                      const int32_t* pos, const float* weights, int topk, void* y, int64_t ldy,
                      hipStream_t st) {
  const dim3 b = exchange_block(cols, Elem<T>::kPer);
  in_launches(tokens, b.y, [&](int64_t t, int64_t n) {
    const dim3 g((unsigned)((n + b.y - 1) / b.y));
    const T* r = static_cast<const T*>(rows);
    T* out = static_cast<T*>(y) + t * ldy;
    if (weights)
      k_combine<T, true><<<g, b, 0, st>>>(r, n, cols, ldr, pos + t * topk, weights + t * topk, topk,
                                          out, ldy, tokens * topk);
    else
      k_combine<T, false><<<g, b, 0, st>>>(r, n, cols, ldr, pos + t * topk, nullptr, topk, out, ldy,
                                           tokens * topk);
  });
}

hipError_t launch_moe_combine(const void* rows, bool bf16, int64_t tokens, int64_t cols,
                              int64_t ldr, const int32_t* pos, const float* weights, int topk,
                              void* y, int64_t ldy, hipStream_t st) {
  if (tokens == 0) return hipSuccess;
  if (bf16)
    combine_t<uint16_t>(rows, tokens, cols, ldr, pos, weights, topk, y, ldy, st);
  else
    combine_t<float>(rows, tokens, cols, ldr, pos, weights, topk, y, ldy, st);
  return hipGetLastError();
}

template <typename T>
static void combine_grad_t(const void* dy, int64_t tokens, int64_t cols, int64_t ldy,
                           const void* rows, int64_t ldr, const int32_t* pos, const float* weights,
                           int topk, void* drows, int64_t lddr, float* dweights, hipStream_t st) {
  // whole tokens a launch: as many as have four slots for each workgroup (topk <= 32)
  const int64_t most = (int64_t)((1 << 24) - 1) * 4 / topk;
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t here = (tokens - t < most ? tokens - t : most) * topk;
    k_combine_grad<T><<<dim3((unsigned)((here + 3) / 4)), 256, 0, st>>>(
        static_cast<const T*>(dy) + t * ldy, here, cols, ldy, static_cast<const T*>(rows), ldr,
        pos + t * topk, weights + t * topk, topk, static_cast<T*>(drows), lddr, dweights + t * topk,
        tokens * topk);
  }
}

hipError_t launch_moe_combine_grad(const void* dy, bool bf16, int64_t tokens, int64_t cols,
                                   int64_t ldy, const void* rows, int64_t ldr, const int32_t* pos,
                                   const float* weights, int topk, void* drows, int64_t lddr,
                                   float* dweights, hipStream_t st) {
  if (tokens == 0) return hipSuccess;
  if (bf16)
    combine_grad_t<uint16_t>(dy, tokens, cols, ldy, rows, ldr, pos, weights, topk, drows, lddr,
                             dweights, st);
  else
    combine_grad_t<float>(dy, tokens, cols, ldy, rows, ldr, pos, weights, topk, drows, lddr,
                          dweights, st);
  return hipGetLastError();
}

}  // namespace averis
