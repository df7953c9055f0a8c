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
  u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (c + i < cols) {
      if constexpr (sizeof(T) == 2)
        v[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
      else
        v[i] = __float_as_uint(row[c + i]);
    }
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
// Router.  G lanes share a token, each with V consecutive logits.
// ---------------------------------------------------------------------------
constexpr float kMasked = -__builtin_inff();

template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int e0, int experts, float* l) {
  constexpr int P = Elem<T>::kPer;
  if constexpr (V % P == 0) {
    if (e0 + V <= experts) {
#pragma unroll
      for (int v = 0; v < V; v += P)
        Elem<T>::unpack(*reinterpret_cast<const piece_t*>(row + e0 + v), l + v);
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = e0 + v < experts ? Elem<T>::f32(row[e0 + v]) : kMasked;
}

// Top-k by k rounds of a group maximum.  A logit's key orders as its value
// (NaN above +inf, -0 equal to +0); 0 stands for masked, absent and taken.
// A round is a maximum of keys over the lane's V and the group, then the
// smallest index that has it: ties go to the lowest expert.
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void k_route(const T* __restrict__ logits, int64_t tokens,
                                               int experts, int64_t ld, int topk, int renorm,
                                               int32_t* __restrict__ ids,
                                               float* __restrict__ weights) {
  constexpr int KO = kMaxTopk > G ? kMaxTopk / G : 1;
  const int g = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const bool live = t < tokens;   // the others repeat the last token, unstored
  const T* row = logits + (live ? t : tokens - 1) * ld;
  float l[V];
  load_logits<T, V>(row, g * V, experts, l);
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    key[v] = f32_ordered(l[v] + 0.0f);
    if (l[v] != l[v]) key[v] = 0xFFFFFFFFu;
    if (l[v] == kMasked) key[v] = 0u;
  }
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
      uint32_t at = 0xFFFFu;
#pragma unroll
      for (int v = V - 1; v >= 0; --v) at = key[v] == best ? (uint32_t)(g * V + v) : at;
      at = group_min<G>(at);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = at == (uint32_t)(g * V + v) ? 0u : key[v];
      const float x = f32_from_ordered(best);
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
      weights[t * topk + j] = val[o] / total;
    }
  }
}

// w = softmax over the chosen (renorm) or all logits.  With s_e = dweights of
// the slot that chose e (0 if none) and m = sum over the chosen of w s:
// dl_e = w_e (s_e - m), zero outside the chosen when renorm.
template <typename T, int G, int V>
__global__ __launch_bounds__(256) void k_route_grad(const T* logits, int64_t tokens,
                                                    int experts, int64_t ld, int topk, int renorm,
                                                    const int32_t* __restrict__ ids,
                                                    const float* __restrict__ dweights,
                                                    T* dlogits, int64_t ldd) {
  const int g = threadIdx.x % G;
  const int64_t t = (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G;
  const bool live = t < tokens;
  const int64_t tr = live ? t : tokens - 1;
  float l[V], s[V];
  load_logits<T, V>(logits + tr * ld, g * V, experts, l);
  uint32_t chosen = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = 0.0f;
  for (int j = 0; j < topk; ++j) {
    const int e = ids[tr * topk + j] - g * V;
    const float d = dweights[tr * topk + j];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (e == v) {
        s[v] = d;
        chosen |= 1u << v;
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
  mean = mean / total;
  if (!live) return;
  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool in = (chosen >> v) & 1u;
    d[v] = (in || !renorm) ? l[v] / total * (s[v] - mean) : 0.0f;
  }
  T* out = dlogits + t * ldd;
  constexpr int P = Elem<T>::kPer;
  const int e0 = g * V;
  if constexpr (V % P == 0) {
    if (e0 + V <= experts) {
#pragma unroll
      for (int v = 0; v < V; v += P)
        *reinterpret_cast<piece_t*>(out + e0 + v) = Elem<T>::pack(d + v);
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (e0 + v < experts) out[e0 + v] = Elem<T>::from(d[v]);
}

// ---------------------------------------------------------------------------
// Stable counting sort of the slots by expert.  A slot without a valid expert
// goes to bucket `experts`, the tail.  Each wavefront owns a run of slots:
// its counts per bucket are turned into its first rows per bucket (buckets,
// then wavefronts, in order), then it ranks its slots 64 at a time by ballots
// over the bucket's bits.  No step depends on the order of atomics.
// ---------------------------------------------------------------------------
constexpr int kSortSteps = 8;   // 64-slot steps of a wavefront

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
template <int WAVES>
__device__ __forceinline__ void sort_count(const int32_t* ids, int64_t first, int64_t n,
                                           int experts, int* cnt, int* b) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nb = experts + 1;
  const int64_t s0 = first + (int64_t)w * (64 * kSortSteps);
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i) {
    const int64_t s = s0 + 64 * i + lane;
    b[i] = s < n ? bucket_of(ids[s], experts) : -1;
  }
  for (int i = threadIdx.x; i < WAVES * nb; i += 64 * WAVES) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i)
    if (b[i] >= 0) atomicAdd(&cnt[w * nb + b[i]], 1);
  __syncthreads();
}

// rows of the wavefront's slots from its first rows in cnt[wave][bucket]
__device__ __forceinline__ void sort_place(int64_t first, int64_t n, int experts, int* cnt,
                                           const int* b, int32_t* pos, int32_t* src) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, nb = experts + 1;
  const int64_t s0 = first + (int64_t)w * (64 * kSortSteps);
  const uint64_t below = (1ull << lane) - 1ull;
  const int bits = 32 - __builtin_clz(experts);   // buckets 0 .. experts
  volatile int* row0 = cnt + w * nb;
#pragma unroll
  for (int i = 0; i < kSortSteps; ++i) {
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

constexpr int kSortWavesOne = 16;    // one workgroup for everything
constexpr int kSortWavesMany = 4;    // workgroups of a larger sort
constexpr int64_t kSortOne = (int64_t)kSortWavesOne * 64 * kSortSteps;     // 8192 slots
constexpr int64_t kSortChunk = (int64_t)kSortWavesMany * 64 * kSortSteps;  // 2048 slots

__global__ __launch_bounds__(64 * kSortWavesOne) void k_sort_one(
    const int32_t* __restrict__ ids, int n, int experts, int64_t* __restrict__ offsets,
    int32_t* __restrict__ pos, int32_t* __restrict__ src) {
  extern __shared__ int cnt[];   // [waves][experts + 1]
  __shared__ int sh[kSortWavesOne];
  int b[kSortSteps];
  const int nb = experts + 1;
  sort_count<kSortWavesOne>(ids, 0, n, experts, cnt, b);
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
  sort_place(0, n, experts, cnt, b, pos, src);
}

// counts of a chunk -> hist[bucket][chunk]
__global__ __launch_bounds__(64 * kSortWavesMany) void k_sort_hist(
    const int32_t* __restrict__ ids, int64_t n, int experts, int chunks, int* __restrict__ hist) {
  extern __shared__ int cnt[];
  int b[kSortSteps];
  sort_count<kSortWavesMany>(ids, (int64_t)blockIdx.x * kSortChunk, n, experts, cnt, b);
  const int nb = experts + 1;
  for (int e = threadIdx.x; e < nb; e += 64 * kSortWavesMany) {
    int c = 0;
    for (int w = 0; w < kSortWavesMany; ++w) c += cnt[w * nb + e];
    hist[(int64_t)e * chunks + blockIdx.x] = c;
  }
}

// exclusive prefix sum of hist, bucket by bucket, in place; a bucket's first
// value is its offset.  One workgroup, each thread a contiguous run.
__global__ __launch_bounds__(1024) void k_sort_scan(int* __restrict__ hist, int experts, int chunks,
                                                    int64_t* __restrict__ offsets) {
  __shared__ int sh[16];
  const int64_t len = (int64_t)(experts + 1) * chunks;
  const int64_t per = (len + 1023) / 1024;
  const int64_t i0 = per * threadIdx.x, i1 = i0 + per < len ? i0 + per : len;
  int sum = 0;
  for (int64_t i = i0; i < i1; ++i) sum += hist[i];
  int total;
  int run = block_exclusive<16>(sum, sh, total);
  if (i0 >= i1) return;
  int64_t next = (i0 + chunks - 1) / chunks * chunks;   // the next bucket's first place
  for (int64_t i = i0; i < i1; ++i) {
    const int c = hist[i];
    hist[i] = run;
    if (i == next) {
      offsets[i / chunks] = run;
      next += chunks;
    }
    run += c;
  }
}

__global__ __launch_bounds__(64 * kSortWavesMany) void k_sort_place(
    const int32_t* __restrict__ ids, int64_t n, int experts, int chunks,
    const int* __restrict__ hist, int32_t* __restrict__ pos, int32_t* __restrict__ src) {
  extern __shared__ int cnt[];
  int b[kSortSteps];
  const int64_t first = (int64_t)blockIdx.x * kSortChunk;
  sort_count<kSortWavesMany>(ids, first, n, experts, cnt, b);
  const int nb = experts + 1;
  for (int e = threadIdx.x; e < nb; e += 64 * kSortWavesMany) {
    int run = hist[(int64_t)e * chunks + blockIdx.x];
    for (int w = 0; w < kSortWavesMany; ++w) {
      const int c = cnt[w * nb + e];
      cnt[w * nb + e] = run;
      run += c;
    }
  }
  __syncthreads();
  sort_place(first, n, experts, cnt, b, pos, src);
}

__global__ void k_zero_offsets(int64_t* offsets, int count) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < count) offsets[i] = 0;
}

// ---------------------------------------------------------------------------
// Token exchange.  blockDim.x lanes (whole wavefronts) go along a token's
// columns in 16-byte pieces, blockDim.y tokens to a workgroup.  Rows outside
// the tokens * topk there are, which only malformed positions name, are
// neither read nor written.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// a token is read once and written to its k rows
template <typename T>
__global__ __launch_bounds__(256) void k_dispatch(const T* __restrict__ x, int64_t tokens,
                                                  int64_t cols, int64_t ldx,
                                                  const int32_t* __restrict__ pos, int topk,
                                                  T* __restrict__ rows, int64_t ldr) {
  constexpr int P = Elem<T>::kPer;
  const int64_t t = uniform64((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= tokens) return;
  const int32_t* pt = pos + t * topk;
  const int64_t slots = tokens * topk;
  for (int64_t c = (int64_t)threadIdx.x * P; c < cols; c += (int64_t)blockDim.x * P) {
    const u32x4_t v = load_piece(x + t * ldx, c, cols);
    for (int j = 0; j < topk; ++j) {
      const int p = pt[j];
      const int64_t r = p < 0 ? ~p : p;
      if (r < slots) store_piece(rows + r * ldr, c, cols, p < 0 ? u32x4_t{0u, 0u, 0u, 0u} : v);
    }
  }
}

// y_t = sum_j w_tj rows[pos_tj], slots in order, fp32; eight rows in flight
template <typename T, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_combine(const T* __restrict__ rows, int64_t tokens,
                                                 int64_t cols, int64_t ldr,
                                                 const int32_t* __restrict__ pos,
                                                 const float* __restrict__ weights, int topk,
                                                 T* __restrict__ y, int64_t ldy) {
  constexpr int P = Elem<T>::kPer, U = 8;
  const int64_t t = uniform64((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
  if (t >= tokens) return;
  const int64_t slots = tokens * topk;
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
// wavefront a slot, neighbouring slots share dy_t through the cache
template <typename T>
__global__ __launch_bounds__(256) void k_combine_grad(const T* __restrict__ dy, int64_t slots,
                                                      int64_t cols, int64_t ldy,
                                                      const T* rows, int64_t ldr,
                                                      const int32_t* __restrict__ pos,
                                                      const float* __restrict__ weights, int topk,
                                                      T* drows, int64_t lddr,
                                                      float* __restrict__ dweights) {
  constexpr int P = Elem<T>::kPer;
  const int lane = threadIdx.x & 63;
  const uint32_t s = __builtin_amdgcn_readfirstlane(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (s >= (uint64_t)slots) return;
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
// lanes per token and logits per lane by the number of experts
#define AVERIS_ROUTE_SHAPES(CALL)      \
  if (experts <= 8) {                  \
    CALL(8, 1);                        \
  } else if (experts <= 32) {          \
    CALL(8, 4);                        \
  } else if (experts <= 64) {          \
    CALL(8, 8);                        \
  } else if (experts <= 128) {         \
    CALL(16, 8);                       \
  } else if (experts <= 256) {         \
    CALL(32, 8);                       \
  } else if (experts <= 512) {         \
    CALL(64, 8);                       \
  } else {                             \
    CALL(64, 16);                      \
  }

template <typename T>
static void route_t(const T* l, int64_t tokens, int experts, int64_t ld, int topk, bool renorm,
                    int32_t* ids, float* w, hipStream_t st) {
#define AVERIS_ROUTE(G, V)                                                                      \
  k_route<T, G, V><<<dim3((unsigned)((tokens + 256 / G - 1) / (256 / G))), 256, 0, st>>>(        \
      l, tokens, experts, ld, topk, renorm, ids, w)
  AVERIS_ROUTE_SHAPES(AVERIS_ROUTE)
#undef AVERIS_ROUTE
}

template <typename T>
static void route_grad_t(const T* l, int64_t tokens, int experts, int64_t ld, int topk,
                         bool renorm, const int32_t* ids, const float* dw, T* dl, int64_t ldd,
                         hipStream_t st) {
#define AVERIS_ROUTE(G, V)                                                                      \
  k_route_grad<T, G, V><<<dim3((unsigned)((tokens + 256 / G - 1) / (256 / G))), 256, 0, st>>>(   \
      l, tokens, experts, ld, topk, renorm, ids, dw, dl, ldd)
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
  return ((size_t)sort_chunks(slots) * (size_t)(experts + 1) * 4 + 255) & ~(size_t)255;
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
  k_sort_scan<<<1, 1024, 0, st>>>(hist, experts, chunks, offsets);
  k_sort_place<<<chunks, 64 * kSortWavesMany, lds, st>>>(ids, slots, experts, chunks, hist, pos,
                                                         src);
  return hipGetLastError();
}

hipError_t launch_moe_dispatch(const void* x, bool bf16, int64_t tokens, int64_t cols, int64_t ldx,
                               const int32_t* pos, int topk, void* rows, int64_t ldr,
                               hipStream_t st) {
  if (tokens == 0) return hipSuccess;
  const dim3 b = exchange_block(cols, bf16 ? 8 : 4);
  const dim3 g((unsigned)((tokens + b.y - 1) / b.y));
  if (bf16)
    k_dispatch<uint16_t><<<g, b, 0, st>>>(static_cast<const uint16_t*>(x), tokens, cols, ldx, pos,
                                          topk, static_cast<uint16_t*>(rows), ldr);
  else
    k_dispatch<float><<<g, b, 0, st>>>(static_cast<const float*>(x), tokens, cols, ldx, pos, topk,
                                       static_cast<float*>(rows), ldr);
  return hipGetLastError();
}

template <typename T>
static void combine_t(const void* rows, int64_t tokens, int64_t cols, int64_t ldr,
                      const int32_t* pos, const float* weights, int topk, void* y, int64_t ldy,
                      hipStream_t st) {
  const dim3 b = exchange_block(cols, Elem<T>::kPer);
  const dim3 g((unsigned)((tokens + b.y - 1) / b.y));
  if (weights)
    k_combine<T, true><<<g, b, 0, st>>>(static_cast<const T*>(rows), tokens, cols, ldr, pos,
                                        weights, topk, static_cast<T*>(y), ldy);
  else
    k_combine<T, false><<<g, b, 0, st>>>(static_cast<const T*>(rows), tokens, cols, ldr, pos,
                                         nullptr, topk, static_cast<T*>(y), ldy);
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
  const int64_t slots = tokens * topk;
  k_combine_grad<T><<<dim3((unsigned)((slots + 3) / 4)), 256, 0, st>>>(
      static_cast<const T*>(dy), slots, cols, ldy, static_cast<const T*>(rows), ldr, pos, weights,
      topk, static_cast<T*>(drows), lddr, dweights);
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
