// The global norm over a list of gradients and the clipped gradients.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   coef = min(1, max_norm / (norm + eps)) (1 for 0 / 0),  out = g coef
//
// Both passes walk the same 32 KiB chunks of the listed tensors.  A launch
// takes a table of up to kClipTensors tensors by value (nothing is copied to
// the device first); a workgroup finds its next chunk's tensor from its last
// one's.  The first pass leaves one fp64 partial per workgroup.  Up to
// kClipTensors tensors (one launch a pass, at most 16 KB of partials) every
// workgroup of the second pass sums them all itself, and there is no launch
// between the two; past that one workgroup does it once, since partials and
// workgroups both grow with the launches (graph replay, all summed by each /
// once: 2 launches of 256 tensors of 100 24.8 / 25.2 us, 2000 tensors of 256 KB
// 601 / 431 us, 12000 of 512 KB 21.3 / 4.0 ms).  The order is the same and
// fixed: no atomic, and the same bits on every call.
// Squares and sums are fp64: exact squares, and no overflow for any finite
// gradient.
//
// Both are bound by memory: the first reads every gradient, with the next
// chunk's loads in flight while a chunk is squared; the second reads and writes
// them, last chunk first, so that what the first pass read last may still be in
// a cache.  1 GiB of fp32 in 310 tensors: 0.22 ms (4.9 TB/s; without a second
// pass between, 0.19) and 0.41 ms (5.3 TB/s); 7 bf16 tensors of 31 MB together:
// 9 and 16 us.
// Up to 2048 workgroups a launch: eight on a CU keep enough loads in flight.
#include <hip/hip_runtime.h>
#include <alloca.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_common.hpp"
#include "launch.hpp"

namespace averis {
namespace {

constexpr int kClipTensors = 128;          // tensors of one launch
constexpr int64_t kClipBytes = 32768;      // bytes of a chunk
constexpr int kClipThreads = 256;
constexpr int kClipPieces = (int)(kClipBytes / 16 / kClipThreads);   // 16-byte pieces a thread takes
constexpr int kClipBlocks = 2048;          // workgroups (and partials) of one launch, at most

struct ClipTable {
  const void* g[kClipTensors];
  void* out[kClipTensors];
  int64_t n[kClipTensors];
  uint32_t first[kClipTensors + 1];        // a tensor's first chunk; [count]: all chunks
  uint8_t bf16[kClipTensors];
  int count;
};
static_assert(sizeof(ClipTable) + 64 <= 4096, "passed by value");

// 16 bytes at element alignment
typedef u32x4_t piece_t __attribute__((aligned(2)));

// tensor of chunk c, `from` the tensor of some chunk before it (after it, with
// DOWN)
template <bool DOWN>
__device__ __forceinline__ int tensor_of(const ClipTable& t, uint32_t c, int from) {
  // mostly the same tensor or a neighbour; else by bisection
  if (DOWN ? t.first[from] <= c : c < t.first[from + 1]) return from;
  int lo = DOWN ? 0 : from + 1, hi = DOWN ? from - 1 : t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// a chunk: its bytes
struct Chunk {
  const char* g;
  char* out;
  int bytes;
  bool bf16;
};
__device__ __forceinline__ Chunk chunk_of(const ClipTable& t, uint32_t c, int i) {
  Chunk k;
  k.bf16 = t.bf16[i] != 0;
  const int64_t at = (int64_t)(c - t.first[i]) * kClipBytes;
  const int64_t left = t.n[i] * (k.bf16 ? 2 : 4) - at;
  k.g = static_cast<const char*>(t.g[i]) + at;
  k.out = static_cast<char*>(t.out[i]) + at;
  k.bytes = (int)(left < kClipBytes ? left : kClipBytes);
  return k;
}
// the thread's 16-byte pieces of a chunk, 0 past its end
__device__ __forceinline__ void load_chunk(const Chunk& k, u32x4_t* v) {
  if (k.bytes == kClipBytes) {
    const char* g = k.g + threadIdx.x * 16;
#pragma unroll
    for (int i = 0; i < kClipPieces; ++i)
      v[i] = *reinterpret_cast<const piece_t*>(g + i * (kClipThreads * 16));
    return;
  }
#pragma unroll
  for (int i = 0; i < kClipPieces; ++i) {
    const int at = (i * kClipThreads + (int)threadIdx.x) * 16;
    v[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (at + 16 <= k.bytes) {
      v[i] = *reinterpret_cast<const piece_t*>(k.g + at);
    } else if (at < k.bytes) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + 2 * j < k.bytes)
          v[i][j / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(k.g + at + 2 * j) << (16 * (j & 1));
    }
  }
}

__device__ __forceinline__ void add_square(double& s, float v) {
  const double d = (double)v;
  s = __builtin_fma(d, d, s);
}

// sum over the workgroup (every thread gets it), in a fixed order
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  const double r = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  __syncthreads();
  return r;
}

__global__ __launch_bounds__(kClipThreads) void k_square_sums(ClipTable t, double* __restrict__ part) {
  __shared__ double sh[4];
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  uint32_t c = blockIdx.x;   // the grid has no more workgroups than chunks
  int i = tensor_of<false>(t, c, 0);
  Chunk k = chunk_of(t, c, i);
  u32x4_t v[kClipPieces];
  load_chunk(k, v);
  while (true) {
    const bool bf16 = k.bf16;
    c += gridDim.x;
    const bool more = c < t.first[t.count];
    u32x4_t w[kClipPieces];
    if (more) {
      i = tensor_of<false>(t, c, i);
      k = chunk_of(t, c, i);
      load_chunk(k, w);
    }
    if (bf16) {
#pragma unroll
      for (int p = 0; p < kClipPieces; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          add_square(s[j], bf16_lo(v[p][j]));
          add_square(s[j], bf16_hi(v[p][j]));
        }
    } else {
#pragma unroll
      for (int p = 0; p < kClipPieces; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) add_square(s[j], __uint_as_float(v[p][j]));
    }
    if (!more) break;
#pragma unroll
    for (int p = 0; p < kClipPieces; ++p) v[p] = w[p];
  }
  const double r = block_sum((s[0] + s[1]) + (s[2] + s[3]), sh);
  if (threadIdx.x == 0) part[blockIdx.x] = r;
}

__device__ __forceinline__ double norm_of(const double* part, int parts, double* sh) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  int i = threadIdx.x;
  for (; i + 3 * kClipThreads < parts; i += 4 * kClipThreads) {
#pragma unroll
    for (int u = 0; u < 4; ++u) s[u] += part[i + u * kClipThreads];
  }
#pragma unroll
  for (int u = 0; u < 3; ++u)
    if (i + u * kClipThreads < parts) s[u] += part[i + u * kClipThreads];
  return sqrt(block_sum((s[0] + s[1]) + (s[2] + s[3]), sh));
}

// whole (optional): the norm before its rounding
__global__ __launch_bounds__(kClipThreads) void k_norm(const double* __restrict__ part, int parts,
                                                       float* __restrict__ norm,
                                                       double* __restrict__ whole) {
  __shared__ double sh[4];
  const double r = norm_of(part, parts, sh);
  if (threadIdx.x == 0) {
    *norm = (float)r;
    if (whole) *whole = r;
  }
}

// times pre coef
__device__ __forceinline__ u32x4_t scaled(u32x4_t v, bool bf16, float pre, float coef) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = bf16 ? bf16x2_rne(bf16_lo(v[j]) * pre * coef, bf16_hi(v[j]) * pre * coef)
                : __float_as_uint(__uint_as_float(v[j]) * pre * coef);
  return v;
}

// parts 0: part holds the norm itself
__global__ __launch_bounds__(kClipThreads) void k_clip(ClipTable t, const double* __restrict__ part,
                                                       int parts, double max_norm, double eps,
                                                       float* __restrict__ norm) {
  __shared__ double sh[4];
  // the first chunk is on its way while the partials are summed
  int64_t c = (int64_t)t.first[t.count] - 1 - blockIdx.x;
  int i = tensor_of<true>(t, (uint32_t)c, t.count - 1);
  Chunk k = chunk_of(t, (uint32_t)c, i);
  u32x4_t v[kClipPieces];
  load_chunk(k, v);
  const double r = parts > 0 ? norm_of(part, parts, sh) : *part;
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)r;
  // (a norm of 0 without eps leaves zeros as they are)
  const double c64 = r + eps == 0.0 ? 1.0 : max_norm / (r + eps);
  // A factor that is no normal fp32 number would lose bits (a norm past 2^126
  // max_norm: finite gradients reach 2^148): a power of two, which is exact on
  // every value that does not end below fp32's range, takes 2^-64 of it.
  const float pre = c64 < 0x1p-64 ? 0x1p-64f : 1.0f;
  const float coef = c64 > 1.0 ? 1.0f : (float)(c64 < 0x1p-64 ? c64 * 0x1p64 : c64);   // NaN stays NaN
  while (true) {
    if (coef != 1.0f || k.g != k.out) {   // else in place and unchanged
#pragma unroll
      for (int p = 0; p < kClipPieces; ++p) v[p] = scaled(v[p], k.bf16, pre, coef);
      if (k.bytes == kClipBytes) {
        char* o = k.out + threadIdx.x * 16;
#pragma unroll
        for (int p = 0; p < kClipPieces; ++p)
          *reinterpret_cast<piece_t*>(o + p * (kClipThreads * 16)) = v[p];
      } else {
#pragma unroll
        for (int p = 0; p < kClipPieces; ++p) {
          const int at = (p * kClipThreads + (int)threadIdx.x) * 16;
          if (at + 16 <= k.bytes) {
            *reinterpret_cast<piece_t*>(k.out + at) = v[p];
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (at + 2 * j < k.bytes)
                *reinterpret_cast<uint16_t*>(k.out + at + 2 * j) = (uint16_t)(v[p][j / 2] >> (16 * (j & 1)));
          }
        }
      }
    }
    c -= gridDim.x;
    if (c < 0) break;
    i = tensor_of<true>(t, (uint32_t)c, i);
    k = chunk_of(t, (uint32_t)c, i);
    if (coef != 1.0f || k.g != k.out) load_chunk(k, v);
  }
}

// the tensors of one launch, from w[i0]; empty ones are left out
int fill_table(const GradTensor* w, int n, int i0, ClipTable& t) {
  t.count = 0;
  t.first[0] = 0;
  int i = i0;
  for (; i < n && t.count < kClipTensors; ++i) {
    if (w[i].n == 0) continue;
    const int64_t per = kClipBytes >> (w[i].bf16 ? 1 : 2);
    const int64_t chunks = (w[i].n + per - 1) / per;
    // the prefix counts are 32 bits wide: 2^32 chunks are 128 TiB
    t.g[t.count] = w[i].g;
    t.out[t.count] = w[i].out;
    t.n[t.count] = w[i].n;
    t.bf16[t.count] = w[i].bf16;
    t.first[t.count + 1] = t.first[t.count] + (uint32_t)chunks;
    ++t.count;
  }
  return i;
}

inline unsigned clip_grid(const ClipTable& t) {
  const uint32_t c = t.first[t.count];
  return c < (uint32_t)kClipBlocks ? c : (unsigned)kClipBlocks;
}

}  // namespace

size_t grad_norm_ws_bytes(int n) {
  const size_t launches = ((size_t)n + kClipTensors - 1) / kClipTensors;
  return ((launches ? launches : 1) * kClipBlocks + 1) * sizeof(double);   // partials, the norm
}

hipError_t launch_grad_clip(int n, const GradTensor* w, bool scale, double max_norm, double eps,
                            float* norm, void* ws, hipStream_t st) {
  double* part = static_cast<double*>(ws);
  int parts = 0, launches = 0;
  int* begin = static_cast<int*>(alloca(((size_t)n / kClipTensors + 1) * sizeof(int)));
  ClipTable t;
  for (int i = 0; i < n;) {
    const int from = i;
    i = fill_table(w, n, i, t);
    if (t.count == 0) break;
    begin[launches++] = from;
    const unsigned g = clip_grid(t);
    k_square_sums<<<g, kClipThreads, 0, st>>>(t, part + parts);
    parts += (int)g;
  }
  double* whole = launches > 1 ? part + parts : nullptr;
  if (!scale || parts == 0 || whole) {
    k_norm<<<1, kClipThreads, 0, st>>>(part, parts, norm, whole);
    if (!scale || parts == 0) return hipGetLastError();
    if (whole) {
      part = whole;
      parts = 0;
      norm = nullptr;
    }
  }
  // the last launch's tensors first: what was read last
  for (int l = launches - 1; l >= 0; --l) {
    fill_table(w, n, begin[l], t);
    k_clip<<<clip_grid(t), kClipThreads, 0, st>>>(t, part, parts, max_norm, eps, norm);
    norm = nullptr;   // written once
  }
  return hipGetLastError();
}

}  // namespace averis
