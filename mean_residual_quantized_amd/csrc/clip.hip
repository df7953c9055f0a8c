// The global norm over a list of gradients and the clipped gradients.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   coef = min(1, max_norm / (norm + eps)),  out = g coef
//
// Both passes walk the same 32 KiB chunks of the listed tensors.  A launch
// takes a table of up to kClipTensors tensors by value (nothing is copied to
// the device first); a workgroup finds its chunk's tensor by a binary search
// of the chunks' prefix counts.  The first pass leaves one fp64 partial per
// workgroup; every workgroup of the second sums all the partials itself, in
// the same fixed order, so there is no launch between the two, no atomic, and
// the same bits on every call.  Squares and sums are fp64: exact squares, and
// no overflow for any finite gradient.
#include <hip/hip_runtime.h>
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
constexpr int kClipBlocks = 1024;          // workgroups (and partials) of one launch, at most

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

// tensor of chunk c
__device__ __forceinline__ int tensor_of(const ClipTable& t, uint32_t c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
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

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, int64_t n, double s) {
  constexpr int P = 16 / (int)sizeof(T);
  u32x4_t v[kClipPieces];
#pragma unroll
  for (int i = 0; i < kClipPieces; ++i) {
    const int64_t e = ((int64_t)i * kClipThreads + threadIdx.x) * P;
    v[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (e + P <= n) {
      v[i] = *reinterpret_cast<const piece_t*>(g + e);
    } else if (e < n) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (e + j < n) {
          if constexpr (sizeof(T) == 2) v[i][j / 2] |= (uint32_t)g[e + j] << (16 * (j & 1));
          else v[i][j] = __float_as_uint(g[e + j]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kClipPieces; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 2) {
        add_square(s, bf16_lo(v[i][j]));
        add_square(s, bf16_hi(v[i][j]));
      } else {
        add_square(s, __uint_as_float(v[i][j]));
      }
    }
  }
  return s;
}

__global__ __launch_bounds__(kClipThreads) void k_square_sums(ClipTable t, double* __restrict__ part) {
  __shared__ double sh[4];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t per = kClipBytes >> (t.bf16[i] ? 1 : 2);
    const int64_t e0 = (int64_t)(c - t.first[i]) * per;
    const int64_t n = t.n[i] - e0 < per ? t.n[i] - e0 : per;
    if (t.bf16[i])
      s = chunk_squares(static_cast<const uint16_t*>(t.g[i]) + e0, n, s);
    else
      s = chunk_squares(static_cast<const float*>(t.g[i]) + e0, n, s);
  }
  s = block_sum(s, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double norm_of(const double* part, int parts, double* sh) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) s += part[i];
  return sqrt(block_sum(s, sh));
}

__global__ __launch_bounds__(kClipThreads) void k_norm(const double* __restrict__ part, int parts,
                                                       float* __restrict__ norm) {
  __shared__ double sh[4];
  const double r = norm_of(part, parts, sh);
  if (threadIdx.x == 0) *norm = (float)r;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* g, T* out, int64_t n, float coef) {
  constexpr int P = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < kClipPieces; ++i) {
    const int64_t e = ((int64_t)i * kClipThreads + threadIdx.x) * P;
    if (e + P <= n) {
      u32x4_t v = *reinterpret_cast<const piece_t*>(g + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2)
          v[j] = bf16x2_rne(bf16_lo(v[j]) * coef, bf16_hi(v[j]) * coef);
        else
          v[j] = __float_as_uint(__uint_as_float(v[j]) * coef);
      }
      *reinterpret_cast<piece_t*>(out + e) = v;
    } else {
      for (int j = 0; j < P && e + j < n; ++j) {
        if constexpr (sizeof(T) == 2)
          out[e + j] = (uint16_t)bf16x2_rne(bf16_lo(g[e + j]) * coef, 0.0f);
        else
          out[e + j] = g[e + j] * coef;
      }
    }
  }
}

__global__ __launch_bounds__(kClipThreads) void k_clip(ClipTable t, const double* __restrict__ part,
                                                       int parts, double max_norm, double eps,
                                                       float* __restrict__ norm) {
  __shared__ double sh[4];
  const double r = norm_of(part, parts, sh);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)r;
  const double c64 = max_norm / (r + eps);
  const float coef = c64 > 1.0 ? 1.0f : (float)c64;   // NaN stays NaN
  for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int i = tensor_of(t, c);
    if (coef == 1.0f && t.g[i] == t.out[i]) continue;   // in place and unchanged
    const int64_t per = kClipBytes >> (t.bf16[i] ? 1 : 2);
    const int64_t e0 = (int64_t)(c - t.first[i]) * per;
    const int64_t n = t.n[i] - e0 < per ? t.n[i] - e0 : per;
    if (t.bf16[i])
      chunk_scale(static_cast<const uint16_t*>(t.g[i]) + e0, static_cast<uint16_t*>(t.out[i]) + e0, n, coef);
    else
      chunk_scale(static_cast<const float*>(t.g[i]) + e0, static_cast<float*>(t.out[i]) + e0, n, coef);
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
  return (launches ? launches : 1) * kClipBlocks * sizeof(double);
}

hipError_t launch_grad_clip(int n, const GradTensor* w, bool scale, double max_norm, double eps,
                            float* norm, void* ws, hipStream_t st) {
  double* part = static_cast<double*>(ws);
  int parts = 0;
  ClipTable t;
  for (int i = 0; i < n;) {
    i = fill_table(w, n, i, t);
    if (t.count == 0) break;
    const unsigned g = clip_grid(t);
    k_square_sums<<<g, kClipThreads, 0, st>>>(t, part + parts);
    parts += (int)g;
  }
  if (!scale || parts == 0) {
    k_norm<<<1, kClipThreads, 0, st>>>(part, parts, norm);
    return hipGetLastError();
  }
  for (int i = 0; i < n;) {
    i = fill_table(w, n, i, t);
    if (t.count == 0) break;
    k_clip<<<clip_grid(t), kClipThreads, 0, st>>>(t, part, parts, max_norm, eps, norm);
    norm = nullptr;   // written once
  }
  return hipGetLastError();
}

}  // namespace averis
