// Root-mean-square norm with the residual's addition, its output in block-scaled
// fp8 (fp8_common.hpp) and in its own type, and the gradient, for gfx950.
//
//   h = x + r, rounded to the type;  f = 1 / sqrt(mean_j h_j^2 + eps)
//   y_j = (h_j f) w_j, rounded to the type;  codes of y as k_fp8_rows gives them
//   c = mean_j (dy_j w_j)(h_j f)
//   dh_j = f (dy_j w_j - (h_j f) c) + dres_j;  dw_j = sum over the rows of dy_j h_j f
//
// The sum of squares is in fp64: a bf16 value's square is exact there and sums
// of them nearly always are, so f, y and every code come out the same whatever
// order a kernel adds in (the transposed copy is made by another one), and no
// sum overflows.  An fp64 addition costs what an fp32 one does.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8_eight.hpp"
#include "launch.hpp"
#include "segments.hpp"

namespace averis {
namespace {

template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// EIGHTS: rows of whole pieces (cols a multiple of 8), whose loads and stores
// need no code for a row's last elements (with it the gradient of 16384 x 1001
// takes 45 us, of 16384 x 1024 30)
template <bool EIGHTS, typename T>
__device__ __forceinline__ void load8(Eight<T>& v, const T* row, int64_t c, int64_t cols) {
  if constexpr (EIGHTS) {
    v.zero();
    if (c < cols) v.load(row + c, 0, 8);
  } else {
    v.load(row, c, cols);
  }
}
template <bool EIGHTS, typename T>
__device__ __forceinline__ void store8(const Eight<T>& v, T* row, int64_t c, int64_t cols) {
  if constexpr (EIGHTS) {
    if (c < cols) v.store(row + c, 0, 8);
  } else {
    v.store(row, c, cols);
  }
}
template <bool EIGHTS>
__device__ __forceinline__ void weight8(const void* w, bool bf16, int64_t c, int64_t cols, float* f) {
  if constexpr (EIGHTS) {
    if (bf16) {
      Eight<uint16_t> v;
      load8<true>(v, static_cast<const uint16_t*>(w), c, cols);
      v.f32(f);
    } else {
      Eight<float> v;
      load8<true>(v, static_cast<const float*>(w), c, cols);
      v.f32(f);
    }
  } else {
    load_vector(w, bf16, c, cols, f);
  }
}

// columns of the lane's piece i: 512 to a wavefront and step, so that sixteen
// lanes hold a block of 128
template <int W>
__device__ __forceinline__ int64_t piece_at(int lane, int g, int i) {
  return 512 * (int64_t)(g + W * i) + 8 * lane;
}

// W wavefronts hold a row, I pieces of eight elements a lane: the row is read
// once, into registers.  Bound by memory: 32768 x 2048 bf16 with a residual and
// codes 79 us (470 MB, 5.9 TB/s; a copy reaches 5.3), 2999 x 1000 fp32 8 us
// (latency), 16 x 2048 4.2 us.  The transposed copy is k_fp8_tile's, from h and f:
// 38 us more (201 MB): its runs go across 128 rows, more than a workgroup holds.
template <typename T, int W, int I, bool EIGHTS>
__global__ __launch_bounds__(W > 4 ? 64 * W : 256) void k_norm(NormArgs a, int64_t row0, int64_t rows,
                                                               int64_t cols, double inv_cols, Fp8Out out) {
  constexpr int PER = W > 4 ? 1 : 4 / W;   // rows a workgroup
  __shared__ double part[PER][W];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = w % W, mine = w / W;
  const int64_t r = row0 + (int64_t)blockIdx.x * PER + mine;
  const bool live = r < rows;   // the others repeat the last row, unstored
  const int64_t row = live ? r : rows - 1;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  Eight<T> h[I];
#pragma unroll
  for (int i = 0; i < I; ++i) load8<EIGHTS>(h[i], x, piece_at<W>(lane, g, i), cols);
  if (a.res) {
    const T* res = static_cast<const T*>(a.res) + row * a.ldres;
    Eight<T> v[I];
#pragma unroll
    for (int i = 0; i < I; ++i) load8<EIGHTS>(v[i], res, piece_at<W>(lane, g, i), cols);
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float f[8], e[8];
      h[i].f32(f);
      v[i].f32(e);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] += e[q];
      h[i].set(f);
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < I; ++i)
        store8<EIGHTS>(h[i], static_cast<T*>(a.h) + row * a.ldh, piece_at<W>(lane, g, i), cols);
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    float f[8];
    h[i].f32(f);
#pragma unroll
    for (int q = 0; q < 8; ++q) sum = __builtin_fma((double)f[q], (double)f[q], sum);
  }
  sum = wave_sum(sum);
  if constexpr (W > 1) {
    if (lane == 0) part[mine][g] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int q = 0; q < W; ++q) sum += part[mine][q];
  }
  const float f = (float)rsqrt(sum * inv_cols + a.eps);
  if (!live) return;
  if (g == 0 && lane == 0) a.rstd[row] = f;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int64_t c = piece_at<W>(lane, g, i);
    if (c - 8 * lane >= cols) break;
    float v[8], wt[8];
    h[i].f32(v);
    weight8<EIGHTS>(a.weight, a.wbf16, c, cols, wt);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = v[q] * f * wt[q];
    Eight<T> y;
    y.set(v);
    if (a.y) store8<EIGHTS>(y, static_cast<T*>(a.y) + row * a.ldy, c, cols);
    if (out.codes) {
      uint32_t byte;
      u32x2_t q = eight_codes(y, row16_max(y.amax()), byte);
      if (c - 8 * lane + 512 > cols) q = without_pad(q, c, cols);
      const uint32_t word = __builtin_amdgcn_readlane(byte, 0) | __builtin_amdgcn_readlane(byte, 16) << 8 |
                            __builtin_amdgcn_readlane(byte, 32) << 16 |
                            __builtin_amdgcn_readlane(byte, 48) << 24;
      if (c < out.pitch) *reinterpret_cast<u32x2_t*>(out.codes + row * out.pitch + c) = q;
      if (lane == 0) *reinterpret_cast<uint32_t*>(out.scales + row * out.spitch + 4 * (g + W * i)) = word;
    }
  }
}

// Workgroup b takes rows b PER + .., each gridDim.x PER further on, and adds up
// the weight's gradient of them in registers: part[b][cols].  Bound by memory:
// 32768 x 2048 bf16 107 us (537 MB and 8 MB of partial sums, 5.1 TB/s).
template <typename T, int W, int I, bool EIGHTS>
__global__ __launch_bounds__(W > 4 ? 64 * W : 256) void k_norm_grad(NormGradArgs a, int64_t rows,
                                                                    int64_t cols, float inv_cols,
                                                                    float* __restrict__ part) {
  constexpr int PER = W > 4 ? 1 : 4 / W;
  __shared__ float dot[2][PER][W];
  extern __shared__ float dwl[];   // [PER][cols], where PER > 1
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = w % W, mine = w / W;
  float wt[I][8], dw[I][8];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    weight8<EIGHTS>(a.weight, a.wbf16, piece_at<W>(lane, g, i), cols, wt[i]);
#pragma unroll
    for (int q = 0; q < 8; ++q) dw[i][q] = 0.0f;
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * PER; r0 < rows; r0 += (int64_t)gridDim.x * PER, turn ^= 1) {
    const int64_t row = r0 + mine;
    const bool live = row < rows;
    const int64_t at = live ? row : rows - 1;
    Eight<T> dy[I], h[I], res[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      load8<EIGHTS>(dy[i], static_cast<const T*>(a.dy) + at * a.lddy, piece_at<W>(lane, g, i), cols);
      load8<EIGHTS>(h[i], static_cast<const T*>(a.h) + at * a.ldh, piece_at<W>(lane, g, i), cols);
    }
    if (a.dres) {
#pragma unroll
      for (int i = 0; i < I; ++i)
        load8<EIGHTS>(res[i], static_cast<const T*>(a.dres) + at * a.lddres, piece_at<W>(lane, g, i), cols);
    }
    const float f = a.rstd[at];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float d[8], v[8];
      dy[i].f32(d);
      h[i].f32(v);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float xh = v[q] * f;
        c = __builtin_fmaf(d[q] * wt[i][q], xh, c);
        if (live) dw[i][q] = __builtin_fmaf(d[q], xh, dw[i][q]);
      }
    }
    c = wave_sum(c);
    if constexpr (W > 1) {
      // two places in turn: a barrier a row
      if (lane == 0) dot[turn][mine][g] = c;
      __syncthreads();
      c = 0.0f;
#pragma unroll
      for (int q = 0; q < W; ++q) c += dot[turn][mine][q];
    }
    c *= inv_cols;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float d[8], v[8], e[8];
      dy[i].f32(d);
      h[i].f32(v);
      if (a.dres) res[i].f32(e);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        d[q] = f * (d[q] * wt[i][q] - v[q] * f * c);
        if (a.dres) d[q] += e[q];
      }
      Eight<T> o;
      o.set(d);
      store8<EIGHTS>(o, static_cast<T*>(a.dh) + at * a.lddh, piece_at<W>(lane, g, i), cols);
    }
  }
  if (!part) return;
  float* dst = part + (int64_t)blockIdx.x * cols;
  if constexpr (PER == 1) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t c = piece_at<W>(lane, g, i);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < cols) dst[c + q] = dw[i][q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int64_t c = piece_at<W>(lane, g, i);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < cols) dwl[mine * cols + c + q] = dw[i][q];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += 256) {
      float s = dwl[c];
#pragma unroll
      for (int m = 1; m < PER; ++m) s += dwl[m * cols + c];
      dst[c] = s;
    }
  }
}

// 64 columns and kSumSegs segments a workgroup of 16 wavefronts.  A segment's chunks are
// divided in order into sixteen parts, and the parts' sums added in order: by all
// wavefronts, one such segment after the other, or by one of them where no part has
// more than one chunk.  Bound by latency: 1024 x 2048 6.5 us, chunks of 768 columns in 64
// segments 4.8, in 512 7.0 (a segment a workgroup, each looking for its own from the
// first on, 5.1 and 47; sixteen 5.7 and 5.9).
constexpr int kSumWaves = 16, kSumSegs = 8;

__global__ __launch_bounds__(64 * kSumWaves) void k_column_sums(const float* __restrict__ part,
                                                                int64_t rows, int64_t ch, int64_t cols,
                                                                const int64_t* offs, int nseg,
                                                                int64_t chunks,
                                                                float* __restrict__ out) {
  __shared__ float sh[kSumWaves][64];
  __shared__ int64_t before[kSumWaves], first[kSumSegs + 1];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int seg0 = blockIdx.y * kSumSegs, segs = nseg - seg0 < kSumSegs ? nseg - seg0 : kSumSegs;
  auto count = [&](int s) {
    int64_t a, e;
    seg_bounds(offs, s, rows, a, e);
    return (e - a + ch - 1) / ch;
  };
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  // by all wavefronts
  auto together = [&](int seg, int64_t c0, int64_t m) __attribute__((always_inline)) {
    const int64_t i0 = c0 + m * w / kSumWaves, i1 = c0 + m * (w + 1) / kSumWaves;
    float v = 0.0f;
    if (c < cols) {
      int64_t i = i0;
      for (; i + 8 <= i1; i += 8) {
        float e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = part[(i + q) * cols + c];
#pragma unroll
        for (int q = 0; q < 8; ++q) v += e[q];
      }
      for (; i < i1; ++i) v += part[i * cols + c];
    }
    sh[w][lane] = v;
    __syncthreads();
    if (w == 0 && c < cols) {
#pragma unroll
      for (int q = 1; q < kSumWaves; ++q) v += sh[q][lane];
      out[(int64_t)seg * cols + c] = v;
    }
  };
  if (!offs) {
    together(0, 0, (rows + ch - 1) / ch);
    return;
  }
  // the chunks of the segments before, then of the workgroup's own
  int64_t n = 0;
  for (int s = threadIdx.x; s < seg0; s += 64 * kSumWaves) n += count(s);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d, 64);
  if (lane == 0) before[w] = n;
  const int64_t own = w == 0 && lane < segs ? count(seg0 + lane) : 0;
  __syncthreads();
  if (w == 0) {
    int64_t at = own;
#pragma unroll
    for (int d = 1; d < kSumSegs; d <<= 1) {
      const int64_t o = __shfl_up(at, d, 64);
      if (lane >= d) at += o;
    }
    int64_t all = 0;
    for (int q = 0; q < kSumWaves; ++q) all += before[q];
    // within the array whatever the offsets hold (decreasing ones may claim rows twice)
    at += all;
    if (lane < kSumSegs) first[lane + 1] = at < chunks ? at : chunks;
    if (lane == 0) first[0] = all < chunks ? all : chunks;
  }
  __syncthreads();
  if (w < segs) {
    const int64_t c0 = first[w], m = first[w + 1] - c0;
    if (m <= kSumWaves && c < cols) {
      float e[kSumWaves], v = 0.0f;
#pragma unroll
      for (int q = 0; q < kSumWaves; ++q) e[q] = q < m ? part[(c0 + q) * cols + c] : 0.0f;
#pragma unroll
      for (int q = 0; q < kSumWaves; ++q) v += e[q];
      out[(int64_t)(seg0 + w) * cols + c] = v;
    }
  }
  for (int s = 0; s < segs; ++s) {
    const int64_t c0 = first[s], m = first[s + 1] - c0;
    if (m <= kSumWaves) continue;
    together(seg0 + s, c0, m);
    __syncthreads();
  }
}

// f(W, I) for a row of `cols`.  Two pieces a lane (us, bf16: 32768 x 2048 one / two / four pieces 86.6 /
// 82.6 / 84.9, 8192 x 8192 92.6 / 85.0 / 87.7, 16384 x 1024 22.0 / 19.7).
template <typename F>
auto norm_shape(int64_t cols, F f) {
  using std::integral_constant;
  if (cols <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (cols <= 1024) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (cols <= 2048) return f(integral_constant<int, 2>{}, integral_constant<int, 2>{});
  if (cols <= 4096) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (cols <= 8192) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 8>{}, integral_constant<int, 4>{});
}
// The gradient: one piece, for its registers (one / two / four: 32768 x 2048 107.2 / 109.3 / 107.2, 16384 x
// 4096 105 / 113 / 109, 8192 x 8192 108 / 112 / 123, 2999 x 1000 fp32 15.9 / 17.2).
template <typename F>
auto grad_shape(int64_t cols, F f) {
  using std::integral_constant;
  if (cols <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (cols <= 1024) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
  if (cols <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (cols <= 4096) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (cols <= 8192) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}

// f(a value of the type, whether rows are of whole pieces)
template <typename F>
void of_kind(bool bf16, int64_t cols, F f) {
  if (bf16 && cols % 8 == 0) f(uint16_t{}, std::true_type{});
  else if (bf16) f(uint16_t{}, std::false_type{});
  else if (cols % 8 == 0) f(float{}, std::true_type{});
  else f(float{}, std::false_type{});
}

// workgroups of the gradient: four of four wavefronts a CU, or two larger ones
constexpr int64_t kNormGradBlocks = 1024;

int64_t norm_grad_blocks(int64_t rows, int64_t cols) {
  return grad_shape(cols, [&](auto wc, auto) {
    constexpr int W = decltype(wc)::value, PER = W > 4 ? 1 : 4 / W;
    const int64_t most = W > 4 ? kNormGradBlocks / 2 : kNormGradBlocks, need = (rows + PER - 1) / PER;
    return need < most ? need : most;
  });
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool bf16, int64_t rows, int64_t cols, const Fp8Out& out,
                       hipStream_t st) {
  const double inv = 1.0 / (double)cols;
  norm_shape(cols, [&](auto wc, auto ic) {
    constexpr int W = decltype(wc)::value, I = decltype(ic)::value, PER = W > 4 ? 1 : 4 / W;
    // a grid has fewer than 2^32 threads: further rows in further launches
    constexpr int64_t kMost = (int64_t)1 << 22;
    for (int64_t r = 0; r < rows; r += kMost * PER) {
      const int64_t n = (rows - r + PER - 1) / PER;
      const dim3 grid((unsigned)(n < kMost ? n : kMost)), block(W > 4 ? 64 * W : 256);
      of_kind(bf16, cols, [&](auto t, auto ec) {
        k_norm<decltype(t), W, I, decltype(ec)::value><<<grid, block, 0, st>>>(a, r, rows, cols, inv, out);
      });
    }
    return 0;
  });
  return hipGetLastError();
}

size_t norm_grad_ws_bytes(int64_t rows, int64_t cols) {
  return ((size_t)norm_grad_blocks(rows, cols) * cols * 4 + 255) & ~(size_t)255;
}

hipError_t launch_norm_grad(const NormGradArgs& a, bool bf16, int64_t rows, int64_t cols, void* ws,
                            hipStream_t st) {
  const int64_t blocks = norm_grad_blocks(rows, cols);
  float* part = a.dweight ? static_cast<float*>(ws) : nullptr;
  if (rows > 0) {
    grad_shape(cols, [&](auto wc, auto ic) {
      constexpr int W = decltype(wc)::value, I = decltype(ic)::value, PER = W > 4 ? 1 : 4 / W;
      const dim3 grid((unsigned)blocks), block(W > 4 ? 64 * W : 256);
      static_assert(PER == 1 || PER * 512 * W * I * 4 <= 8192, "LDS for four workgroups a CU and more");
      const size_t lds = part && PER > 1 ? (size_t)PER * cols * 4 : 0;
      const float inv = (float)(1.0 / (double)cols);
      of_kind(bf16, cols, [&](auto t, auto ec) {
        k_norm_grad<decltype(t), W, I, decltype(ec)::value><<<grid, block, lds, st>>>(a, rows, cols, inv, part);
      });
      return 0;
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return a.dweight ? launch_column_sums(part, blocks, 1, cols, nullptr, 1, a.dweight, st) : hipSuccess;
}

hipError_t launch_column_sums(const float* part, int64_t rows, int64_t ch, int64_t cols,
                              const int64_t* offs, int nseg, float* out, hipStream_t st) {
  k_column_sums<<<dim3((unsigned)((cols + 63) / 64), (unsigned)((nseg + kSumSegs - 1) / kSumSegs)), 64 * kSumWaves, 0, st>>>(
      part, rows, ch, cols, offs, nseg, chunk_upper_bound(rows, offs ? nseg : 1, ch), out);
  return hipGetLastError();
}

}  // namespace averis
