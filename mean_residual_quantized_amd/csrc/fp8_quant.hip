// Quantization to block-scaled fp8 (fp8_common.hpp) for gfx950.
//
//   k_fp8_rows   runs of 128 along the columns: one read of the input, no LDS
//   k_fp8_tile   128 x 128 tiles through LDS: the transposed copy (runs along
//                the rows), with or without the plain copy, from one read; or
//                both copies of a weight with one scale for the whole tile; of a
//                matrix, of a norm's output, or of a gradient before an
//                activation with its column sums
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "activation.hpp"
#include "fp8_eight.hpp"
#include "launch.hpp"
#include "segments.hpp"

namespace averis {
namespace {

// A wavefront takes 512 columns (four blocks, sixteen lanes each, eight
// elements a lane) of kRowsPerWave rows: all rows' loads in flight, then per
// row the blocks' maxima by four DPP steps, the codes (8 bytes a lane, 512
// contiguous bytes a row) and the four scale bytes as one word.  Bound by memory:
// 16384 x 3072 bf16 26.0 us (5.8 TB/s; the tile kernel with both copies 38.2, so
// it is taken only where the transposed copy is wanted), 16 x 2048 3.2 us.
constexpr int kRowsPerWave = 4;

template <typename T>
__global__ __launch_bounds__(256) void k_fp8_rows(const T* __restrict__ a, int64_t rows,
                                                  int64_t cols, int64_t lda, int groups,
                                                  uint8_t* __restrict__ codes, int64_t pitch,
                                                  uint8_t* __restrict__ scales, int64_t spitch) {
  const int lane = threadIdx.x & 63;
  const uint32_t task = __builtin_amdgcn_readfirstlane(blockIdx.x * 4u + (threadIdx.x >> 6));
  const int g = (int)(task % (uint32_t)groups);
  const int64_t r0 = (int64_t)(task / (uint32_t)groups) * kRowsPerWave;
  if (r0 >= rows) return;
  const int64_t c = 512 * (int64_t)g + 8 * lane;
  Eight<T> v[kRowsPerWave];
#pragma unroll
  for (int i = 0; i < kRowsPerWave; ++i) {
    v[i].zero();
    if (r0 + i < rows) v[i].load(a + (r0 + i) * lda, c, cols);
  }
#pragma unroll
  for (int i = 0; i < kRowsPerWave; ++i) {
    uint32_t byte;
    u32x2_t q = eight_codes(v[i], row16_max(v[i].amax()), byte);
    if (512 * (int64_t)(g + 1) > cols) q = without_pad(q, c, cols);
    const uint32_t word = __builtin_amdgcn_readlane(byte, 0) | __builtin_amdgcn_readlane(byte, 16) << 8 |
                          __builtin_amdgcn_readlane(byte, 32) << 16 |
                          __builtin_amdgcn_readlane(byte, 48) << 24;
    if (r0 + i >= rows) break;
    if (c < pitch) *reinterpret_cast<u32x2_t*>(codes + (r0 + i) * pitch + c) = q;
    if (lane == 0) *reinterpret_cast<uint32_t*>(scales + (r0 + i) * spitch + 4 * g) = word;
  }
}

// ---------------------------------------------------------------------------
// What a tile's values come from, eight columns of a row at a time: `load` (all
// of a thread's loads are in flight before the first is used), then `make`.
// ---------------------------------------------------------------------------
template <typename T>
struct PlainSrc {   // a matrix as it is
  using Type = T;
  static constexpr bool kSums = false, kLastFirst = false;
  const T* a;
  int64_t ld, bstride;
  using Raw = Eight<T>;
  struct Columns {};
  __device__ __forceinline__ void columns(Columns&, int64_t, int64_t) const {}
  __device__ __forceinline__ void load(Raw& v, int64_t b, int64_t row, int64_t c, int64_t cols) const {
    v.load(a + b * bstride + row * ld, c, cols);
  }
  __device__ __forceinline__ void make(Eight<T>& v, const Raw& x, Columns&) const { v = x; }
};

// a norm's output from the sum it is of and each row's factor: the same
// operations as k_norm's, so the same values.  Last rows first: after k_norm
// 32768 x 2048 45 -> 38 us.
template <typename T>
struct NormSrc {
  using Type = T;
  static constexpr bool kSums = false, kLastFirst = true;
  const T* h;
  int64_t ld;
  const float* rstd;
  const void* weight;
  bool wbf16;
  struct Raw {
    Eight<T> h;
    float rstd;
    __device__ __forceinline__ void zero() {
      h.zero();
      rstd = 0.0f;
    }
  };
  struct Columns {
    float w[8];
  };
  __device__ __forceinline__ void columns(Columns& at, int64_t c, int64_t cols) const {
    load_vector(weight, wbf16, c, cols, at.w);
  }
  __device__ __forceinline__ void load(Raw& v, int64_t, int64_t row, int64_t c, int64_t cols) const {
    v.h.load(h + row * ld, c, cols);
    v.rstd = rstd[row];
  }
  __device__ __forceinline__ void make(Eight<T>& v, const Raw& x, Columns& at) const {
    float f[8];
    x.h.f32(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * x.rstd * at.w[i];
    v.set(f);
  }
};

// dy act'(z), and its sums over the rows (in fp32, before it is rounded).  Both
// copies: 16384 x 4096 gelu bf16 88 us (403 MB, 4.6 TB/s; the vector pipes are busy
// for 61 of them), 32768 x 768 in 64 segments 39 us.
template <typename T>
struct ActSrc {
  using Type = T;
  static constexpr bool kSums = true, kLastFirst = false;
  const T* dy;
  const T* z;
  int64_t lddy, ldz;
  int act;
  float* part;   // [chunk][column], or nullptr
  struct Raw {
    Eight<T> dy, z;
    __device__ __forceinline__ void zero() {
      dy.zero();
      z.zero();
    }
  };
  struct Columns {
    float sum[8];
  };
  __device__ __forceinline__ void columns(Columns& at, int64_t, int64_t) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) at.sum[i] = 0.0f;
  }
  __device__ __forceinline__ void load(Raw& v, int64_t, int64_t row, int64_t c, int64_t cols) const {
    v.dy.load(dy + row * lddy, c, cols);
    if (act != kActNone) v.z.load(z + row * ldz, c, cols);
  }
  __device__ __forceinline__ void make(Eight<T>& v, const Raw& x, Columns& at) const {
    float f[8], z[8];
    x.dy.f32(f);
    x.z.f32(z);
    if (act == kActRelu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = z[i] <= 0.0f ? 0.0f : f[i];   // (a NaN z lets f by)
    } else if (act == kActSilu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= act_silu_slope(z[i]);
    } else if (act == kActGelu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= act_gelu_slope(z[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) at.sum[i] += f[i];
    v.set(f);
  }
};

// One 128 x 128 tile per workgroup of eight wavefronts.  Thread (r = t / 16,
// i = t % 16) holds eight columns of rows r, r + 32, ..; a row's run is sixteen
// lanes, so the plain copy comes from the registers.  The values go to LDS as
// loaded; for the transposed copy a thread takes a column's (bf16: a column
// pair's) run of rows from there, and the codes go back through LDS (in the
// place of the values: bf16 34 KB in all, four workgroups a CU; fp32 66 KB, two,
// 16384 x 2048 37.5 us, 44.6 with a place of their own and one) so that eight
// lanes store a 128-byte row of the transposed copy.  Bound by memory: each
// value is read once and each code written once.  Neighbouring workgroups take
// neighbouring tiles of the same rows.  Workgroup w runs on die w mod 8; where
// tiles share lines (`near`) eight in a row go to one die, which then reads most
// of the lines once (16384 x 3068: 148 -> 107 MB into the L2s, 45.5 -> 42.5 us;
// 2999 x 1333 9.2 -> 8.7; where they share none 16384 x 3072 38.3 -> 39.8, and it
// is left).
//
// TILE: one scale for the tile (both copies then hold the same codes).
//
// Both copies, bf16, us (four wavefronts, row tiles first, values and codes
// apart -> this; TB/s of reads and writes):
//   16384 x 3072                  44.5 -> 39.3 (5.1)
//   32768 x 2048, 64 segments     71.0 -> 53.5 (5.0)
//   2999 x 1000                    9.0 ->  6.5 (latency)
//   weight, 64 x 2048 x 768       77.5 -> 75.7 (5.3)
constexpr int kTileWaves = 8, kTileThreads = 64 * kTileWaves;

template <typename T>
constexpr size_t fp8_tile_lds() {
  return (size_t)128 * 128 * sizeof(T) + kTileWaves * 64 * 4;
}

template <typename Src, bool TILE>
__global__ __launch_bounds__(kTileThreads) void k_fp8_tile(Src source, int64_t rows, int64_t cols,
                                                           const int64_t* offs, int nseg, int tx,
                                                           bool near, Fp8Out out, Fp8Out out_t) {
  using T = typename Src::Type;
  extern __shared__ __attribute__((aligned(16))) unsigned char sm[];
  T* raw = reinterpret_cast<T*>(sm);   // [128][128]
  // codes, [128 columns][128 rows], in the values' place
  unsigned char* ct = sm;
  // maxima: of rows, or a column's (column pair's) part of each wavefront
  uint32_t* red = reinterpret_cast<uint32_t*>(sm + fp8_tile_lds<T>()) - kTileWaves * 64;
  // sums: a column's part of each wavefront
  float* sums = reinterpret_cast<float*>(sm + fp8_tile_lds<T>());
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  // (a source that was written just now: its last rows first, while the last-level cache has them)
  uint32_t id = Src::kLastFirst ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  if (near && id < (gridDim.x & ~63u)) id = (id & ~63u) + (id & 7u) * 8u + (id >> 3 & 7u);
  const int chunk = (int)(id / (uint32_t)tx), block = (int)(id % (uint32_t)tx);
  const int64_t c0 = (int64_t)block * 128;
  // a chunk of 128 rows, of one segment where there are several
  int64_t r0 = 128 * (int64_t)chunk;
  int nr = (int)(rows - r0 < 128 ? rows - r0 : 128);
  if (offs) {
    SegTable segs;
    segs.init(offs, nseg, rows, 128);
    int seg, ra, rb;
    if (!segs.chunk(chunk, seg, ra, rb)) return;
    r0 = ra;
    nr = rb - ra;
  }
  const int64_t b = blockIdx.z;
  const int i = t & 15, r = t >> 4;
  constexpr int PER = 32 / kTileWaves, STEP = 4 * kTileWaves;   // rows a thread
  typename Src::Raw raws[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    raws[p].zero();
    if (r + STEP * p < nr) source.load(raws[p], b, r0 + r + STEP * p, c0 + 8 * i, cols);
  }
  Eight<T> v[PER];
  {
    typename Src::Columns at;
    source.columns(at, c0 + 8 * i, cols);
#pragma unroll
    for (int p = 0; p < PER; ++p) source.make(v[p], raws[p], at);
    if constexpr (Src::kSums) {
      // rows of a wavefront, then (below) its sums, in order
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        at.sum[q] += __shfl_xor(at.sum[q], 16, 64);
        at.sum[q] += __shfl_xor(at.sum[q], 32, 64);
      }
      if (lane < 16) {
#pragma unroll
        for (int q = 0; q < 8; ++q) sums[w * 128 + 8 * i + q] = at.sum[q];
      }
    }
  }
  auto sums_out = [&]() __attribute__((always_inline)) {
    if constexpr (Src::kSums) {
      if (t < 128 && c0 + t < cols && source.part) {
        float s = sums[t];
#pragma unroll
        for (int q = 1; q < kTileWaves; ++q) s += sums[q * 128 + t];
        source.part[(int64_t)chunk * cols + c0 + t] = s;
      }
    }
  };
  uint32_t tile_max = 0;
  if constexpr (TILE) {
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const uint32_t m = v[p].amax();
      tile_max = m > tile_max ? m : tile_max;
    }
    tile_max = row16_max(tile_max);
    if (i == 0) red[r] = tile_max;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < STEP; ++q) tile_max = red[q] > tile_max ? red[q] : tile_max;
  }
  if (out.codes) {
    const int64_t row0 = b * rows + r0 + r;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      uint32_t byte;
      const uint32_t m = TILE ? tile_max : row16_max(v[p].amax());
      u32x2_t q = eight_codes(v[p], m, byte);
      if (c0 + 128 > cols) q = without_pad(q, c0 + 8 * i, cols);
      if (r + STEP * p < nr) {
        *reinterpret_cast<u32x2_t*>(out.codes + (row0 + STEP * p) * out.pitch + c0 + 8 * i) = q;
        if (i == 0) out.scales[(row0 + STEP * p) * out.spitch + block] = (uint8_t)byte;
      }
    }
  }
  if (!out_t.codes) {
    if constexpr (Src::kSums) {
      __syncthreads();
      sums_out();
    }
    return;
  }
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    T* dst = raw + (r + STEP * p) * 128 + 8 * i;
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<u32x4_t*>(dst) = v[p].w;
    } else {
      *reinterpret_cast<u32x4_t*>(dst) = v[p].w[0];
      *reinterpret_cast<u32x4_t*>(dst + 4) = v[p].w[1];
    }
  }
  __syncthreads();
  sums_out();
  const int64_t orow = b * cols + c0;   // row of the transposed copy
  auto scale_out = [&](int col, uint32_t byte) {
    if (c0 + col < cols) out_t.scales[(orow + col) * out_t.spitch + chunk] = (uint8_t)byte;
  };
  // piece q (16 rows) of a column's codes is kept at q ^ (column / 2 mod 8):
  // neighbouring lanes' writes go to different banks
  auto put = [&](int col, int q, u32x4_t x) {
    *reinterpret_cast<u32x4_t*>(ct + col * 128 + 16 * (q ^ ((col >> 1) & 7))) = x;
  };
  if constexpr (sizeof(T) == 2) {
    constexpr int WR = 128 / kTileWaves;   // rows a wavefront
    const uint32_t* src = reinterpret_cast<const uint32_t*>(raw) + WR * w * 64 + lane;
    uint32_t x[WR];
#pragma unroll
    for (int q = 0; q < WR; ++q) x[q] = src[q * 64];
    uint32_t m0 = tile_max, m1 = tile_max;
    if constexpr (TILE) __syncthreads();   // the codes take the values' place
    if constexpr (!TILE) {
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < WR; ++q) m = pk_max_u16(m, x[q] & 0x7FFF7FFFu);
      red[w * 64 + lane] = m;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kTileWaves; ++q) m = pk_max_u16(m, red[q * 64 + lane]);
      m0 = m << 16;
      m1 = m & 0xFFFF0000u;
    }
    const uint32_t b0 = f8_not_finite(m0) ? kF8One : f8_scale_byte(m0);
    const uint32_t b1 = f8_not_finite(m1) ? kF8One : f8_scale_byte(m1);
#pragma unroll
    for (int h = 0; h < WR / 16; ++h) {
      u32x4_t y0, y1;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t* z = x + 16 * h + 4 * q;
        // the low and the high halves of neighbouring rows
        y0[q] = f8_codes4_bf16(__builtin_amdgcn_perm(z[1], z[0], 0x05040100u),
                               __builtin_amdgcn_perm(z[3], z[2], 0x05040100u), b0);
        y1[q] = f8_codes4_bf16(__builtin_amdgcn_perm(z[1], z[0], 0x07060302u),
                               __builtin_amdgcn_perm(z[3], z[2], 0x07060302u), b1);
        if (f8_not_finite(m0)) y0[q] = kF8NanCodes;
        if (f8_not_finite(m1)) y1[q] = kF8NanCodes;
      }
      if (nr < 128) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int left = nr - (WR * w + 16 * h + 4 * q);
          y0[q] = f8_without_pad(y0[q], left);
          y1[q] = f8_without_pad(y1[q], left);
        }
      }
      put(2 * lane, WR / 16 * w + h, y0);
      put(2 * lane + 1, WR / 16 * w + h, y1);
    }
    if (w == 0) {
      scale_out(2 * lane, b0);
      scale_out(2 * lane + 1, b1);
    }
  } else {
    // column t mod 128, rows PR (t / 128) .. PR (t / 128) + PR - 1
    constexpr int PARTS = kTileWaves / 2, PR = 128 / PARTS;
    const int col = t & 127, part = t >> 7;
    const float* src = reinterpret_cast<const float*>(raw) + PR * part * 128 + col;
    float x[PR];
#pragma unroll
    for (int q = 0; q < PR; ++q) x[q] = src[q * 128];
    uint32_t m = tile_max;
    if constexpr (TILE) __syncthreads();   // the codes take the values' place
    if constexpr (!TILE) {
#pragma unroll
      for (int q = 0; q < PR; ++q) {
        const uint32_t z = __float_as_uint(x[q]) & 0x7FFFFFFFu;
        m = z > m ? z : m;
      }
      red[part * 128 + col] = m;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < PARTS; ++q) m = red[q * 128 + col] > m ? red[q * 128 + col] : m;
    }
    const uint32_t byte = f8_not_finite(m) ? kF8One : f8_scale_byte(m);
#pragma unroll
    for (int h = 0; h < PR / 16; ++h) {
      u32x4_t y;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float* z = x + 16 * h + 4 * q;
        y[q] = f8_not_finite(m) ? kF8NanCodes : f8_codes4(z[0], z[1], z[2], z[3], byte);
      }
      if (nr < 128) {
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = f8_without_pad(y[q], nr - (PR * part + 16 * h + 4 * q));
      }
      put(col, PR / 16 * part + h, y);
    }
    if (part == 0) scale_out(col, byte);
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 16 / kTileWaves; ++p) {
    const int col = (t >> 3) + 8 * kTileWaves * p, q = t & 7;
    if (c0 + col < cols)
      *reinterpret_cast<u32x4_t*>(out_t.codes + (orow + col) * out_t.pitch + (int64_t)chunk * 128 +
                                  16 * q) =
          *reinterpret_cast<const u32x4_t*>(ct + col * 128 + 16 * (q ^ ((col >> 1) & 7)));
  }
}

// rows that do not start at a 128-byte line: neighbouring tiles share lines
bool off_lines(const void* a, int64_t row_bytes) {
  return ((reinterpret_cast<uintptr_t>(a) | (uintptr_t)row_bytes) & 127) != 0;
}

template <typename Src, bool TILE>
hipError_t tile_t(const Src& src, bool near, int batch, int64_t rows, int64_t cols,
                  const int64_t* offs, int nseg, const Fp8Out& out, const Fp8Out& out_t,
                  hipStream_t st) {
  constexpr size_t lds = fp8_tile_lds<typename Src::Type>() + (Src::kSums ? kTileWaves * 128 * 4 : 0);
  const hipError_t e = lds_attr_once<&k_fp8_tile<Src, TILE>>((int)lds);
  if (e != hipSuccess) return e;
  const int64_t tx = (cols + 127) / 128;
  const dim3 g((unsigned)(tx * chunk_upper_bound(rows, offs ? nseg : 1, 128)), 1u, (unsigned)batch);
  k_fp8_tile<Src, TILE><<<g, kTileThreads, lds, st>>>(src, rows, cols, offs, nseg, (int)tx, near, out, out_t);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_rows(const void* a, bool bf16, int64_t rows, int64_t cols, int64_t lda,
                           const Fp8Out& out, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const int64_t groups = (cols + 511) / 512;
  // a grid has fewer than 2^32 threads: 2^24 - 1 workgroups of four tasks each;
  // further rows in further launches (groups <= 2^21)
  const int64_t most = (int64_t)((1 << 24) - 1) * 4 / groups * kRowsPerWave;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t here = rows - r < most ? rows - r : most;
    const int64_t tasks = (here + kRowsPerWave - 1) / kRowsPerWave * groups;
    const dim3 g((unsigned)((tasks + 3) / 4));
    uint8_t* codes = out.codes + r * out.pitch;
    uint8_t* scales = out.scales + r * out.spitch;
    if (bf16)
      k_fp8_rows<uint16_t><<<g, 256, 0, st>>>(static_cast<const uint16_t*>(a) + r * lda, here, cols,
                                              lda, (int)groups, codes, out.pitch, scales, out.spitch);
    else
      k_fp8_rows<float><<<g, 256, 0, st>>>(static_cast<const float*>(a) + r * lda, here, cols, lda,
                                           (int)groups, codes, out.pitch, scales, out.spitch);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_tile(const void* a, bool bf16, bool tile, int batch, int64_t rows,
                           int64_t cols, int64_t lda, int64_t bstride, const int64_t* offs,
                           int nseg, const Fp8Out& out, const Fp8Out& out_t, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  auto run = [&](auto t) {
    using T = decltype(t);
    const PlainSrc<T> src{static_cast<const T*>(a), lda, bstride};
    const bool near = off_lines(a, lda * (int64_t)sizeof(T)) ||
                      (batch > 1 && off_lines(nullptr, bstride * (int64_t)sizeof(T)));
    return tile ? tile_t<PlainSrc<T>, true>(src, near, batch, rows, cols, offs, nseg, out, out_t, st)
                : tile_t<PlainSrc<T>, false>(src, near, batch, rows, cols, offs, nseg, out, out_t, st);
  };
  return bf16 ? run(uint16_t{}) : run(float{});
}

hipError_t launch_norm_tile(const void* h, bool bf16, int64_t rows, int64_t cols, int64_t ldh,
                            const void* weight, bool wbf16, const float* rstd, const Fp8Out& out_t,
                            hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const Fp8Out none{nullptr, nullptr, 0, 0};
  auto run = [&](auto t) {
    using T = decltype(t);
    const NormSrc<T> src{static_cast<const T*>(h), ldh, rstd, weight, wbf16};
    return tile_t<NormSrc<T>, false>(src, off_lines(h, ldh * (int64_t)sizeof(T)), 1, rows, cols,
                                     nullptr, 1, none, out_t, st);
  };
  return bf16 ? run(uint16_t{}) : run(float{});
}

size_t act_grad_ws_bytes(int64_t rows, int64_t cols, int nseg) {
  return ((size_t)chunk_upper_bound(rows, nseg, 128) * cols * 4 + 255) & ~(size_t)255;
}

hipError_t launch_act_grad(const void* dy, bool bf16, int64_t rows, int64_t cols, int64_t lddy,
                           const void* z, int64_t ldz, int act, const int64_t* offs, int nseg,
                           const Fp8Out& out, const Fp8Out& out_t, float* dbias, void* ws,
                           hipStream_t st) {
  float* part = dbias ? static_cast<float*>(ws) : nullptr;
  auto run = [&](auto t) {
    using T = decltype(t);
    const ActSrc<T> src{static_cast<const T*>(dy), static_cast<const T*>(z), lddy, ldz, act, part};
    return tile_t<ActSrc<T>, false>(src, off_lines(dy, lddy * (int64_t)sizeof(T)), 1, rows, cols,
                                    offs, nseg, out, out_t, st);
  };
  if (rows > 0) {
    const hipError_t e = bf16 ? run(uint16_t{}) : run(float{});
    if (e != hipSuccess) return e;
  }
  return dbias ? launch_column_sums(part, rows, 128, cols, offs, nseg, dbias, st) : hipSuccess;
}

}  // namespace averis
