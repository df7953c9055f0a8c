// Quantization to block-scaled fp8 (fp8_common.hpp) for gfx950.
//
//   k_fp8_rows   runs of 128 along the columns: one read of the input, no LDS
//   k_fp8_tile   128 x 128 tiles through LDS: the transposed copy (runs along
//                the rows), with or without the plain copy, from one read; or
//                both copies of a weight with one scale for the whole tile
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_common.hpp"
#include "launch.hpp"
#include "segments.hpp"

namespace averis {
namespace {

// eight consecutive elements of a row, as loaded
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  u32x4_t w;
  __device__ __forceinline__ void zero() { w = u32x4_t{0u, 0u, 0u, 0u}; }
  // elements c .. c + 7 of a row of cols elements, 0 past its end
  __device__ __forceinline__ void load(const uint16_t* row, int64_t c, int64_t cols) {
    if (c + 8 <= cols) {
      w = *reinterpret_cast<const f8_piece_t*>(row + c);
      return;
    }
    zero();
    if (c >= cols) return;
    // all loads at once, those past the end of the last element (one by one, each
    // behind its own branch: 16384 x 3071 53.7 us instead of 47.0)
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = row[c + i < cols ? c + i : cols - 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 2] |= (c + i < cols ? (uint32_t)e[i] : 0u) << (16 * (i & 1));
  }
  // bits of the largest magnitude, as fp32
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t k = 0x7FFF7FFFu;
    const uint32_t m = pk_max_u16(pk_max_u16(w[0] & k, w[1] & k), pk_max_u16(w[2] & k, w[3] & k));
    const uint32_t lo = m << 16, hi = m & 0xFFFF0000u;
    return lo > hi ? lo : hi;
  }
  __device__ __forceinline__ u32x2_t codes(uint32_t byte) const {
    return u32x2_t{f8_codes4_bf16(w[0], w[1], byte), f8_codes4_bf16(w[2], w[3], byte)};
  }
};
template <>
struct Eight<float> {
  u32x4_t w[2];
  __device__ __forceinline__ void zero() { w[0] = w[1] = u32x4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void load(const float* row, int64_t c, int64_t cols) {
    if (c + 8 <= cols) {
      w[0] = *reinterpret_cast<const f8_piece_t*>(row + c);
      w[1] = *reinterpret_cast<const f8_piece_t*>(row + c + 4);
      return;
    }
    zero();
    if (c >= cols) return;
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = row[c + i < cols ? c + i : cols - 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4][i % 4] = c + i < cols ? __float_as_uint(e[i]) : 0u;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = w[i / 4][i % 4] & 0x7FFFFFFFu;
      m = a > m ? a : m;
    }
    return m;
  }
  __device__ __forceinline__ u32x2_t codes(uint32_t byte) const {
    auto f = [&](int i) { return __uint_as_float(w[i / 4][i % 4]); };
    return u32x2_t{f8_codes4(f(0), f(1), f(2), f(3), byte), f8_codes4(f(4), f(5), f(6), f(7), byte)};
  }
};

template <typename T>
__device__ __forceinline__ u32x2_t eight_codes(const Eight<T>& v, uint32_t amax, uint32_t& byte) {
  byte = f8_scale_byte(amax);
  if (__builtin_expect(f8_not_finite(amax), 0)) {
    byte = kF8One;
    return u32x2_t{kF8NanCodes, kF8NanCodes};
  }
  return v.codes(byte);
}

// the codes of eight elements from column c on, those past the row's end 0
__device__ __forceinline__ u32x2_t without_pad(u32x2_t q, int64_t c, int64_t cols) {
  const int left = (int)(cols - c < 8 ? cols - c : 8);
  return u32x2_t{f8_without_pad(q[0], left), f8_without_pad(q[1], left - 4)};
}

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

// One 128 x 128 tile per workgroup of eight wavefronts.  Thread (r = t / 16,
// i = t % 16) holds eight columns of rows r, r + 32, ..; a row's run is sixteen
// lanes, so the plain copy comes from the registers.  The values go to LDS as
// loaded; for the transposed copy a thread takes a column's (bf16: a column
// pair's) run of rows from there, and the codes go back through LDS (bf16: in
// the place of the values, 36 KB in all, four workgroups a CU) so that eight
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
  return (size_t)128 * 128 * sizeof(T) + (sizeof(T) == 2 ? 0 : 128 * 128) + kTileWaves * 64 * 4;
}

template <typename T, bool TILE>
__global__ __launch_bounds__(kTileThreads) void k_fp8_tile(
    const T* __restrict__ a, int64_t rows, int64_t cols, int64_t lda, int64_t bstride,
    const int64_t* offs, int nseg, int tx, bool near, Fp8Out out, Fp8Out out_t) {
  extern __shared__ __attribute__((aligned(16))) unsigned char sm[];
  T* raw = reinterpret_cast<T*>(sm);   // [128][128]
  // codes, [128 columns][128 rows]
  unsigned char* ct = sm + (sizeof(T) == 2 ? 0 : 128 * 128 * sizeof(T));
  // maxima: of rows, or a column's (column pair's) part of each wavefront
  uint32_t* red = reinterpret_cast<uint32_t*>(sm + fp8_tile_lds<T>()) - kTileWaves * 64;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  uint32_t id = blockIdx.x;
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
  a += b * bstride;
  const int i = t & 15, r = t >> 4;
  constexpr int PER = 32 / kTileWaves, STEP = 4 * kTileWaves;   // rows a thread
  Eight<T> v[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    v[p].zero();
    if (r + STEP * p < nr) v[p].load(a + (r0 + r + STEP * p) * lda, c0 + 8 * i, cols);
  }
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
  if (!out_t.codes) return;
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
    uint32_t m = tile_max;
    if constexpr (!TILE) {
      for (int q = 0; q < PR; ++q) {
        const uint32_t z = __float_as_uint(src[q * 128]) & 0x7FFFFFFFu;
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
        const float* z = src + (16 * h + 4 * q) * 128;
        y[q] = f8_not_finite(m) ? kF8NanCodes : f8_codes4(z[0], z[128], z[256], z[384], byte);
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

template <typename T, bool TILE>
hipError_t tile_t(const void* a, int batch, int64_t rows, int64_t cols, int64_t lda,
                  int64_t bstride, const int64_t* offs, int nseg, const Fp8Out& out,
                  const Fp8Out& out_t, hipStream_t st) {
  constexpr size_t lds = fp8_tile_lds<T>();
  const hipError_t e = lds_attr_once<&k_fp8_tile<T, TILE>>((int)lds);
  if (e != hipSuccess) return e;
  const int64_t tx = (cols + 127) / 128;
  // rows that do not start at a 128-byte line: neighbouring tiles share lines
  const bool near = ((reinterpret_cast<uintptr_t>(a) | (uintptr_t)(lda * (int64_t)sizeof(T)) |
                      (uintptr_t)(batch > 1 ? bstride * (int64_t)sizeof(T) : 0)) & 127) != 0;
  const dim3 g((unsigned)(tx * chunk_upper_bound(rows, offs ? nseg : 1, 128)), 1u, (unsigned)batch);
  k_fp8_tile<T, TILE><<<g, kTileThreads, lds, st>>>(static_cast<const T*>(a), rows, cols, lda, bstride,
                                           offs, nseg, (int)tx, near, out, out_t);
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
  if (bf16)
    return tile ? tile_t<uint16_t, true>(a, batch, rows, cols, lda, bstride, offs, nseg, out, out_t, st)
                : tile_t<uint16_t, false>(a, batch, rows, cols, lda, bstride, offs, nseg, out, out_t, st);
  return tile ? tile_t<float, true>(a, batch, rows, cols, lda, bstride, offs, nseg, out, out_t, st)
              : tile_t<float, false>(a, batch, rows, cols, lda, bstride, offs, nseg, out, out_t, st);
}

}  // namespace averis
