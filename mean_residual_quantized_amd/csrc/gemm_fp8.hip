// NT products of block-scaled fp8 operands (fp8_common.hpp) for gfx950:
//   C[m][n] = sum over blocks kb of 2^(sa[m][kb] + sb[n][kb] - 254)
//                                   sum over the block's 128 k of a[m][k] b[n][k]
//
// Both factors of a block's scale are powers of two in E8M0, the form
// v_mfma_scale_f32_32x32x64_f8f6f4 takes per row and 32 k, so the accumulators
// stay in the accumulation registers for the whole K loop and scaling costs no
// vector instruction.
//
// Accuracy.  The fp8 matrix instructions add the products of eight consecutive
// k with each term cut at 2^-13 of the largest of the eight, and add those
// sums and C in fp32.  So |error| <= 7 * 2^-13 sum |a b| at worst and, on
// random operands, 1.2e-5 of the result's norm: a choice taken with the
// format, whose own rounding is 2^-4 of each operand, for the instruction's
// rate (twice that of bf16).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_common.hpp"
#include "launch.hpp"
#include "segments.hpp"

namespace averis {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kF8Threads = 256;   // four wavefronts, 2 x 2 over the tile
constexpr int kF8BM = 256;        // rows of a tile

// two slots of a stage's codes (128 bytes a row) and two of scale words (four
// stages, 4 bytes a row); the epilogue stages the bf16 tile over them
constexpr size_t f8_ring_bytes(int fn) { return (size_t)(kF8BM + 64 * fn) * (2 * 128 + 2 * 4); }
constexpr size_t f8_epi_row(int fn) { return (size_t)2 * 64 * fn + 16; }
constexpr size_t f8_lds_bytes(int fn) {
  return f8_ring_bytes(fn) > kF8BM * f8_epi_row(fn) ? f8_ring_bytes(fn) : kF8BM * f8_epi_row(fn);
}

template <int V>
struct F8Step {
  static constexpr int value = V;
};

__device__ __forceinline__ i32x8_t frag(u32x4_t a, u32x4_t b) {
  return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// ---------------------------------------------------------------------------
// The tiled kernel: 256 x 64 FN outputs a workgroup, one workgroup a CU, each
// wavefront 128 x 32 FN of them (4 x FN accumulators of 32 x 32).
//
// A stage is one block of 128 k: two k-steps of 64.  Its codes come straight
// from memory to LDS (16 bytes a lane, eight lanes to a row, the row's pieces
// in the order piece ^ (row mod 8) so that fragment reads meet no bank
// twice).  Two slots: stage s computes k-step 0 from registers while it reads
// k-step 1's fragments; then (its slot read out, stage s + 1 landed) one
// barrier; then k-step 1 while stage s + 2 is loaded into the slot and stage s
// + 1's first fragments are read.
//
// Scale bytes come four stages at a time, one aligned word a row, the same
// way.
// ---------------------------------------------------------------------------
template <int FN, bool OUT_BF16>
__global__ __launch_bounds__(kF8Threads, 1) void k_gemm_f8(Fp8Operand A, Fp8Operand B, int64_t m,
                                                           int64_t n, int k_blocks, int mode,
                                                           const int64_t* offs, int nseg,
                                                           int64_t seg_rows, void* c, int64_t ldc,
                                                           int64_t c_split) {
  constexpr int BM = kF8BM, BN = 64 * FN, ROWS = BM + BN;
  constexpr int SLOT = ROWS * 128, SSLOT = ROWS * 4;
  constexpr int CPW = ROWS / 8 / 4;    // code loads a wavefront issues for a stage
  constexpr int SPW = (ROWS / 64 + 3) / 4;   // scale loads for four stages, at most
  constexpr int NF = 4 + FN;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_f8[];
  unsigned char* ring = smem_f8;
  unsigned char* sring = smem_f8 + 2 * SLOT;

  int64_t tile_x, tile_y;
  xcd_tile(tile_x, tile_y);
  int64_t m0 = tile_y * BM, m_end = m;
  int kb0 = 0, kb1 = k_blocks;
  int64_t boff = 0;
  if (mode == kF8RowSegs) {
    const SegRange sr = locate_chunk(offs, nseg, m, BM, tile_y);
    if (sr.seg < 0) return;
    m0 = sr.r0;
    m_end = sr.r1;
    boff = (int64_t)sr.seg * n;
  } else if (mode == kF8BlockSegs) {
    const SegRange sr = describe_segment(offs, nseg, seg_rows, 128, blockIdx.z);
    kb0 = (int)sr.c0;
    kb1 = (int)sr.c1;
  } else if (gridDim.z > 1) {   // a split's share of the blocks
    kb0 = (int)((int64_t)k_blocks * blockIdx.z / gridDim.z);
    kb1 = (int)((int64_t)k_blocks * (blockIdx.z + 1) / gridDim.z);
  }
  c = static_cast<char*>(c) + (int64_t)blockIdx.z * c_split * (OUT_BF16 ? 2 : 4);
  const int64_t n0 = tile_x * BN;
  const int nk = kb1 - kb0;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int rows_here = (int)(m_end - m0 < BM ? m_end - m0 : BM);
  const int cols_here = (int)(n - n0 < BN ? n - n0 : BN);

  f32x16_t acc[4][FN];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  if (nk > 0) {
    const uint8_t* a_c = A.codes + m0 * A.pitch + (int64_t)kb0 * 128;
    const uint8_t* b_c = B.codes + (boff + n0) * B.pitch + (int64_t)kb0 * 128;
    // word g of a row: its stages 4 g .. 4 g + 3 counted from kb0 rounded down
    const int ph = kb0 & 3;
    const uint8_t* a_s = A.scales + m0 * A.spitch + (kb0 - ph);
    const uint8_t* b_s = B.scales + (boff + n0) * B.spitch + (kb0 - ph);
    const int g_last = (ph + nk - 1) >> 2;

    // code load j: rows 8 j .. 8 j + 7 of the tile's A rows, then B rows; rows
    // past the edge repeat the last one (their products are never stored)
    const int lr = lane >> 3;
    const uint32_t piece_off = 16u * (uint32_t)((lane & 7) ^ lr);
    uint32_t cofs[CPW], sofs[SPW];
#pragma unroll
    for (int q = 0; q < CPW; ++q) {
      const int j = wave + 4 * q;
      const bool isa = 8 * j < BM;
      const int r = (isa ? 8 * j : 8 * j - BM) + lr;
      const int lim = isa ? rows_here : cols_here;
      cofs[q] = (uint32_t)((r < lim ? r : lim - 1) * (isa ? A.pitch : B.pitch)) + piece_off;
    }
#pragma unroll
    for (int q = 0; q < SPW; ++q) {
      const int i = wave + 4 * q;
      const bool isa = 64 * i < BM;
      const int r = (isa ? 64 * i : 64 * i - BM) + lane;
      const int lim = isa ? rows_here : cols_here;
      sofs[q] = (uint32_t)((r < lim ? r : lim - 1) * (isa ? A.spitch : B.spitch));
    }
    auto load_codes = [&](int s, int slot) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < CPW; ++q) {
        const int j = wave + 4 * q;
        // 8 j < BM exactly when q < BM / 32
        const uint8_t* base = (q < BM / 32 ? a_c : b_c) + 128 * (int64_t)s;
        __builtin_amdgcn_global_load_lds((const void*)(base + cofs[q]),
                                         (lds_void*)(ring + slot * SLOT + j * 1024), 16, 0, 0);
      }
    };
    auto load_scales = [&](int g) __attribute__((always_inline)) {
      const int gl = g < g_last ? g : g_last;
#pragma unroll
      for (int q = 0; q < SPW; ++q) {
        const int i = wave + 4 * q;
        if (ROWS / 64 % 4 == 0 || i < ROWS / 64) {
          // 64 i < BM exactly when q < BM / 256
          const uint8_t* base = (q < BM / 256 ? a_s : b_s) + 4 * (int64_t)gl;
          __builtin_amdgcn_global_load_lds((const void*)(base + sofs[q]),
                                           (lds_void*)(sring + (g & 1) * SSLOT + i * 256), 4, 0, 0);
        }
      }
    };
    const int lrow = lane & 31, lh = lane >> 5;
    auto row_of = [&](int f) { return f < 4 ? wm * 128 + 32 * f : BM + wn * 32 * FN + 32 * (f - 4); };
    i32x8_t fr[2][NF];
    // fragments of k-step js (lane half h: pieces 4 js + 2 h and the next)
    auto read_step = [&](int slot, auto jc) __attribute__((always_inline)) {
      constexpr int js = decltype(jc)::value;
      const unsigned char* sl = ring + slot * SLOT + lrow * 128;
      const int p0 = 16 * ((4 * js + 2 * lh) ^ (lane & 7)), p1 = 16 * ((4 * js + 2 * lh + 1) ^ (lane & 7));
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(sl + row_of(f) * 128 + p0);
        const u32x4_t y = *reinterpret_cast<const u32x4_t*>(sl + row_of(f) * 128 + p1);
        fr[js][f] = frag(x, y);
      }
    };
    uint32_t words[NF];
    auto read_words = [&](int g) __attribute__((always_inline)) {
#pragma unroll
      for (int f = 0; f < NF; ++f)
        words[f] = *reinterpret_cast<const uint32_t*>(sring + (g & 1) * SSLOT + (row_of(f) + lrow) * 4);
    };
    int sc[NF];
    // B's fragment first: a lane then holds four consecutive columns of a row
    auto mfmas = [&](auto jc) __attribute__((always_inline)) {
      constexpr int js = decltype(jc)::value;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fr[js][4 + j], fr[js][i], acc[i][j], 0, 0, 0, sc[4 + j], 0, sc[i]);
    };
    auto barrier = []() __attribute__((always_inline)) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    constexpr F8Step<0> step0{};
    constexpr F8Step<1> step1{};

    load_scales(0);
    load_scales(1);
    load_codes(0, 0);
    load_codes(nk > 1 ? 1 : 0, 1);
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): nothing else is counted
    barrier();
    read_words(0);
    read_step(0, step0);
    for (int s = 0; s < nk; ++s) {
      const int slot = s & 1, q = s + ph;
#pragma unroll
      for (int f = 0; f < NF; ++f) sc[f] = (int)(words[f] >> (8 * (q & 3)));
      read_step(slot, step1);
      mfmas(step0);
      // this slot read out and stage s + 1 landed, for every wavefront
      __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
      barrier();
      if (s + 2 < nk) load_codes(s + 2, slot);
      if (s > 0 && (q & 3) == 0) load_scales((q >> 2) + 1);
      if (s + 1 < nk) {
        read_step(slot ^ 1, step0);
        if (((q + 1) & 3) == 0) read_words((q + 1) >> 2);
      }
      mfmas(step1);
    }
    mfma_drain();
    __builtin_amdgcn_s_waitcnt(0x0F70);
  }

  // ------------------------------------------------------------------ epilogue
  const int srow = wm * 128 + (lane & 31);
  const int scol = wn * 32 * FN + (lane >> 5) * 4;
  if constexpr (OUT_BF16) {
    __syncthreads();   // every wavefront done with the ring
    constexpr int kStLd = (int)f8_epi_row(FN);
    unsigned char* stg = smem_f8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const u32x2_t pk = {bf16x2_rne(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                              bf16x2_rne(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
          *reinterpret_cast<u32x2_t*>(stg + (srow + 32 * i) * kStLd + 2 * (scol + j * 32 + 8 * q)) = pk;
        }
    __syncthreads();
    constexpr int CPR = 2 * BN / 16;   // 16-byte pieces of a tile row
    uint16_t* cb = static_cast<uint16_t*>(c) + m0 * ldc + n0;
    const bool st_vec = (ldc % 8 == 0) && ((reinterpret_cast<uintptr_t>(c) & 15) == 0);
#pragma unroll 4
    for (int it = 0; it < BM * CPR / kF8Threads; ++it) {
      const int cidx = t + kF8Threads * it;
      const int r = cidx / CPR, cc = cidx - r * CPR;
      if (r >= rows_here) continue;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stg + r * kStLd + cc * 16);
      uint16_t* dst = cb + (int64_t)r * ldc + cc * 8;
      if (st_vec && cc * 8 + 8 <= cols_here) {
        store_stream(v, reinterpret_cast<u32x4_t*>(dst));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (cc * 8 + e < cols_here) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      }
    }
  } else {
    const bool vec = rows_here == BM && cols_here == BN && (ldc % 4 == 0) &&
                     ((reinterpret_cast<uintptr_t>(c) & 15) == 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = srow + 32 * i;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int cl = scol + j * 32 + 8 * q;
          float* dst = static_cast<float*>(c) + (m0 + r) * ldc + n0 + cl;
          const f32x4_t y = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                             acc[i][j][4 * q + 3]};
          if (vec) {
            store_out(y, reinterpret_cast<f32x4_t*>(dst));
          } else if (r < rows_here) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (cl + e < cols_here) dst[e] = y[e];
          }
        }
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: 16 columns (rows of b) and 16 MF rows of a to a workgroup of eight
// wavefronts that divide the blocks among them; a wavefront's operands come
// straight to registers (a block of a row: 32 bytes a lane), and the partial
// sums meet in LDS.
// ---------------------------------------------------------------------------
constexpr int kSkinnyWaves = 8;

template <int MF, bool OUT_BF16>
__global__ __launch_bounds__(64 * kSkinnyWaves) void k_gemm_f8_skinny(
    Fp8Operand A, Fp8Operand B, int64_t m, int64_t n, int k_blocks, const int64_t* offs, int nseg,
    void* c, int64_t ldc) {
  __shared__ float part[kSkinnyWaves][16][16 * MF + 4];   // [..][column][row]
  int64_t m0 = (int64_t)blockIdx.y * 16 * MF, m_end = m, boff = 0;
  if (offs) {
    const SegRange sr = locate_chunk(offs, nseg, m, 16 * MF, blockIdx.y);
    if (sr.seg < 0) return;
    m0 = sr.r0;
    m_end = sr.r1;
    boff = (int64_t)sr.seg * n;
  }
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int rows_here = (int)(m_end - m0 < 16 * MF ? m_end - m0 : 16 * MF);
  const int cols_here = (int)(n - n0 < 16 ? n - n0 : 16);
  // rows past the edge repeat the last one (their products are never stored)
  const int64_t br = boff + n0 + (r < cols_here ? r : cols_here - 1);
  const uint8_t* bc = B.codes + br * B.pitch + 32 * g;
  const uint8_t* bs = B.scales + br * B.spitch;
  const uint8_t *ac[MF], *as[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t ar = m0 + (16 * i + r < rows_here ? 16 * i + r : rows_here - 1);
    ac[i] = A.codes + ar * A.pitch + 32 * g;
    as[i] = A.scales + ar * A.spitch;
  }
  f32x4_t acc[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int kb0 = k_blocks * w / kSkinnyWaves, kb1 = k_blocks * (w + 1) / kSkinnyWaves;
  for (int kb = kb0; kb < kb1; ++kb) {
    const int64_t k = (int64_t)kb * 128;
    const i32x8_t bf = frag(*reinterpret_cast<const u32x4_t*>(bc + k),
                            *reinterpret_cast<const u32x4_t*>(bc + k + 16));
    const int sb = bs[kb];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      const i32x8_t af = frag(*reinterpret_cast<const u32x4_t*>(ac[i] + k),
                              *reinterpret_cast<const u32x4_t*>(ac[i] + k + 16));
      acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf, af, acc[i], 0, 0, 0, sb, 0,
                                                                (int)as[i][kb]);
    }
  }
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) part[w][4 * g + v][16 * i + r] = acc[i][v];
  __syncthreads();
  for (int e = threadIdx.x; e < 256 * MF; e += 64 * kSkinnyWaves) {
    const int col = e & 15, row = e >> 4;
    if (row >= rows_here || col >= cols_here) continue;
    float s = part[0][col][row];
#pragma unroll
    for (int q = 1; q < kSkinnyWaves; ++q) s += part[q][col][row];
    const int64_t o = (m0 + row) * ldc + n0 + col;
    if constexpr (OUT_BF16)
      static_cast<uint16_t*>(c)[o] = (uint16_t)bf16x2_rne(s, 0.0f);
    else
      static_cast<float*>(c)[o] = s;
  }
}

// sums the splits' fp32 partials in order
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void k_f8_reduce(const float* __restrict__ part, int splits,
                                                   int64_t m, int64_t n, void* c, int64_t ldc) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int64_t mn = m * n;
  if (e >= mn) return;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool whole = e + 4 <= mn && (mn & 3) == 0;   // every split's part 16-byte aligned
  for (int z = 0; z < splits; ++z) {
    const float* p = part + z * mn + e;
    if (whole) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e + i < mn) s[i] += p[i];
    }
  }
  const int64_t row = e / n, col = e - row * n;
  if (OUT_BF16 && whole && col + 4 <= n && ldc % 4 == 0 && (n & 3) == 0 &&
      (reinterpret_cast<uintptr_t>(c) & 7) == 0) {
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(c) + row * ldc + col) =
        u32x2_t{bf16x2_rne(s[0], s[1]), bf16x2_rne(s[2], s[3])};
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (e + i >= mn) break;
    const int64_t rr = (e + i) / n, cc = (e + i) - rr * n;
    if constexpr (OUT_BF16)
      static_cast<uint16_t*>(c)[rr * ldc + cc] = (uint16_t)bf16x2_rne(s[i], 0.0f);
    else
      static_cast<float*>(c)[rr * ldc + cc] = s[i];
  }
}

// ---------------------------------------------------------------------------
// What runs a product
// ---------------------------------------------------------------------------
struct Fp8Plan {
  int skinny;   // 16-row fragments of the few-rows kernel, 0: the tiled one
  int fn;       // tile width / 64
  int splits;   // of the blocks
};

Fp8Plan fp8_plan(int64_t m, int64_t n, int64_t k_blocks, Fp8Mode mode, int nseg) {
  Fp8Plan p{0, 4, 1};
  if (mode != kF8BlockSegs) {
    const int64_t avg = mode == kF8RowSegs ? (m + nseg - 1) / nseg : m;
    if (avg <= 64) {
      p.skinny = avg <= 16 ? 1 : avg <= 32 ? 2 : 4;
      return p;
    }
  }
  const int64_t tm = mode == kF8RowSegs ? chunk_upper_bound(m, nseg, kF8BM) : (m + kF8BM - 1) / kF8BM;
  auto tiles = [&](int fn) {
    return tm * ((n + 64 * fn - 1) / (64 * fn)) * (mode == kF8BlockSegs ? nseg : 1);
  };
  // the wider tile unless the narrower one needs less time in rounds of 256
  const int64_t c4 = (tiles(4) + 255) / 256 * 4, c2 = (tiles(2) + 255) / 256 * 2;
  if (c2 < c4) p.fn = 2;
  if (mode == kF8All) {
    const int64_t tl = tiles(p.fn);
    while (p.splits < 16 && tl * p.splits * 2 <= 256 && k_blocks / (p.splits * 2) >= 4) p.splits *= 2;
  }
  return p;
}

template <int FN, bool OB>
hipError_t gemm_f8_t(const Fp8Gemm& g, int splits, void* c, int64_t ldc, int64_t c_split,
                     hipStream_t st) {
  constexpr size_t lds = f8_lds_bytes(FN);
  static_assert(lds + 64 <= 160 * 1024, "fits one CU's LDS");
  const hipError_t e = lds_attr_once<&k_gemm_f8<FN, OB>>((int)lds);
  if (e != hipSuccess) return e;
  const int64_t tm = g.mode == kF8RowSegs ? chunk_upper_bound(g.m, g.nseg, kF8BM)
                                          : (g.m + kF8BM - 1) / kF8BM;
  const dim3 grid((unsigned)((g.n + 64 * FN - 1) / (64 * FN)), (unsigned)tm,
                  (unsigned)(g.mode == kF8BlockSegs ? g.nseg : splits));
  k_gemm_f8<FN, OB><<<grid, kF8Threads, lds, st>>>(g.a, g.b, g.m, g.n, (int)g.k_blocks, g.mode,
                                                   g.offs, g.nseg, g.rows, c, ldc, c_split);
  return hipGetLastError();
}

template <int MF>
hipError_t skinny_t(const Fp8Gemm& g, hipStream_t st) {
  const dim3 grid((unsigned)((g.n + 15) / 16),
                  (unsigned)chunk_upper_bound(g.m, g.offs ? g.nseg : 1, 16 * MF));
  if (g.c_bf16)
    k_gemm_f8_skinny<MF, true><<<grid, 64 * kSkinnyWaves, 0, st>>>(
        g.a, g.b, g.m, g.n, (int)g.k_blocks, g.offs, g.nseg, g.c, g.ldc);
  else
    k_gemm_f8_skinny<MF, false><<<grid, 64 * kSkinnyWaves, 0, st>>>(
        g.a, g.b, g.m, g.n, (int)g.k_blocks, g.offs, g.nseg, g.c, g.ldc);
  return hipGetLastError();
}

}  // namespace

size_t fp8_gemm_ws_bytes(int64_t m, int64_t n, int64_t k_blocks, Fp8Mode mode, int nseg) {
  const Fp8Plan p = fp8_plan(m, n, k_blocks, mode, nseg);
  return p.splits > 1 ? ((size_t)p.splits * m * n * 4 + 255) & ~(size_t)255 : 0;
}

hipError_t launch_fp8_gemm(const Fp8Gemm& g, void* ws, hipStream_t st) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  const Fp8Plan p = fp8_plan(g.m, g.n, g.k_blocks, g.mode, g.nseg);
  if (p.skinny == 1) return skinny_t<1>(g, st);
  if (p.skinny == 2) return skinny_t<2>(g, st);
  if (p.skinny == 4) return skinny_t<4>(g, st);
  if (p.splits > 1) {
    hipError_t e = p.fn == 4 ? gemm_f8_t<4, false>(g, p.splits, ws, g.n, g.m * g.n, st)
                             : gemm_f8_t<2, false>(g, p.splits, ws, g.n, g.m * g.n, st);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((g.m * g.n + 1023) / 1024));
    if (g.c_bf16)
      k_f8_reduce<true><<<grid, 256, 0, st>>>(static_cast<const float*>(ws), p.splits, g.m, g.n, g.c, g.ldc);
    else
      k_f8_reduce<false><<<grid, 256, 0, st>>>(static_cast<const float*>(ws), p.splits, g.m, g.n, g.c, g.ldc);
    return hipGetLastError();
  }
  const int64_t cs = g.mode == kF8BlockSegs ? g.m * g.ldc : 0;
  if (g.c_bf16)
    return p.fn == 4 ? gemm_f8_t<4, true>(g, 1, g.c, g.ldc, cs, st)
                     : gemm_f8_t<2, true>(g, 1, g.c, g.ldc, cs, st);
  return p.fn == 4 ? gemm_f8_t<4, false>(g, 1, g.c, g.ldc, cs, st)
                   : gemm_f8_t<2, false>(g, 1, g.c, g.ldc, cs, st);
}

}  // namespace averis
