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
// random operands, 1.2e-5 to 1.5e-5 of the result's norm in fp32 output (a sum
// in fp32 alone: 1e-7).  In bf16 output it moves one rounding in 90 to the
// neighbour, 2.3e-4 of the norm, beside the 1.66e-3 of bf16's rounding itself.
// A choice taken with the format, whose own rounding is 2^-4 of each operand,
// for the instruction's rate (twice that of bf16).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "activation.hpp"
#include "fp8_eight.hpp"
#include "launch.hpp"
#include "segments.hpp"

namespace averis {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kF8Threads = 256;   // four wavefronts, 2 x 2 over the tile
constexpr int kF8Cus = 256;       // CUs of the card: one workgroup each

// two slots of a stage's codes (128 bytes a row), two of scale words (four
// stages, 4 bytes a row), and 4 KB a wavefront for its output (in the small
// tile, two of which fill a CU's LDS, in the second slot)
constexpr int kF8Stage = 4096;
constexpr size_t f8_lds_bytes(int f) {
  return (size_t)(2 * 64 * f) * (2 * 128 + 2 * 4) + (f == 4 ? 4 * kF8Stage : 0);
}

template <int V>
struct F8Step {
  static constexpr int value = V;
};

__device__ __forceinline__ i32x8_t frag(u32x4_t a, u32x4_t b) {
  return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// f(F8Step<0>), .., f(F8Step<N - 1>)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each_step(F f) {
  if constexpr (I < N) {
    f(F8Step<I>{});
    each_step<N, I + 1>(f);
  }
}

// items [p N / P, (p + 1) N / P) go with step p of P: the step of item k
template <int N, int P>
constexpr int step_of(int k) {
  int p = 0;
  while ((p + 1) * N / P <= k) ++p;
  return p;
}

// s_waitcnt vmcnt(N) (vmcnt in bits 3:0 and 15:14; the others not waited for)
template <int N>
__device__ __forceinline__ void f8_wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// One output tile: rows m0 .. m0 + rows - 1, columns n0 .. n0 + cols - 1 and
// the blocks kb0 .. kb0 + nk - 1 it contracts (all uniform).
struct F8Tile {
  int m0, n0, seg;   // seg: matrix of a stacked b, or plane of c
  int rows, cols, kb0, nk;
};

// ---------------------------------------------------------------------------
// Epilogues
// ---------------------------------------------------------------------------
// kinds of them in the tiled kernel: each code of its own, for the instruction cache's sake
constexpr int kEpiNone = 0, kEpiPlain = 1, kEpiResidual = 2;
struct NoEpilogue {};
template <bool EPI>
using EpilogueArg = std::conditional_t<EPI, Fp8Epilogue, NoEpilogue>;

// at element alignment, as f8_piece_t
typedef u32x2_t f8_half_piece_t __attribute__((aligned(2)));
template <bool BF16>
using Four = std::conditional_t<BF16, u32x2_t, u32x4_t>;

// elements at .. at + 3 of p, the first `left` of them (the others 0)
template <bool BF16>
__device__ __forceinline__ Four<BF16> four_in(const void* p, int64_t at, int left) {
  Four<BF16> v = {};
  if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if (left >= 4) return *reinterpret_cast<const f8_half_piece_t*>(q);
#pragma unroll
    for (int x = 0; x < 3; ++x)
      if (x < left) v[x / 2] |= (uint32_t)q[x] << (16 * (x & 1));
  } else {
    const uint32_t* q = static_cast<const uint32_t*>(p) + at;
    if (left >= 4) return *reinterpret_cast<const f8_piece_t*>(q);
#pragma unroll
    for (int x = 0; x < 3; ++x)
      if (x < left) v[x] = q[x];
  }
  return v;
}
__device__ __forceinline__ float vector_at(const void* p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16)
              : static_cast<const float*>(p)[i];
}
// z and the residual in whole pieces of 16 bytes below 2^31 bytes a tile
__host__ __device__ __forceinline__ bool epilogue_whole(const Fp8Epilogue& e, int es) {
  auto ok = [&](const void* p, int64_t ld) {
    return !p || (ld * es % 16 == 0 && ld <= (1 << 21) && (reinterpret_cast<uintptr_t>(p) & 15) == 0);
  };
  return ok(e.z, e.ldz) && ok(e.res, e.ldr);
}
template <bool BF16>
__device__ __forceinline__ f32x4_t four_f32(Four<BF16> v) {
  if constexpr (BF16)
    return f32x4_t{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u),
                   __uint_as_float(v[1] << 16), __uint_as_float(v[1] & 0xFFFF0000u)};
  else
    return __builtin_bit_cast(f32x4_t, v);
}
// 16 bytes to elements of a row of which `left` are there
template <bool BF16>
__device__ __forceinline__ void piece_out(char* dst, u32x4_t v, int left) {
  if (left >= (BF16 ? 8 : 4)) {
    *reinterpret_cast<f8_piece_t*>(dst) = v;
    return;
  }
#pragma unroll
  for (int x = 0; x < (BF16 ? 8 : 4); ++x) {
    if (x >= left) continue;
    if constexpr (BF16)
      reinterpret_cast<uint16_t*>(dst)[x] = (uint16_t)(v[x / 2] >> (16 * (x & 1)));
    else
      reinterpret_cast<uint32_t*>(dst)[x] = v[x];
  }
}

__device__ __forceinline__ float activated(float z, int act) {
  if (act == kActNone) return z;
  if (act == kActRelu) return z < 0.0f ? 0.0f : z;
  return act == kActSilu ? act_silu(z) : act_gelu(z);
}
template <int N>
__device__ __forceinline__ void activate(f32x4_t (&v)[N][4], int act) {
  auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 16 * N; ++i) v[i / 16][i / 4 % 4][i % 4] = f(v[i / 16][i / 4 % 4][i % 4]);
  };
  if (act == kActGelu) each([](float z) { return act_gelu(z); });
  else if (act == kActSilu) each([](float z) { return act_silu(z); });
  else if (act == kActRelu) each([](float z) { return z < 0.0f ? 0.0f : z; });   // (a NaN stays)
}

// the epilogue of one value: row, column of c, column j of the bias
template <bool OUT_BF16>
__device__ __forceinline__ void epilogue_one(const Fp8Epilogue& e, void* c, int64_t ldc, int64_t row,
                                             int64_t col, int64_t j, float s) {
  auto out = [](void* p, int64_t at, float v) {
    if constexpr (OUT_BF16) static_cast<uint16_t*>(p)[at] = (uint16_t)bf16x2_rne(v, 0.0f);
    else static_cast<float*>(p)[at] = v;
  };
  if (e.bias) s += vector_at(e.bias, e.bias_bf16, j);
  if (e.z) out(e.z, row * e.ldz + col, s);
  s = activated(s, e.act);
  if (e.res) s += vector_at(e.res, OUT_BF16, row * e.ldr + col);
  out(c, row * ldc + col, s);
}

// ---------------------------------------------------------------------------
// The tiled kernel: 64 F x 64 F outputs a tile, each of four wavefronts 32 F x
// 32 F of them (F x F accumulators of 32 x 32): F = 4, one workgroup a CU, or 2
// (128 x 128), two.
//
// A stage is one block of 128 k: two k-steps of 64.  Its codes come straight
// from memory to LDS (16 bytes a lane, eight lanes to a row, the row's pieces
// in the order piece ^ (row / 2 mod 8): sixteen rows' reads of a piece go to
// sixteen places, and the counter of bank conflicts stays at 0; by row mod 8 it
// was 0.46 of the LDS cycles, at the same speed).  Two slots: stage s computes
// k-step 0 from registers while it reads k-step 1's fragments; then (its slot
// read out, stage s + 1 landed) one barrier; then k-step 1 while stage s + 2 is
// loaded into the slot and stage s + 1's first fragments are read.  Per MFMA
// one LDS read and one load, the order held by a scheduling barrier after each.
// Scale bytes come four stages at a time, one aligned word a row, the same way.
//
// A workgroup takes several tiles (block segments, of very different lengths:
// one, the longest segments' first).  The barrier inside a tile's last stage
// frees both slots, so the next tile's first two stages are on their way
// before this tile's output is; the output goes through 4 KB of LDS of the
// wavefront's own (no barrier) to whole 128-byte lines, and its stores drain
// under the next tile's products (the waits of the first stage count them).
//
// Bound by the matrix pipes' power on large products: 8192^3 395 us (2.78
// PFLOP/s; the instruction alone, from registers, 3.26 on random operands),
// 16384 x 1024 x 3072 45 us (2.3); by the output of each round of tiles where K
// is short (16384 x 3072 x 1024 57 us, 1.8: 9 us of products, 7 of the rest a
// round); and by memory by expert segments (32768 rows in 64 segments, 768 x
// 2048: 62 us with its operands in the last-level cache, 77 without).
// Four slots of 64 k instead of two of 128, loads twice as far ahead: 10 %
// slower on large products (half lines a load, a barrier more a block) and no
// faster where the operands come from memory.
// ---------------------------------------------------------------------------
template <int F, bool OUT_BF16, int MODE, int EPI>
__global__ __launch_bounds__(kF8Threads, F == 4 ? 1 : 2) void k_gemm_f8(
    Fp8Operand A, Fp8Operand B, int m, int n, int k_blocks, const int64_t* offs, int nseg,
    int64_t seg_rows, int splits, int tx, int ty, void* c, int64_t ldc, int64_t c_split,
    EpilogueArg<EPI != kEpiNone> epi) {
  constexpr bool RES = EPI == kEpiResidual;
  constexpr bool MANY = MODE != kF8BlockSegs;   // several tiles a workgroup
  constexpr int SLOTS = F == 4 ? kF8Cus : 2 * kF8Cus;   // workgroups the card holds
  constexpr int BM = 64 * F, BN = 64 * F, ROWS = BM + BN;
  constexpr int SLOT = ROWS * 128, SSLOT = ROWS * 4;
  constexpr int CPW = ROWS / 8 / 4;    // code loads a wavefront issues for a stage
  constexpr int SPW = ROWS / 64 / 4;   // scale loads for four stages
  static_assert(SPW * 256 == ROWS, "every wavefront's loads are whole");
  constexpr int NF = 2 * F;
  constexpr int ES = OUT_BF16 ? 2 : 4;
  constexpr int GROUP = 128 / ES;      // columns of an output pass: 128 bytes
  constexpr int PASSES = (32 * F + GROUP - 1) / GROUP;   // of a 32-row fragment
  extern __shared__ __attribute__((aligned(16))) unsigned char smem_f8[];
  unsigned char* ring = smem_f8;
  unsigned char* sring = smem_f8 + 2 * SLOT;

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  // output: 4 KB in rows of 128 bytes, eight rows every STG_STEP: the
  // wavefront's own, or the part of the second slot that its last HELD loads
  // of a stage fill
  constexpr int HELD = F == 4 ? 0 : 4, STG_STEP = F == 4 ? 1024 : 4096;
  unsigned char* stg = F == 4 ? smem_f8 + 2 * SLOT + 2 * SSLOT + wave * kF8Stage
                              : smem_f8 + SLOT + (wave + 4 * (CPW - HELD)) * 1024;

  SegTable segs;
  if constexpr (MODE == kF8RowSegs) segs.init(offs, nseg, m, BM);
  if constexpr (MODE == kF8BlockSegs) segs.init(offs, nseg, seg_rows, 128);

  // Tiles are numbered plane by plane (split or segment), within a plane by
  // groups of four tile rows, column by column.  Workgroup w runs on die w
  // mod 8; with a workgroup a CU each die takes an eighth of the numbers, its
  // workgroups side by side, so the tiles a die runs together share operand
  // rows in its L2.  With a workgroup a tile (fewer tiles than the card holds,
  // or block segments, left to the dispatcher) that is done plane by plane.
  if constexpr (MODE == kF8RowSegs) ty = segs.count();   // the grid is for as many as there may be
  const int txy = tx * ty, total = txy * (MODE == kF8BlockSegs ? nseg : splits);
  const int w = blockIdx.x, grid = gridDim.x;
  int id, id_end, id_step;
  if (MANY && grid == SLOTS) {
    const int x = w % kXcds, per = SLOTS / kXcds;
    id = total / kXcds * x + total % kXcds * x / kXcds + w / kXcds;
    id_end = total / kXcds * (x + 1) + total % kXcds * (x + 1) / kXcds;
    id_step = per;
  } else {
    if (w >= total) return;
    const int z = w / txy, r = w - z * txy, even = txy - txy % kXcds;
    id = z * txy + (r < even ? (r % kXcds) * (even / kXcds) + r / kXcds : r);
    id_end = id + 1;
    id_step = 1;
  }

  // the next tile with rows, from number id on; false: none
  auto next_tile = [&](F8Tile& tl) __attribute__((always_inline)) -> bool {
    for (; id < id_end; id += id_step) {
      const int z = id / txy, r = id - z * txy;
      const int g = r / (4 * tx), rr = r - g * 4 * tx;
      const int gm = ty - 4 * g < 4 ? ty - 4 * g : 4;
      const int x = rr / gm, y = 4 * g + (rr - x * gm);
      tl.n0 = x * BN;
      tl.cols = n - tl.n0 < BN ? n - tl.n0 : BN;
      tl.m0 = y * BM;
      int m_end = m;
      tl.seg = z;
      tl.kb0 = 0;
      tl.nk = k_blocks;
      if constexpr (MODE == kF8RowSegs) {
        if (!segs.chunk(y, tl.seg, tl.m0, m_end)) continue;
      } else if constexpr (MODE == kF8BlockSegs) {
        int kb1;
        tl.seg = segs.by_length(z);
        segs.segment(tl.seg, tl.kb0, kb1);
        // within the operands whatever the offsets hold
        kb1 = kb1 < k_blocks ? kb1 : k_blocks;
        tl.kb0 = tl.kb0 < kb1 ? tl.kb0 : kb1;
        tl.nk = kb1 - tl.kb0;
      } else {
        // (k_blocks < 2^23, splits <= 16)
        tl.kb0 = k_blocks * z / splits;
        tl.nk = k_blocks * (z + 1) / splits - tl.kb0;
      }
      tl.rows = m_end - tl.m0 < BM ? m_end - tl.m0 : BM;
      // the quotients come from vector registers: back to scalar ones, which
      // every base address below then stays in
      tl.m0 = __builtin_amdgcn_readfirstlane(tl.m0);
      tl.n0 = __builtin_amdgcn_readfirstlane(tl.n0);
      tl.seg = __builtin_amdgcn_readfirstlane(tl.seg);
      tl.rows = __builtin_amdgcn_readfirstlane(tl.rows);
      tl.cols = __builtin_amdgcn_readfirstlane(tl.cols);
      tl.kb0 = __builtin_amdgcn_readfirstlane(tl.kb0);
      tl.nk = __builtin_amdgcn_readfirstlane(tl.nk);
      id += id_step;
      return true;
    }
    return false;
  };

  // what the loads of a tile go by
  const uint8_t *a_c, *b_c, *a_s, *b_s;
  uint32_t cofs[CPW], sofs[SPW];
  int ph, g_last;
  auto set_tile = [&](const F8Tile& tl) __attribute__((always_inline)) {
    const int64_t brow = (MODE == kF8RowSegs ? (int64_t)tl.seg * n : 0) + tl.n0;
    a_c = A.codes + tl.m0 * A.pitch + (int64_t)tl.kb0 * 128;
    b_c = B.codes + brow * B.pitch + (int64_t)tl.kb0 * 128;
    // word g of a row: its stages 4 g .. 4 g + 3 counted from kb0 rounded down
    ph = tl.kb0 & 3;
    a_s = A.scales + tl.m0 * A.spitch + (tl.kb0 - ph);
    b_s = B.scales + brow * B.spitch + (tl.kb0 - ph);
    g_last = (ph + tl.nk - 1) >> 2;
    // code load j: rows 8 j .. 8 j + 7 of the tile's A rows, then B rows; rows
    // past the edge repeat the last one (their products are never stored)
    const uint32_t ap = (uint32_t)A.pitch, bp = (uint32_t)B.pitch;
    const uint32_t row = 8 * wave + (lane >> 3), piece = 16u * (uint32_t)((lane & 7) ^ (4 * (wave & 1) + (lane >> 4)));
    const uint32_t a_last = (uint32_t)(tl.rows - 1) * ap, b_last = (uint32_t)(tl.cols - 1) * bp;
#pragma unroll
    for (int q = 0; q < CPW; ++q) {
      const bool isa = q < BM / 32;   // exactly when 8 j < BM
      const uint32_t o = isa ? row * ap + q * 32 * ap : row * bp + (q - BM / 32) * 32 * bp;
      const uint32_t last = isa ? a_last : b_last;
      cofs[q] = (o < last ? o : last) + piece;
    }
#pragma unroll
    for (int q = 0; q < SPW; ++q) {
      const int i = wave + 4 * q;
      const bool isa = 64 * i < BM;
      const int r = (isa ? 64 * i : 64 * i - BM) + lane;
      const int lim = isa ? tl.rows : tl.cols;
      sofs[q] = (uint32_t)(r < lim ? r : lim - 1) * (uint32_t)(isa ? A.spitch : B.spitch);
    }
  };
  // where stage s's codes start, in scalar registers (a load then takes base and
  // offset as they are, with no address arithmetic a lane)
  auto scalar_base = [&](const uint8_t* p) __attribute__((always_inline)) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t*>(((uint64_t)hi << 32) | lo);
  };
  auto stage_base = [&](const uint8_t* p, int s) __attribute__((always_inline)) {
    return scalar_base(p + 128 * (int64_t)s);
  };
  // the wavefront's code load q of the stage that starts at ab, bb
  auto load_code = [&](const uint8_t* ab, const uint8_t* bb, int slot, int q) __attribute__((always_inline)) {
    __builtin_amdgcn_global_load_lds((const void*)((q < BM / 32 ? ab : bb) + cofs[q]),
                                     (lds_void*)(ring + slot * SLOT + (wave + 4 * q) * 1024), 16, 0, 0);
  };
  // the wavefront's scale load q of word g
  auto load_scale = [&](int g, int q) __attribute__((always_inline)) {
    const int gl = g < g_last ? g : g_last;
    const uint8_t* base = scalar_base((64 * (wave + 4 * q) < BM ? a_s : b_s) + 4 * (int64_t)gl);
    __builtin_amdgcn_global_load_lds((const void*)(base + sofs[q]),
                                     (lds_void*)(sring + (g & 1) * SSLOT + (wave + 4 * q) * 256), 4, 0, 0);
  };
  auto load_scales = [&](int g) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < SPW; ++q) load_scale(g, q);
  };
  // the first loads of a tile of nk stages, one by one: two words of scales,
  // stage 0, stage 1
  constexpr int FIRST0 = 2 * SPW + CPW, FIRST = FIRST0 + CPW;
  auto first_load = [&](int k, int nk) __attribute__((always_inline)) {
    if (k < 2 * SPW) {
      load_scale(k / SPW, k % SPW);
    } else {
      const int s = k < FIRST0 ? 0 : 1, q = k - (s ? FIRST0 : 2 * SPW), st = s < nk ? s : 0;
      load_code(stage_base(a_c, st), stage_base(b_c, st), s, q);
    }
  };
  auto first_loads = [&](int nk) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < FIRST; ++k) first_load(k, nk);
  };

  f32x16_t acc[F][F];
  const int lrow = lane & 31, lh = lane >> 5;
  auto row_of = [&](int f) { return f < F ? wm * 32 * F + 32 * f : BM + wn * 32 * F + 32 * (f - F); };
  i32x8_t fr[2][NF];
  // half x of fragment f of k-step js (lane half h: piece 4 js + 2 h + x)
  auto read_half = [&](int slot, int js, int f, int x) __attribute__((always_inline)) {
    const int piece = 16 * ((4 * js + 2 * lh + x) ^ ((lane >> 1) & 7));
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(ring + slot * SLOT + (row_of(f) + lrow) * 128 + piece);
#pragma unroll
    for (int e = 0; e < 4; ++e) fr[js][f][4 * x + e] = (int)v[e];
  };
  auto read_step = [&](int slot, int js) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      read_half(slot, js, f, 0);
      read_half(slot, js, f, 1);
    }
  };
  uint32_t words[NF];
  auto read_words = [&](int g) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < NF; ++f)
      words[f] = *reinterpret_cast<const uint32_t*>(sring + (g & 1) * SSLOT + (row_of(f) + lrow) * 4);
  };
  int sc[NF];
  // A k-step's products one by one, each with its share of what runs beside
  // them: the reads of the other k-step's fragments from slot rslot (READ), and
  // stage ls's loads into slot lslot (LOAD).  Loads keep the path from the
  // cache to LDS busy for 16 cycles each, 64 of them a stage: issued in a row
  // they would hold up the products behind them.  B's fragment goes first: a
  // lane then holds four consecutive columns of a row.
  auto k_step = [&](auto jc, auto readc, int rslot, auto loadc, int ls, int lslot) __attribute__((always_inline)) {
    constexpr int js = decltype(jc)::value, N = F * F;
    const uint8_t *ab = nullptr, *bb = nullptr;
    if constexpr (decltype(loadc)::value != 0) {
      ab = stage_base(a_c, ls);
      bb = stage_base(b_c, ls);
    }
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int i = x / F, j = x % F;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          fr[js][F + j], fr[js][i], acc[i][j], 0, 0, 0, sc[F + j], 0, sc[i]);
      if constexpr (decltype(loadc)::value != 0) {
#pragma unroll
        for (int q = x * CPW / N; q < (x + 1) * CPW / N; ++q) load_code(ab, bb, lslot, q);
      }
      if constexpr (decltype(readc)::value != 0) {
#pragma unroll
        for (int r = x * 2 * NF / N; r < (x + 1) * 2 * NF / N; ++r) read_half(rslot, js ^ 1, r / 2, r % 2);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // a barrier without a fence (which would wait for every load in flight)
  auto barrier = []() __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  constexpr F8Step<0> step0{};
  constexpr F8Step<1> step1{};
  // The loads of stage 0 (later: of stage 1) landed.  A whole tile's output
  // passes each issue a share of them and then four stores: behind them are
  // the stores of the pass that issued the last one and all that followed.
  constexpr int OUT_PASSES = F * PASSES;
  constexpr int AFTER0 = CPW + 4 * (OUT_PASSES - step_of<FIRST - HELD, OUT_PASSES>(FIRST0 - 1));
  static_assert(HELD > 0 || step_of<FIRST, OUT_PASSES>(FIRST - 1) == OUT_PASSES - 1,
                "stage 1's last load is the last pass's");
  bool behind = false;   // the first loads went out with a whole tile's output
  auto wait_loads = [&](auto firstc) __attribute__((always_inline)) {
    // (the small tile's epilogue has four stores a pass at least behind them and four
    // behind the HELD of stage 1, the large one's stage 1 itself behind stage 0)
    if (behind)
      f8_wait_vm<(decltype(firstc)::value != 0 ? (!EPI ? AFTER0 : F == 4 ? CPW : 4 * OUT_PASSES)
                  : EPI && F == 4              ? 0 : 4)>();
    else f8_wait_vm<0>();
  };
  // stage s in slot s & 1; on entry its first fragments and scale words are
  // in registers.  NEXT: there is a stage s + 1; LOAD: a stage s + 2.
  auto stage = [&](int s, auto nextc, auto loadc) __attribute__((always_inline)) {
    constexpr bool NEXT = decltype(nextc)::value != 0;
    const int slot = s & 1, q = s + ph;
#pragma unroll
    for (int f = 0; f < NF; ++f) sc[f] = (int)(words[f] >> (8 * (q & 3)));
    __builtin_amdgcn_sched_barrier(0);
    k_step(step0, step1, slot, step0, 0, 0);
    // this slot read out and stage s + 1 landed, for every wavefront
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
    wait_loads(step0);
    behind = false;
    barrier();
    if constexpr (NEXT) {
      if ((q & 3) == 0) load_scales((q >> 2) + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (NEXT) read_words((q + 1) >> 2);
    k_step(step1, nextc, slot ^ 1, loadc, s + 2, slot);
  };
  auto zero = [&](int i, int j) __attribute__((always_inline)) {
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  };

  F8Tile cur;
  if (!next_tile(cur)) return;
  if (cur.nk > 0) {
    set_tile(cur);
    first_loads(cur.nk);
  }
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) zero(i, j);
  while (true) {
    const int nk = cur.nk;
    if (nk > 0) {
      wait_loads(step1);
      barrier();
      read_words(0);
      read_step(0, 0);
      int s = 0;
      for (; s + 2 < nk; ++s) stage(s, step1, step1);
      if (s + 1 < nk) stage(s++, step1, step0);
      stage(s, step0, step0);
      mfma_drain();
    }
    F8Tile nxt;
    const bool more = MANY && next_tile(nxt), loads = more && nxt.nk > 0;
    __builtin_amdgcn_sched_barrier(0);
    if (loads) set_tile(nxt);
    __builtin_amdgcn_sched_barrier(0);

    // ---------------------------------------------------------------- output
    // In passes of 32 rows x 128 bytes.  A lane holds four consecutive columns
    // of a row, lane + 32 the next four; for bf16 the halves swap so that each
    // has eight (16 bytes).  To LDS (row r's 16-byte piece p at p ^ (r mod 8):
    // no bank twice), back eight lanes to a row, and out.  A pass's values are
    // formed while the one before comes back from LDS.  The LDS writes are
    // asm: the compiler would wait for every load to LDS in flight before a
    // write of its own.  A wavefront's LDS accesses are in order.
    char* cb = static_cast<char*>(c) +
               ((MODE == kF8RowSegs ? 0 : cur.seg * c_split) + cur.m0 * ldc + cur.n0) * ES;
    // whole pieces: stores through a descriptor of the tile's bytes, which
    // drops those past its rows and columns and counts them all the same
    const bool pieces = (ldc * ES) % 16 == 0 && (c_split * ES) % 16 == 0 && ldc <= (1 << 21) &&
                        (reinterpret_cast<uintptr_t>(c) & 15) == 0 && cur.cols * ES % 16 == 0;
    // the lane's places are formed anew for each tile: kept over the products
    // they would not fit the registers
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const uint32_t wr = (uint32_t)(uintptr_t)(lds_void*)stg + ((ln & 31) >> 3) * STG_STEP +
                        (ln & 7) * 128 + 16 * ((ln & 7) ^ (ln >> 5));   // piece h; piece p + h at ^ 16 p
    const unsigned char* src = stg + (ln >> 3) * 128 + 16 * ((ln & 7) ^ (ln >> 3));
    constexpr int FPP = GROUP / 32;   // fragments of a pass
    static_assert(F % FPP == 0, "whole passes");
    u32x4_t out[4];   // a bf16 pass's values: pieces of two fragments
    auto form = [&](auto pc) __attribute__((always_inline)) {
      constexpr int i = decltype(pc)::value / PASSES, p = decltype(pc)::value % PASSES;
      if constexpr (OUT_BF16) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          // fragment u / 2, column groups 8 q and 8 q + 8, q = 2 (u mod 2)
          const f32x16_t& y = acc[i][p * FPP + u / 2];
          const int q = 8 * (u & 1);
          const auto a = __builtin_amdgcn_permlane32_swap(bf16x2_rne(y[q], y[q + 1]),
                                                          bf16x2_rne(y[q + 4], y[q + 5]), false, false);
          const auto b = __builtin_amdgcn_permlane32_swap(bf16x2_rne(y[q + 2], y[q + 3]),
                                                          bf16x2_rne(y[q + 6], y[q + 7]), false, false);
          out[u] = u32x4_t{a[0], b[0], a[1], b[1]};
        }
      }
    };
    // pieces 2 u + h; fp32 straight from the accumulation registers
    auto to_lds = [&](auto pc) __attribute__((always_inline)) {
      constexpr int i = decltype(pc)::value / PASSES, p = decltype(pc)::value % PASSES;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t at = wr ^ (32 * u);
        if constexpr (OUT_BF16) {
          const u32x4_t v = out[u];
          asm volatile("ds_write_b128 %0, %1" ::"v"(at), "v"(v) : "memory");
        } else {
          const f32x16_t& y = acc[i][p];
          const f32x4_t v = {y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]};
          asm volatile("ds_write_b128 %0, %1" ::"v"(at), "a"(v) : "memory");
        }
      }
    };
    const int row0 = wm * 32 * F + (ln >> 3), col0 = wn * 32 * F + (ln & 7) * (16 / ES);
    auto clear = [&](auto pc) __attribute__((always_inline)) {
      constexpr int i = decltype(pc)::value / PASSES, p = decltype(pc)::value % PASSES;
#pragma unroll
      for (int f = 0; f < FPP; ++f) zero(i, p * FPP + f);
    };
    bool behind_next = false;
    const int64_t shift = (MODE == kF8RowSegs ? (int64_t)cur.seg * n : 0) + cur.n0;   // of the bias
    if constexpr (EPI != kEpiNone && F == 4) {
      // The large tile's epilogue, of whole eights of columns: 32 rows of the wavefront's at
      // a time to LDS in fp32 (in the blocks of the second slot that its own loads fill;
      // piece p of row r at p ^ (p / 8 mod 2) ^ (r mod 8): neither the writes, of one piece
      // of neighbouring rows, nor the reads, of a row's even or odd pieces, meet a bank
      // twice), and from there in steps of four rows, a lane eight columns.  A SIMD has this
      // one wavefront, so nothing else runs under a wait of its own: four steps are formed
      // together, while the next four's values come back from LDS and their residual from
      // memory, with no branch between.  The steps are a loop: with every pass unrolled, as
      // the small tile has them, the code outgrows the instruction cache and the accumulators
      // leave their registers.  16384 x 1024 x 4096: bias 76 us (the product alone 76; 92 with
      // one step at a time), gelu 86, z kept as well 101 (112; 268 MB written, 51 us at a
      // copy's rate), residual 90 (127; the small tile 114); 16384 x 4096 x 1024 with a
      // residual 59 (alone 54), 64 experts (32768 rows, 2048 -> 768) silu with z 70 (57).
      if (loads) {
#pragma unroll
        for (int k = 0; k < FIRST0; ++k) first_load(k, nxt.nk);
      }
      const uint32_t to = (uint32_t)(uintptr_t)(lds_void*)(smem_f8 + SLOT + wave * 1024 + (ln & 31) / 2 * 4096 +
                                                           (ln & 1) * 512) + 16 * ((ln & 7) ^ (ln >> 5));
      const int k = ln & 15, rl = ln >> 4, col = wn * 128 + 8 * k;
      // row 4 it + rl, pieces 2 k and 2 k + 1 (the odd steps' at ^ 64: r mod 8 = rl + 4 (it mod 2))
      const unsigned char* from = smem_f8 + SLOT + wave * 1024 + rl / 2 * 4096 + rl % 2 * 512 + 128 * (k >> 2);
      const int sw = (k >> 2 & 1) ^ rl, lo0 = 16 * ((2 * k & 6) ^ sw), hi0 = 16 * ((2 * k & 6 | 1) ^ sw);
      const bool in = col < cur.cols;
      float bias[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) bias[x] = 0.0f;
      if (epi.bias && in) load_vector(epi.bias, epi.bias_bf16, shift + col, shift + col + 8, bias);
      // through descriptors of the tile's bytes: what lies past its rows and columns is
      // neither read nor written, with no branch for it
      auto tile_of = [&](const void* p, int64_t ld) __attribute__((always_inline)) {
        const uint8_t* base = static_cast<const uint8_t*>(p) + ((int64_t)cur.m0 * ld + cur.n0) * ES;
        return __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(scalar_base(base)), 0,
            (int)((uint32_t)(cur.rows - 1) * (uint32_t)(ld * ES) + (uint32_t)(cur.cols * ES)), 0x00027000);
      };
      auto place = [&](int64_t ld) __attribute__((always_inline)) {
        return ((uint32_t)(wm * 128 + rl) * (uint32_t)(ld * ES) + (uint32_t)(col * ES)) | (in ? 0u : 0x80000000u);
      };
      const __amdgpu_buffer_rsrc_t c_tile = tile_of(c, ldc), z_tile = tile_of(epi.z, epi.ldz);
      const __amdgpu_buffer_rsrc_t r_tile = tile_of(RES ? epi.res : c, RES ? epi.ldr : ldc);
      const uint32_t c_at = place(ldc), z_at = place(epi.ldz), r_at = RES ? place(epi.ldr) : 0;
      const uint32_t c_step = 4 * (uint32_t)(ldc * ES), z_step = 4 * (uint32_t)(epi.ldz * ES);
      const uint32_t r_step = RES ? 4 * (uint32_t)(epi.ldr * ES) : 0;
      // (bf16 streams, as the product's alone does: gelu with z 103 us, 115 if neither does, where a
      // step's activations are in memory; a program that writes the same z again has it in the last-level cache)
      auto store8 = [&](const float (&f)[8], __amdgpu_buffer_rsrc_t tile,
                        uint32_t at) __attribute__((always_inline)) {
        if constexpr (OUT_BF16) {
          const u32x4_t v = {bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                             bf16x2_rne(f[6], f[7])};
          __builtin_amdgcn_raw_buffer_store_b128(v, tile, (int)at, 0, 2);
        } else {
          const f32x4_t lo = {f[0], f[1], f[2], f[3]}, hi = {f[4], f[5], f[6], f[7]};
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, lo), tile, (int)at, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, hi), tile, (int)(at + 16), 0, 0);
        }
      };
      constexpr int U = 4;   // steps that are formed together
      constexpr int RV = OUT_BF16 ? 1 : 2;
      u32x4_t ahead[U][RV];   // the next steps' residual
      auto load_res = [&](int it) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int x = 0; x < RV; ++x)
            ahead[u][x] = __builtin_amdgcn_raw_buffer_load_b128(
                r_tile, (int)(r_at + (uint32_t)(it + u) * r_step + 16 * x), 0, 0);
      };
      if constexpr (RES) load_res(0);
      each_step<F>([&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value;
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16_t& y = acc[i][j];
            const f32x4_t v = {y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]};
            asm volatile("ds_write_b128 %0, %1 offset:%2" ::"v"(to ^ (32 * q) ^ (16 * (j & 1))), "a"(v), "i"(128 * j)
                         : "memory");
          }
        f32x4_t next[U][2];
        auto read = [&](int it) __attribute__((always_inline)) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int flip = 64 * ((it + u) & 1);
            const unsigned char* p = from + (it + u) * 8192;
            next[u][0] = *reinterpret_cast<const f32x4_t*>(p + (lo0 ^ flip));
            next[u][1] = *reinterpret_cast<const f32x4_t*>(p + (hi0 ^ flip));
          }
        };
        read(0);
#pragma unroll
        for (int j = 0; j < F; ++j) zero(i, j);
        auto steps = [&](auto act) __attribute__((always_inline)) {
#pragma unroll 1
          for (int it = 0; it < 8; it += U) {
            float f[U][8];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int y = 0; y < 8; ++y) f[u][y] = next[u][y / 4][y % 4] + bias[y];
            u32x4_t add[U][RV];
            if constexpr (RES) {
#pragma unroll
              for (int u = 0; u < U; ++u)
#pragma unroll
                for (int x = 0; x < RV; ++x) add[u][x] = ahead[u][x];
              if (i + 1 < F || it + U < 8) load_res(8 * i + it + U);
            }
            read((it + U) & 7);   // (behind the last ones the first again, unused)
            __builtin_amdgcn_sched_barrier(0);
            const uint32_t row = (uint32_t)(8 * i + it);
            if (epi.z) {
#pragma unroll
              for (int u = 0; u < U; ++u) store8(f[u], z_tile, z_at + (row + u) * z_step);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int y = 0; y < 8; ++y) f[u][y] = act(f[u][y]);
            if constexpr (RES) {
#pragma unroll
              for (int u = 0; u < U; ++u)
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                  if constexpr (OUT_BF16)
                    f[u][y] += __uint_as_float(y & 1 ? add[u][0][y / 2] & 0xFFFF0000u : add[u][0][y / 2] << 16);
                  else
                    f[u][y] += __uint_as_float(add[u][y / 4][y % 4]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) store8(f[u], c_tile, c_at + (row + u) * c_step);
          }
        };
        if (epi.act == kActGelu) steps([](float z) { return act_gelu(z); });
        else if (epi.act == kActSilu) steps([](float z) { return act_silu(z); });
        else if (epi.act == kActRelu) steps([](float z) { return z < 0.0f ? 0.0f : z; });
        else steps([](float z) { return z; });
      });
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the last values are out of their place
      if (loads) {
#pragma unroll
        for (int k = FIRST0; k < FIRST; ++k) first_load(k, nxt.nk);
      }
      behind_next = loads;
    } else if constexpr (EPI != kEpiNone) {
      // The small tile's: the same passes as below, each formed from the accumulators' own
      // layout: bias, then (where it is kept) z through LDS and out, then the activation
      // and the residual, whose loads are a pass ahead, and c through LDS.  A pass's values
      // are formed while those of the pass before come back.  The next tile's first loads
      // go out ahead of all: no wait for them is one for the stores.
      if (loads) {
#pragma unroll
        for (int k = 0; k < FIRST - HELD; ++k) first_load(k, nxt.nk);
      }
      const bool whole = pieces && epilogue_whole(epi, ES);
      // fragment j's columns 8 u + 4 h .. + 3, h = lane / 32, of row lane mod 32
      const int colf = wn * 32 * F + 4 * (ln >> 5), rowf = wm * 32 * F + (ln & 31);
      f32x4_t bias[F][4];
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          bias[j][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
          const int col = colf + 32 * j + 8 * u;
          if (epi.bias)
            bias[j][u] = epi.bias_bf16 ? four_f32<true>(four_in<true>(epi.bias, shift + col, cur.cols - col))
                                       : four_f32<false>(four_in<false>(epi.bias, shift + col, cur.cols - col));
        }
      Four<OUT_BF16> ahead[2][FPP][4];
      auto load_res = [&](auto pc) __attribute__((always_inline)) {
        constexpr int P = decltype(pc)::value, i = P / PASSES, p = P % PASSES;
        if (rowf + 32 * i >= cur.rows) return;
        const int64_t at = (int64_t)(cur.m0 + rowf + 32 * i) * epi.ldr + cur.n0;
#pragma unroll
        for (int f = 0; f < FPP; ++f)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int col = colf + 32 * (p * FPP + f) + 8 * u;
            ahead[P & 1][f][u] = four_in<OUT_BF16>(epi.res, at + col, cur.cols - col);
          }
      };
      // a pass's values, as pieces 2 u + h of its rows' 128 bytes
      auto pack = [&](const f32x4_t (&y)[FPP][4]) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if constexpr (OUT_BF16) {
            const f32x4_t &l = y[u / 2][2 * (u & 1)], &h = y[u / 2][2 * (u & 1) + 1];
            const auto a = __builtin_amdgcn_permlane32_swap(bf16x2_rne(l[0], l[1]), bf16x2_rne(h[0], h[1]), false, false);
            const auto b = __builtin_amdgcn_permlane32_swap(bf16x2_rne(l[2], l[3]), bf16x2_rne(h[2], h[3]), false, false);
            out[u] = u32x4_t{a[0], b[0], a[1], b[1]};
          } else {
            out[u] = __builtin_bit_cast(u32x4_t, y[0][u]);
          }
        }
      };
      u32x4_t vz[4], vc[4];
      auto through_lds = [&](u32x4_t (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const u32x4_t x = out[u];
          asm volatile("ds_write_b128 %0, %1" ::"v"(wr ^ (32 * u)), "v"(x) : "memory");
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) v[it] = *reinterpret_cast<const u32x4_t*>(src + it * STG_STEP);
        __builtin_amdgcn_sched_barrier(0);
      };
      char* zb = static_cast<char*>(epi.z) + (cur.m0 * epi.ldz + cur.n0) * ES;
      auto store = [&](char* base, int64_t ld, auto pc, const u32x4_t (&v)[4]) __attribute__((always_inline)) {
        constexpr int P = decltype(pc)::value, i = P / PASSES, p = P % PASSES;
        if (whole) {
          const uint32_t ldb = (uint32_t)(ld * ES);
          const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
              const_cast<uint8_t*>(scalar_base(reinterpret_cast<const uint8_t*>(base))), 0,
              (int)((uint32_t)(cur.rows - 1) * ldb + (uint32_t)(cur.cols * ES)), 0x00027000);
          const uint32_t at = ((uint32_t)(row0 + 32 * i) * ldb + (uint32_t)(col0 * ES) + 128 * p) |
                              (col0 + p * GROUP < cur.cols ? 0u : 0x80000000u);
#pragma unroll
          for (int it = 0; it < 4; ++it)
            __builtin_amdgcn_raw_buffer_store_b128(v[it], rsrc, (int)(at + (uint32_t)(8 * it) * ldb), 0, OUT_BF16 ? 2 : 0);
        } else {
          const int left = cur.cols - col0 - p * GROUP;
          char* dst = base + ((int64_t)(row0 + 32 * i) * ld + col0 + p * GROUP) * ES;
#pragma unroll
          for (int it = 0; it < 4; ++it, dst += 8 * ld * ES)
            if (row0 + 32 * i + 8 * it < cur.rows) piece_out<OUT_BF16>(dst, v[it], left);
        }
      };
      if constexpr (RES) load_res(F8Step<0>{});
      each_step<OUT_PASSES>([&](auto pc) __attribute__((always_inline)) {
        constexpr int P = decltype(pc)::value, i = P / PASSES, p = P % PASSES;
        // none of these rows in a part of a tile: nothing to form (16 rows among 64 experts, 2048 ->
        // 768, 18.3 -> 16.9 us)
        if (wm * 32 * F + 32 * i >= cur.rows) {
          clear(pc);
          if constexpr (P > 0 && p == 0) {
            if (wm * 32 * F + 32 * (i - 1) < cur.rows) store(cb, ldc, F8Step<P - 1>{}, vc);
          }
          return;
        }
        f32x4_t y[FPP][4];
#pragma unroll
        for (int f = 0; f < FPP; ++f)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const f32x16_t& a = acc[i][p * FPP + f];
            y[f][u] = f32x4_t{a[4 * u], a[4 * u + 1], a[4 * u + 2], a[4 * u + 3]} + bias[p * FPP + f][u];
          }
        clear(pc);
        if (epi.z) {
          pack(y);
          through_lds(vz);
        }
        if constexpr (RES && P + 1 < OUT_PASSES) load_res(F8Step<P + 1>{});
        activate(y, epi.act);
        if constexpr (RES) {
#pragma unroll
          for (int f = 0; f < FPP; ++f)
#pragma unroll
            for (int u = 0; u < 4; ++u) y[f][u] += four_f32<OUT_BF16>(ahead[P & 1][f][u]);
        }
        pack(y);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (P > 0) store(cb, ldc, F8Step<P - 1>{}, vc);
        if (epi.z) store(zb, epi.ldz, pc, vz);
        through_lds(vc);
      });
      if constexpr (HELD > 0) {
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the last values are out of their place
        if (loads) {
#pragma unroll
          for (int k = FIRST - HELD; k < FIRST; ++k) first_load(k, nxt.nk);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const bool all = wm * 32 * F + 32 * (F - 1) < cur.rows;
      if (all) store(cb, ldc, F8Step<OUT_PASSES - 1>{}, vc);
      behind_next = loads && whole && all;   // (every pass's stores are out)
    } else if (pieces) {
      const uint32_t ldb = (uint32_t)(ldc * ES);
      // below 2^31: a lane past the columns goes to 2^31 and on
      const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(scalar_base(reinterpret_cast<const uint8_t*>(cb))), 0,
          (int)((uint32_t)(cur.rows - 1) * ldb + (uint32_t)(cur.cols * ES)), 0x00027000);
      const uint32_t off = (uint32_t)row0 * ldb + (uint32_t)(col0 * ES);
      form(F8Step<0>{});
      each_step<OUT_PASSES>([&](auto pc) __attribute__((always_inline)) {
        constexpr int P = decltype(pc)::value, i = P / PASSES, p = P % PASSES;
        to_lds(pc);
        clear(pc);
        u32x4_t v[4];   // row 8 it + lane / 8, piece lane mod 8
#pragma unroll
        for (int it = 0; it < 4; ++it) v[it] = *reinterpret_cast<const u32x4_t*>(src + it * STG_STEP);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (P + 1 < OUT_PASSES) form(F8Step<P + 1>{});
        if (loads) {
#pragma unroll
          for (int k = P * (FIRST - HELD) / OUT_PASSES; k < (P + 1) * (FIRST - HELD) / OUT_PASSES; ++k)
            first_load(k, nxt.nk);
          if constexpr (HELD > 0 && P + 1 == OUT_PASSES) {
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the last values are out of their place
#pragma unroll
            for (int k = FIRST - HELD; k < FIRST; ++k) first_load(k, nxt.nk);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        const uint32_t at = (off + 128 * p) | (col0 + p * GROUP < cur.cols ? 0u : 0x80000000u);
#pragma unroll
        for (int it = 0; it < 4; ++it)
          // bf16 streaming (2), as store_stream
          __builtin_amdgcn_raw_buffer_store_b128(v[it], rsrc, (int)(at + (uint32_t)(32 * i + 8 * it) * ldb),
                                                 0, OUT_BF16 ? 2 : 0);
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      // any alignment and size
      if (HELD == 0 && loads) first_loads(nxt.nk);
      each_step<OUT_PASSES>([&](auto pc) __attribute__((always_inline)) {
        constexpr int P = decltype(pc)::value, i = P / PASSES, p = P % PASSES;
        form(pc);
        to_lds(pc);
        clear(pc);
        const int left = cur.cols - col0 - p * GROUP;
        char* dst = cb + ((int64_t)(row0 + 32 * i) * ldc + col0 + p * GROUP) * ES;
        u32x4_t v[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) v[it] = *reinterpret_cast<const u32x4_t*>(src + it * STG_STEP);
#pragma unroll
        for (int it = 0; it < 4; ++it, dst += 8 * ldc * ES) {
          if (row0 + 32 * i + 8 * it >= cur.rows) continue;
          if (left >= 16 / ES) {
            *reinterpret_cast<f8_piece_t*>(dst) = v[it];
          } else {
#pragma unroll
            for (int x = 0; x < 16 / ES; ++x) {
              if (x >= left) continue;
              if constexpr (OUT_BF16)
                reinterpret_cast<uint16_t*>(dst)[x] = (uint16_t)(v[it][x / 2] >> (16 * (x & 1)));
              else
                reinterpret_cast<uint32_t*>(dst)[x] = v[it][x];
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (HELD > 0) {
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        if (loads) first_loads(nxt.nk);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (!more) break;
    behind = EPI ? behind_next : pieces;
    cur = nxt;
  }
}

// ---------------------------------------------------------------------------
// Few rows: 16 columns (rows of b) and 16 MF rows of a to a workgroup of eight
// wavefronts that divide the blocks among them; a wavefront's operands come
// straight to registers (a block of a row: 32 bytes a lane), several blocks'
// loads in flight, and the partial sums meet in LDS.  Bound by latency at small
// weights (16 rows x 1024 x 2048: 4.6 us), by reading the weight at large ones
// (16 x 8192 x 4096: 10.4 us, 3.3 TB/s).
// ---------------------------------------------------------------------------
constexpr int kSkinnyWaves = 8;

template <int MF, bool OUT_BF16, bool EPI>
__global__ __launch_bounds__(64 * kSkinnyWaves) void k_gemm_f8_skinny(Fp8Operand A, Fp8Operand B,
                                                                      int64_t m, int64_t n,
                                                                      int k_blocks, void* c,
                                                                      int64_t ldc,
                                                                      EpilogueArg<EPI> epi) {
  __shared__ float part[kSkinnyWaves][16][16 * MF + 4];   // [..][column][row]
  const int64_t m0 = (int64_t)blockIdx.y * 16 * MF, n0 = (int64_t)blockIdx.x * 16;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int rows_here = (int)(m - m0 < 16 * MF ? m - m0 : 16 * MF);
  const int cols_here = (int)(n - n0 < 16 ? n - n0 : 16);
  // rows past the edge repeat the last one (their products are never stored)
  const int64_t br = n0 + (r < cols_here ? r : cols_here - 1);
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
  // U blocks: every load, then the products
  auto blocks = [&](int kb, auto uc) __attribute__((always_inline)) {
    constexpr int U = decltype(uc)::value;
    i32x8_t bf[U], af[U][MF];
    int sb[U], sa[U][MF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (int64_t)(kb + u) * 128;
      bf[u] = frag(*reinterpret_cast<const u32x4_t*>(bc + k),
                   *reinterpret_cast<const u32x4_t*>(bc + k + 16));
      sb[u] = bs[kb + u];
#pragma unroll
      for (int i = 0; i < MF; ++i) {
        af[u][i] = frag(*reinterpret_cast<const u32x4_t*>(ac[i] + k),
                        *reinterpret_cast<const u32x4_t*>(ac[i] + k + 16));
        sa[u][i] = as[i][kb + u];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MF; ++i)
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[u], af[u][i], acc[i], 0, 0, 0,
                                                                  sb[u], 0, sa[u][i]);
  };
  int kb = (int)((int64_t)k_blocks * w / kSkinnyWaves);
  const int kb1 = (int)((int64_t)k_blocks * (w + 1) / kSkinnyWaves);
  for (; kb + 4 <= kb1; kb += 4) blocks(kb, F8Step<4>{});
  for (; kb + 2 <= kb1; kb += 2) blocks(kb, F8Step<2>{});
  if (kb < kb1) blocks(kb, F8Step<1>{});
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
    if constexpr (EPI) {
      epilogue_one<OUT_BF16>(epi, c, ldc, m0 + row, n0 + col, n0 + col, s);
      continue;
    }
    const int64_t o = (m0 + row) * ldc + n0 + col;
    if constexpr (OUT_BF16)
      static_cast<uint16_t*>(c)[o] = (uint16_t)bf16x2_rne(s, 0.0f);
    else
      static_cast<float*>(c)[o] = s;
  }
}

// sums the splits' fp32 partials in order
template <bool OUT_BF16, bool EPI>
__global__ __launch_bounds__(256) void k_f8_reduce(const float* __restrict__ part, int splits,
                                                   int64_t m, int64_t n, void* c, int64_t ldc,
                                                   EpilogueArg<EPI> epi) {
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
  if constexpr (EPI) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e + i >= mn) break;
      const int64_t rr = (e + i) / n, cc = (e + i) - rr * n;
      epilogue_one<OUT_BF16>(epi, c, ldc, rr, cc, cc, s[i]);
    }
    return;
  }
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
  int skinny;   // 16-row fragments of the few-rows kernel, 0: a tiled one
  int f;        // tile side / 64
  int splits;   // of the blocks, into fp32 partials
};

// The choice minimises an estimate in microseconds, fitted to this card: the
// 256 x 256 tile (a workgroup a CU) takes 1.37 a stage and 7 a round of 256
// tiles, the 128 x 128 tile (two a CU) 1.02 and 2 a round of 512, or 0.62 a
// stage alone on its CU.  Row segments make the small tile's stages a fifth
// longer (it reads a segment's weights twice as often); block segments, each
// tile on its own, cost 2.3 (3.0) more a round.  A split output costs another launch
// and 8 bytes a value and split at 9.5 TB/s; the few-rows kernel reads both
// operands once a workgroup at 6.5 TB/s.
// Measured either side, one product over and over (us, large / small tile).
// Between a step's other kernels, with operands that have left the caches, the
// three by 64 segments take 80, 98 and 149 on the large tile; which side wins
// there was not measured:
//   16384 x 1024 x 3072  44.6 / 55.4    8192 x 2048 x 512     15.8 / 14.4
//   16384 x 3072 x 1024  58.1 / 78.8    65536 x 1024 x 256    38.8 / 34.8
//   32768 rows in 64 segments, 768 x 2048: 73.8 / 86.5, 2048 x 768: 88.9 / 98.6
//   8192 rows in 128 segments, 768 x 2048: 66.9 / 55.0
//   weight gradients of 32768 rows in 64 segments, 2048 x 768: 100.8 / 110.3,
//   of 16384 rows in 8, 1024 x 3072: 72.9 / 67.7
//   weight gradient over 16384 tokens, 1024 x 3072: 140 in one split, 64 in five
//   16 rows x 1024 x 2048: 9.9 small tile, 4.4 few-rows kernel
Fp8Plan fp8_plan(int64_t m, int64_t n, int64_t k_blocks, Fp8Mode mode, int nseg) {
  Fp8Plan best{0, 4, 1};
  double best_us = 1e300;
  auto offer = [&](const Fp8Plan& p, double us) {
    if (us < best_us) {
      best_us = us;
      best = p;
    }
  };
  const double dm = (double)m, dn = (double)n;
  for (int f = 4; f >= 2; f -= 2) {
    const int side = 64 * f, slots = f == 4 ? kF8Cus : 2 * kF8Cus;
    const double tx = (double)((n + side - 1) / side);
    double tiles = tx * (double)((m + side - 1) / side), stages = (double)k_blocks;
    // segments end in part of a tile (a block): half of one on average
    if (mode == kF8RowSegs) tiles = tx * (dm / side + 0.5 * (double)(nseg < m ? nseg : m));
    if (mode == kF8BlockSegs) {
      tiles *= nseg;
      stages = stages / nseg;
    }
    for (int splits = 1; splits <= 16; ++splits) {
      if (splits > 1 && (mode != kF8All || k_blocks < 2 * splits)) break;
      const double t = tiles * splits;
      const double stage = f == 4 ? 1.37 : (t <= kF8Cus ? 0.62 : 1.02) * (mode == kF8RowSegs ? 1.2 : 1.0);
      const double alone = mode != kF8BlockSegs ? 0.0 : f == 4 ? 2.3 : 3.0;
      const double tile = (f == 4 ? 7.0 : t <= kF8Cus ? 1.5 : 2.0) + alone;
      // the last round is not full; how full, the segments leave open
      const double rounds = t <= slots       ? 1.0
                            : mode == kF8All ? (double)(int64_t)((t + slots - 1) / slots)
                                             : t / slots + 0.35;
      const double per = (double)((int64_t)(stages + splits - 1) / splits);
      offer(Fp8Plan{0, f, splits}, 3.0 + rounds * (per * stage + tile) +
                                       (splits > 1 ? 5.0 + splits * dm * dn * 8.0 / 9.5e6 : 0.0));
    }
  }
  if (mode == kF8All) {
    for (int mf = 1; mf <= 4; mf *= 2) {
      const double rows = (double)((m + 16 * mf - 1) / (16 * mf)), wgs = (double)((n + 15) / 16) * rows;
      if (wgs > 65536.0 || rows > 65535.0) continue;   // (the grid's y)
      offer(Fp8Plan{mf, 0, 1}, 3.0 + wgs * (double)k_blocks * 128.0 * (16.0 + 16.0 * mf) / 6.5e6 + 0.5 * mf);
    }
  }
  return best;
}

template <int F, bool OB, int MODE, int EPI>
hipError_t gemm_f8_t(const Fp8Gemm& g, int splits, void* c, int64_t ldc, int64_t c_split,
                     const EpilogueArg<EPI != kEpiNone>& epi, hipStream_t st) {
  constexpr size_t lds = f8_lds_bytes(F);
  static_assert(lds <= 160 * 1024 / (F == 4 ? 1 : 2), "fits one CU's LDS");
  const hipError_t e = lds_attr_once<&k_gemm_f8<F, OB, MODE, EPI>>((int)lds);
  if (e != hipSuccess) return e;
  const int64_t ty = MODE == kF8RowSegs ? chunk_upper_bound(g.m, g.nseg, 64 * F)
                                        : (g.m + 64 * F - 1) / (64 * F);
  const int64_t tx = (g.n + 64 * F - 1) / (64 * F);
  const int64_t tiles = tx * ty * (MODE == kF8BlockSegs ? g.nseg : splits);
  constexpr int slots = F == 4 ? kF8Cus : 2 * kF8Cus;
  const int64_t grid = MODE != kF8BlockSegs && tiles > slots ? slots : tiles;
  k_gemm_f8<F, OB, MODE, EPI><<<dim3((unsigned)grid), kF8Threads, lds, st>>>(
      g.a, g.b, (int)g.m, (int)g.n, (int)g.k_blocks, g.offs, g.nseg, g.rows, splits, (int)tx,
      (int)ty, c, ldc, c_split, epi);
  return hipGetLastError();
}

template <int F, bool OB>
hipError_t gemm_f8_mode(const Fp8Gemm& g, int splits, void* c, int64_t ldc, int64_t c_split,
                        const Fp8Epilogue* epi, hipStream_t st) {
  if (epi && g.mode == kF8RowSegs)   // (of a product by block segments: none)
    return epi->res ? gemm_f8_t<F, OB, kF8RowSegs, kEpiResidual>(g, splits, c, ldc, c_split, *epi, st)
                    : gemm_f8_t<F, OB, kF8RowSegs, kEpiPlain>(g, splits, c, ldc, c_split, *epi, st);
  if (epi)
    return epi->res ? gemm_f8_t<F, OB, kF8All, kEpiResidual>(g, splits, c, ldc, c_split, *epi, st)
                    : gemm_f8_t<F, OB, kF8All, kEpiPlain>(g, splits, c, ldc, c_split, *epi, st);
  const NoEpilogue no;
  switch (g.mode) {
    case kF8RowSegs: return gemm_f8_t<F, OB, kF8RowSegs, kEpiNone>(g, splits, c, ldc, c_split, no, st);
    case kF8BlockSegs: return gemm_f8_t<F, OB, kF8BlockSegs, kEpiNone>(g, splits, c, ldc, c_split, no, st);
    default: return gemm_f8_t<F, OB, kF8All, kEpiNone>(g, splits, c, ldc, c_split, no, st);
  }
}

hipError_t gemm_f8(const Fp8Gemm& g, const Fp8Plan& p, bool bf16, void* c, int64_t ldc,
                   int64_t c_split, const Fp8Epilogue* epi, hipStream_t st) {
  if (p.f == 2)
    return bf16 ? gemm_f8_mode<2, true>(g, p.splits, c, ldc, c_split, epi, st)
                : gemm_f8_mode<2, false>(g, p.splits, c, ldc, c_split, epi, st);
  return bf16 ? gemm_f8_mode<4, true>(g, p.splits, c, ldc, c_split, epi, st)
              : gemm_f8_mode<4, false>(g, p.splits, c, ldc, c_split, epi, st);
}

template <int MF, bool EPI>
hipError_t skinny_t(const Fp8Gemm& g, const EpilogueArg<EPI>& epi, hipStream_t st) {
  const dim3 grid((unsigned)((g.n + 15) / 16), (unsigned)((g.m + 16 * MF - 1) / (16 * MF)));
  if (g.c_bf16)
    k_gemm_f8_skinny<MF, true, EPI><<<grid, 64 * kSkinnyWaves, 0, st>>>(
        g.a, g.b, g.m, g.n, (int)g.k_blocks, g.c, g.ldc, epi);
  else
    k_gemm_f8_skinny<MF, false, EPI><<<grid, 64 * kSkinnyWaves, 0, st>>>(
        g.a, g.b, g.m, g.n, (int)g.k_blocks, g.c, g.ldc, epi);
  return hipGetLastError();
}

template <bool EPI>
hipError_t reduce_t(const Fp8Gemm& g, const void* part, int splits, const EpilogueArg<EPI>& epi,
                    hipStream_t st) {
  const dim3 grid((unsigned)((g.m * g.n + 1023) / 1024));
  if (g.c_bf16)
    k_f8_reduce<true, EPI><<<grid, 256, 0, st>>>(static_cast<const float*>(part), splits, g.m, g.n, g.c, g.ldc, epi);
  else
    k_f8_reduce<false, EPI><<<grid, 256, 0, st>>>(static_cast<const float*>(part), splits, g.m, g.n, g.c, g.ldc, epi);
  return hipGetLastError();
}

template <int MF>
hipError_t skinny(const Fp8Gemm& g, hipStream_t st) {
  return g.epilogue ? skinny_t<MF, true>(g, *g.epilogue, st) : skinny_t<MF, false>(g, NoEpilogue{}, st);
}

}  // namespace

size_t fp8_gemm_ws_bytes(int64_t m, int64_t n, int64_t k_blocks, Fp8Mode mode, int nseg) {
  const Fp8Plan p = fp8_plan(m, n, k_blocks, mode, nseg);
  return p.splits > 1 ? ((size_t)p.splits * m * n * 4 + 255) & ~(size_t)255 : 0;
}

hipError_t launch_fp8_gemm(const Fp8Gemm& g, void* ws, hipStream_t st) {
  if (g.m == 0 || g.n == 0) return hipSuccess;
  Fp8Plan p = fp8_plan(g.m, g.n, g.k_blocks, g.mode, g.nseg);
  if (p.skinny == 1) return skinny<1>(g, st);
  if (p.skinny == 2) return skinny<2>(g, st);
  if (p.skinny == 4) return skinny<4>(g, st);
  // the large tile's epilogue takes eight columns a lane, in pieces of 16 bytes; any other form the small one's
  if (g.epilogue && p.f == 4 && p.splits == 1) {
    const int es = g.c_bf16 ? 2 : 4;
    if (!(g.n % 8 == 0 && g.ldc * es % 16 == 0 && g.ldc <= (1 << 21) &&
          (reinterpret_cast<uintptr_t>(g.c) & 15) == 0 && epilogue_whole(*g.epilogue, es)))
      p.f = 2;
  }
  if (p.splits > 1) {
    const hipError_t e = gemm_f8(g, p, false, ws, g.n, g.m * g.n, nullptr, st);
    if (e != hipSuccess) return e;
    return g.epilogue ? reduce_t<true>(g, ws, p.splits, *g.epilogue, st)
                      : reduce_t<false>(g, ws, p.splits, NoEpilogue{}, st);
  }
  return gemm_f8(g, p, g.c_bf16, g.c, g.ldc, g.mode == kF8BlockSegs ? g.m * g.ldc : 0, g.epilogue, st);
}

}  // namespace averis
