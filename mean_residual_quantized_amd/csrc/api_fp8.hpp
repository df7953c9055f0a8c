// Argument checks of the calls on fp8 tensors.
#pragma once

#include "api_common.hpp"
#include "launch.hpp"

namespace averis {

constexpr int64_t kMaxDim = (int64_t)1 << 30;   // rows and columns of one operand
constexpr int64_t kMaxK = kMaxDim / 256;        // a tile's 256 rows of codes in 32-bit offsets
constexpr int64_t kMaxTiles = (1 << 23) - 1;   // of 128 x 128, 512 threads each: below 2^32 threads

inline averis_status_t check_fp8(const averis_fp8_t* t, int64_t rows, int64_t cols) {
  if (!t) return AVERIS_E_NULL;
  if (t->rows != rows || t->cols != cols) return AVERIS_E_SHAPE;
  if (rows > 0 && cols > 0 && (!t->codes || !t->scales)) return AVERIS_E_NULL;
  return aligned(t->codes, 16) && aligned(t->scales, 4) ? AVERIS_OK : AVERIS_E_ALIGN;
}

inline Fp8Out out_of(const averis_fp8_t* t) {
  return t ? Fp8Out{t->codes, t->scales, fp8_pitch(t->cols), fp8_spitch(t->cols)}
           : Fp8Out{nullptr, nullptr, 0, 0};
}
inline Fp8Operand operand_of(const averis_fp8_t* t) {
  return Fp8Operand{t->codes, t->scales, fp8_pitch(t->cols), fp8_spitch(t->cols)};
}

inline averis_status_t check_segs(const int64_t* offs, int nseg) {
  if (nseg < 1 || nseg > kMaxSeg || (!offs && nseg != 1)) return AVERIS_E_ARG;
  return aligned(offs, 8) ? AVERIS_OK : AVERIS_E_ALIGN;
}

inline averis_status_t check_c(const void* c, averis_dtype_t dtype, int64_t m, int64_t n, int64_t ldc) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  if (ldc < n) return AVERIS_E_SHAPE;
  if (m > 0 && n > 0 && !c) return AVERIS_E_NULL;
  return aligned(c, elem_size(dtype)) ? AVERIS_OK : AVERIS_E_ALIGN;
}

inline int64_t tiles_of(int64_t n) { return (n + 127) / 128; }

inline averis_status_t check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need && (!ws || ws_bytes < need)) return AVERIS_E_WORKSPACE;
  return ws && !aligned(ws, 256) ? AVERIS_E_ALIGN : AVERIS_OK;
}

}  // namespace averis
