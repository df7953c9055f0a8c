// C ABI of what stands around a block's linears: the norm with the residual's
// addition, and the way back through a linear's activation and bias.  Every
// check runs before the first HIP call.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_fp8.hpp"
#include "segments.hpp"

using namespace averis;

static_assert(AVERIS_MAX_NORM_COLS == kMaxNormCols && AVERIS_ACT_NONE == kActNone &&
                  AVERIS_ACT_RELU == kActRelu && AVERIS_ACT_SILU == kActSilu &&
                  AVERIS_ACT_GELU == kActGelu, "limits and names");

namespace {

// a rows x cols matrix (optional: p may be NULL)
averis_status_t check_rows(const void* p, averis_dtype_t dtype, int64_t rows, int64_t cols,
                           int64_t ld, bool optional) {
  if (!p) return optional || rows == 0 ? AVERIS_OK : AVERIS_E_NULL;
  if (ld < cols) return AVERIS_E_SHAPE;
  return aligned(p, elem_size(dtype)) ? AVERIS_OK : AVERIS_E_ALIGN;
}

averis_status_t check_vector(const void* p, averis_dtype_t dtype, bool optional) {
  if (!p) return optional ? AVERIS_OK : AVERIS_E_NULL;
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  return aligned(p, elem_size(dtype)) ? AVERIS_OK : AVERIS_E_ALIGN;
}

averis_status_t check_norm(averis_dtype_t dtype, int64_t rows, int64_t cols, const void* weight,
                           averis_dtype_t wdtype, const float* rstd) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  if (rows < 0 || rows > kMaxDim || cols <= 0 || cols > kMaxNormCols) return AVERIS_E_SHAPE;
  if (rows > 0 && !rstd) return AVERIS_E_NULL;
  if (!aligned(rstd, 4)) return AVERIS_E_ALIGN;
  return check_vector(weight, wdtype, false);
}

}  // namespace

extern "C" {

averis_status_t averis_rmsnorm(const void* x, averis_dtype_t dtype, int64_t rows, int64_t cols,
                               int64_t ldx, const void* residual, int64_t ldres,
                               const void* weight, averis_dtype_t wdtype, double eps, void* h,
                               int64_t ldh, void* y, int64_t ldy, float* rstd,
                               const averis_fp8_t* out, const averis_fp8_t* out_t,
                               hipStream_t stream) {
  averis_status_t s = check_norm(dtype, rows, cols, weight, wdtype, rstd);
  if (s != AVERIS_OK) return s;
  if (!(eps >= 0.0) || (h && !residual)) return AVERIS_E_ARG;
  if (!y && !out && !out_t) return AVERIS_E_NULL;
  if ((s = check_rows(x, dtype, rows, cols, ldx, false)) != AVERIS_OK) return s;
  if ((s = check_rows(residual, dtype, rows, cols, ldres, true)) != AVERIS_OK) return s;
  if ((s = check_rows(h, dtype, rows, cols, ldh, !residual)) != AVERIS_OK) return s;
  if ((s = check_rows(y, dtype, rows, cols, ldy, true)) != AVERIS_OK) return s;
  if (out && (s = check_fp8(out, rows, cols)) != AVERIS_OK) return s;
  if (out_t) {
    if ((s = check_fp8(out_t, cols, rows)) != AVERIS_OK) return s;
    if (tiles_of(cols) * tiles_of(rows) > kMaxTiles) return AVERIS_E_SHAPE;
  }
  const bool bf16 = dtype == AVERIS_BF16, wbf16 = wdtype == AVERIS_BF16;
  const NormArgs a{x, residual, ldx, ldres, weight, wbf16, eps, h, ldh, y, ldy, rstd};
  s = hip_status(launch_norm(a, bf16, rows, cols, out_of(out), stream));
  if (s != AVERIS_OK || !out_t) return s;
  return hip_status(launch_norm_tile(residual ? h : x, bf16, rows, cols, residual ? ldh : ldx,
                                     weight, wbf16, rstd, out_of(out_t), stream));
}

averis_status_t averis_rmsnorm_grad(const void* dy, averis_dtype_t dtype, int64_t rows,
                                    int64_t cols, int64_t lddy, const void* h, int64_t ldh,
                                    const void* weight, averis_dtype_t wdtype, const float* rstd,
                                    const void* dres, int64_t lddres, void* dh, int64_t lddh,
                                    float* dweight, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
  averis_status_t s = check_norm(dtype, rows, cols, weight, wdtype, rstd);
  if (s != AVERIS_OK) return s;
  if ((s = check_rows(dy, dtype, rows, cols, lddy, false)) != AVERIS_OK) return s;
  if ((s = check_rows(h, dtype, rows, cols, ldh, false)) != AVERIS_OK) return s;
  if ((s = check_rows(dres, dtype, rows, cols, lddres, true)) != AVERIS_OK) return s;
  if ((s = check_rows(dh, dtype, rows, cols, lddh, false)) != AVERIS_OK) return s;
  if (!aligned(dweight, 4)) return AVERIS_E_ALIGN;
  if ((s = check_ws(ws, ws_bytes, dweight ? norm_grad_ws_bytes(rows, cols) : 0)) != AVERIS_OK) return s;
  const NormGradArgs a{dy, h, dres, lddy, ldh, lddres, weight, wdtype == AVERIS_BF16, rstd, dh, lddh,
                       dweight};
  return hip_status(launch_norm_grad(a, dtype == AVERIS_BF16, rows, cols, ws, stream));
}

averis_status_t averis_fp8_act_grad(const void* dy, averis_dtype_t dtype, int64_t rows,
                                    int64_t cols, int64_t lddy, const void* z, int64_t ldz,
                                    averis_act_t act, const int64_t* seg_offsets, int nseg,
                                    const averis_fp8_t* out, const averis_fp8_t* out_t,
                                    float* dbias, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  if (act < AVERIS_ACT_NONE || act > AVERIS_ACT_GELU) return AVERIS_E_ARG;
  if (rows < 0 || rows > kMaxDim || cols <= 0 || cols > kMaxActCols) return AVERIS_E_SHAPE;
  averis_status_t s = check_segs(seg_offsets, nseg);
  if (s != AVERIS_OK) return s;
  if (!out && !out_t && !dbias) return AVERIS_E_NULL;
  if ((s = check_rows(dy, dtype, rows, cols, lddy, false)) != AVERIS_OK) return s;
  if (act != AVERIS_ACT_NONE && (s = check_rows(z, dtype, rows, cols, ldz, false)) != AVERIS_OK)
    return s;
  if (out && (s = check_fp8(out, rows, cols)) != AVERIS_OK) return s;
  if (out_t) {
    const int64_t tc = seg_offsets ? averis_fp8_seg_cols(rows, nseg) : rows;
    if ((s = check_fp8(out_t, cols, tc)) != AVERIS_OK) return s;
  }
  if (tiles_of(cols) * chunk_upper_bound(rows, nseg, 128) > kMaxTiles) return AVERIS_E_SHAPE;
  if (!aligned(dbias, 4)) return AVERIS_E_ALIGN;
  if ((s = check_ws(ws, ws_bytes, dbias ? act_grad_ws_bytes(rows, cols, nseg) : 0)) != AVERIS_OK) return s;
  return hip_status(launch_act_grad(dy, dtype == AVERIS_BF16, rows, cols, lddy, z, ldz, act,
                                    seg_offsets, nseg, out_of(out), out_of(out_t), dbias, ws,
                                    stream));
}

}  // extern "C"
