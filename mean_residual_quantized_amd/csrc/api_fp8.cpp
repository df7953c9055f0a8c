// C ABI of the block-scaled fp8 linears: argument validation and launches.
// Every check runs before the first HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_fp8.hpp"
#include "segments.hpp"

using namespace averis;

extern "C" {

int64_t averis_fp8_seg_cols(int64_t rows, int64_t nseg) {
  if (rows < 0 || rows > kMaxDim || nseg < 1 || nseg > kMaxSeg) return -1;
  return chunk_upper_bound(rows, (int)nseg, 128) * 128;
}

averis_status_t averis_fp8_quant(const void* a, averis_dtype_t dtype, int64_t rows, int64_t cols,
                                 int64_t lda, const int64_t* seg_offsets, int nseg,
                                 const averis_fp8_t* out, const averis_fp8_t* out_t,
                                 hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  if (rows < 0 || cols <= 0 || rows > kMaxDim || cols > kMaxDim || lda < cols) return AVERIS_E_SHAPE;
  averis_status_t s = check_segs(seg_offsets, nseg);
  if (s != AVERIS_OK) return s;
  if ((rows > 0 && !a) || (!out && !out_t)) return AVERIS_E_NULL;
  if (!aligned(a, elem_size(dtype))) return AVERIS_E_ALIGN;
  if (out && (s = check_fp8(out, rows, cols)) != AVERIS_OK) return s;
  if (out_t) {
    const int64_t tc = seg_offsets ? averis_fp8_seg_cols(rows, nseg) : rows;
    if ((s = check_fp8(out_t, cols, tc)) != AVERIS_OK) return s;
    if (tiles_of(cols) * chunk_upper_bound(rows, nseg, 128) > kMaxTiles) return AVERIS_E_SHAPE;
    return hip_status(launch_fp8_tile(a, dtype == AVERIS_BF16, false, 1, rows, cols, lda, 0,
                                      seg_offsets, nseg, out_of(out), out_of(out_t), stream));
  }
  return hip_status(launch_fp8_rows(a, dtype == AVERIS_BF16, rows, cols, lda, out_of(out), stream));
}

averis_status_t averis_fp8_quant_weight(const void* w, averis_dtype_t dtype, int batch,
                                        int64_t rows, int64_t cols, int64_t ldw,
                                        int64_t batch_stride, const averis_fp8_t* out,
                                        const averis_fp8_t* out_t, hipStream_t stream) {
  if (!dtype_ok(dtype)) return AVERIS_E_DTYPE;
  if (batch < 1 || batch > kMaxSeg) return AVERIS_E_ARG;
  if (rows <= 0 || cols <= 0 || rows > kMaxDim || cols > kMaxDim) return AVERIS_E_SHAPE;
  if (ldw < cols || batch_stride < 0) return AVERIS_E_SHAPE;
  if (tiles_of(cols) * tiles_of(rows) > kMaxTiles) return AVERIS_E_SHAPE;
  if (batch > 1 && batch_stride < rows * ldw) return AVERIS_E_SHAPE;
  if (!w || (!out && !out_t)) return AVERIS_E_NULL;
  if (!aligned(w, elem_size(dtype))) return AVERIS_E_ALIGN;
  averis_status_t s;
  if (out && (s = check_fp8(out, (int64_t)batch * rows, cols)) != AVERIS_OK) return s;
  if (out_t && (s = check_fp8(out_t, (int64_t)batch * cols, rows)) != AVERIS_OK) return s;
  return hip_status(launch_fp8_tile(w, dtype == AVERIS_BF16, true, batch, rows, cols, ldw,
                                    batch_stride, nullptr, 1, out_of(out), out_of(out_t), stream));
}

static averis_status_t gemm_common(const averis_fp8_t* a, const averis_fp8_t* b,
                                   const int64_t* seg_offsets, int nseg, void* c,
                                   averis_dtype_t cdtype, int64_t ldc,
                                   const Fp8Epilogue* epilogue, void* ws, size_t ws_bytes,
                                   hipStream_t stream) {
  if (!a || !b) return AVERIS_E_NULL;
  averis_status_t s = check_segs(seg_offsets, nseg);
  if (s != AVERIS_OK) return s;
  const int64_t m = a->rows, k = a->cols;
  if (m < 0 || m > kMaxDim || k <= 0 || k > kMaxK || b->cols != k) return AVERIS_E_SHAPE;
  if (b->rows < 0 || b->rows % nseg != 0) return AVERIS_E_SHAPE;
  const int64_t n = b->rows / nseg;
  // tiles are numbered in 32 bits
  if (n > kMaxDim || tiles_of(n) * chunk_upper_bound(m, nseg, 128) > 1 << 30) return AVERIS_E_SHAPE;
  if ((s = check_fp8(a, m, k)) != AVERIS_OK) return s;
  if ((s = check_fp8(b, b->rows, k)) != AVERIS_OK) return s;
  if ((s = check_c(c, cdtype, m, n, ldc)) != AVERIS_OK) return s;
  if (epilogue) {
    if (epilogue->res && (s = check_c(epilogue->res, cdtype, m, n, epilogue->ldr)) != AVERIS_OK) return s;
    if (epilogue->z && (s = check_c(epilogue->z, cdtype, m, n, epilogue->ldz)) != AVERIS_OK) return s;
  }
  const Fp8Gemm g{operand_of(a), operand_of(b), m, n, (k + 127) / 128,
                  seg_offsets ? kF8RowSegs : kF8All, seg_offsets, nseg, m, c,
                  cdtype == AVERIS_BF16, ldc, epilogue};
  if ((s = check_ws(ws, ws_bytes, fp8_gemm_ws_bytes(m, n, g.k_blocks, g.mode, nseg))) != AVERIS_OK)
    return s;
  return hip_status(launch_fp8_gemm(g, ws, stream));
}

averis_status_t averis_fp8_gemm(const averis_fp8_t* a, const averis_fp8_t* b,
                                const int64_t* seg_offsets, int nseg, void* c,
                                averis_dtype_t cdtype, int64_t ldc, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  return gemm_common(a, b, seg_offsets, nseg, c, cdtype, ldc, nullptr, ws, ws_bytes, stream);
}

averis_status_t averis_fp8_gemm_act(const averis_fp8_t* a, const averis_fp8_t* b, const void* bias,
                                    averis_dtype_t bias_dtype, averis_act_t act,
                                    const void* residual, int64_t ldr, const int64_t* seg_offsets,
                                    int nseg, void* c, averis_dtype_t cdtype, int64_t ldc, void* z,
                                    int64_t ldz, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (act < AVERIS_ACT_NONE || act > AVERIS_ACT_GELU) return AVERIS_E_ARG;
  if (bias && !dtype_ok(bias_dtype)) return AVERIS_E_DTYPE;
  if (bias && !aligned(bias, elem_size(bias_dtype))) return AVERIS_E_ALIGN;
  const Fp8Epilogue e{bias, bias && bias_dtype == AVERIS_BF16, act, residual, ldr, z, ldz};
  return gemm_common(a, b, seg_offsets, nseg, c, cdtype, ldc, &e, ws, ws_bytes, stream);
}

averis_status_t averis_fp8_gemm_wgrad(const averis_fp8_t* xt, const averis_fp8_t* dt,
                                      int64_t rows, const int64_t* seg_offsets, int nseg,
                                      void* dw, averis_dtype_t dwdtype, int64_t lddw, void* ws,
                                      size_t ws_bytes, hipStream_t stream) {
  if (!xt || !dt) return AVERIS_E_NULL;
  averis_status_t s = check_segs(seg_offsets, nseg);
  if (s != AVERIS_OK) return s;
  const int64_t m = xt->rows, n = dt->rows;
  if (m < 0 || n < 0 || m > kMaxDim || n > kMaxDim || rows < 0) return AVERIS_E_SHAPE;
  const int64_t k = seg_offsets ? averis_fp8_seg_cols(rows, nseg) : rows;
  if (k < 0 || k > kMaxK) return AVERIS_E_SHAPE;
  // tiles are numbered in 32 bits; by segment each is a workgroup of 256 threads,
  // fewer than 2^32 in all
  const int64_t most = seg_offsets ? (1 << 24) - 1 : 1 << 30;
  if (tiles_of(n) > most || tiles_of(m) > most / std::max<int64_t>(tiles_of(n), 1) / nseg)
    return AVERIS_E_SHAPE;
  if ((s = check_fp8(xt, m, k)) != AVERIS_OK) return s;
  if ((s = check_fp8(dt, n, k)) != AVERIS_OK) return s;
  if ((s = check_c(dw, dwdtype, m, n, lddw)) != AVERIS_OK) return s;
  const Fp8Gemm g{operand_of(xt), operand_of(dt), m, n, (k + 127) / 128,
                  seg_offsets ? kF8BlockSegs : kF8All, seg_offsets, nseg, rows, dw,
                  dwdtype == AVERIS_BF16, lddw, nullptr};
  if ((s = check_ws(ws, ws_bytes, fp8_gemm_ws_bytes(m, n, g.k_blocks, g.mode, nseg))) != AVERIS_OK)
    return s;
  return hip_status(launch_fp8_gemm(g, ws, stream));
}

}  // extern "C"
