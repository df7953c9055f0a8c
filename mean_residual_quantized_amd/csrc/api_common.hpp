// Argument checks shared by the C ABI files.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/averis.h"

namespace averis {

constexpr int kMaxSeg = 4096;
constexpr int kMaxGrads = 1 << 20;

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t elem_size(averis_dtype_t d) { return d == AVERIS_BF16 ? 2 : 4; }
inline bool dtype_ok(averis_dtype_t d) { return d == AVERIS_F32 || d == AVERIS_BF16; }

// AVERIS_OK, or AVERIS_E_HIP with the error's text for averis_last_error
averis_status_t hip_status(hipError_t e);

}  // namespace averis
