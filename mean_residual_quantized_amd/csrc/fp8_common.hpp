// The block-scaled 8-bit format of the fp8 kernels (gfx950): E4M3FN codes, one
// power-of-two scale (E8M0: 2^(byte - 127)) for each run of 128 elements along
// the contraction axis.  The scale is the smallest power of two with
// amax <= 448 scale (at least 2^-127), so dividing by it is exact, nothing
// saturates, and the one rounding is the code's (to nearest, ties to even).
// It is also the form the scaled matrix instruction takes, which then costs no
// vector instruction for scaling.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.hpp"

namespace averis {

constexpr int kF8Block = 128;   // elements that share a scale

// 16 bytes at element alignment (gfx950 loads them at any address)
typedef u32x4_t f8_piece_t __attribute__((aligned(2)));

// Scale byte from the bits of max |a| (fp32): 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t f8_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e > 0 ? (uint32_t)e : 0u;
}
// a block that holds an infinity or NaN: its codes are all NaN, its scale 1
__device__ __forceinline__ bool f8_not_finite(uint32_t amax_bits) { return amax_bits >= 0x7F800000u; }
constexpr uint32_t kF8NanCodes = 0x7F7F7F7Fu;
constexpr uint32_t kF8One = 127;
// four codes of which the first `left` are elements, the rest pad: 0 (as they
// are already, but in a block of NaN codes)
__device__ __forceinline__ uint32_t f8_without_pad(uint32_t codes, int left) {
  return left >= 4 ? codes : left > 0 ? codes & (0xFFFFFFFFu >> (8 * (4 - left))) : 0u;
}

// four fp32 values times 2^(127 - byte) -> four codes.  The product is exact:
// it is at most 448, and what falls below fp32's range is far below half the
// smallest code.
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d, uint32_t byte) {
  const float inv = __uint_as_float((254u - byte) << 23);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  return (uint32_t)w;
}

typedef short i16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// four bf16 values (two dwords) -> four codes.  The conversion divides by the
// power of two of its scale operand; byte 0 (2^-127, no normal fp32 number)
// takes the multiplication instead.
__device__ __forceinline__ uint32_t f8_codes4_bf16(uint32_t w0, uint32_t w1, uint32_t byte) {
  if (__builtin_expect(byte == 0u, 0))
    return f8_codes4(__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xFFFF0000u),
                     __uint_as_float(w1 << 16), __uint_as_float(w1 & 0xFFFF0000u), byte);
  const float s = __uint_as_float(byte << 23);
  i16x2_t r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, w0), s, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, w1), s, true);
  return __builtin_bit_cast(uint32_t, r);
}

// max over two packed pairs of bf16 magnitudes
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                __builtin_bit_cast(u16x2_t, b)));
}

// max over the 16 lanes of a DPP row (every lane gets it)
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  auto mx = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = mx(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true));    // lane ^ 1
  v = mx(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true));    // lane ^ 2
  v = mx(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true));   // the other four of eight
  return mx(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true));   // the other eight
}

}  // namespace averis
