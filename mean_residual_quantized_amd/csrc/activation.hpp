// The activations of a product's epilogue and of the way back through it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace averis {

// silu(z) = z s(z) and gelu(z) = z s(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3), with s(u) = 1 / (1 +
// e^-u): the tanh form of gelu, for (1 + tanh(v)) / 2 = s(2 v).  e^-u (2 to the power of -u / log 2) and
// the reciprocal are single instructions, an error of 1 ulp each.
constexpr float kActLog2e = 1.4426950408889634f;
constexpr float kGeluA = 1.5957691216057308f, kGeluB = kGeluA * 0.044715f;   // u = z (A + B z^2)

// s(u) of u / log 2
__device__ __forceinline__ float act_sigmoid(float u2) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-u2));
}
__device__ __forceinline__ float act_silu(float z) { return z * act_sigmoid(kActLog2e * z); }
__device__ __forceinline__ float act_gelu(float z) {
  return z * act_sigmoid(z * __builtin_fmaf(kGeluB * kActLog2e, z * z, kGeluA * kActLog2e));
}

// d/dz of z s(u): s + s (1 - s) z du/dz, in this order (gelu of 16384 x 4096 normal z in bf16: every code
// as fp64 gives it; with z s first 790 are a step off).  Past |z| = 100 it is its limit, 1 or 0, and the
// products of its terms might overflow: z is held there (where it is NaN, s is).
__device__ __forceinline__ float act_silu_slope(float z) {
  const float s = act_sigmoid(kActLog2e * z), h = __builtin_amdgcn_fmed3f(z, -100.0f, 100.0f);
  return __builtin_fmaf(s * (1.0f - s), h, s);
}
__device__ __forceinline__ float act_gelu_slope(float z) {
  const float h = __builtin_amdgcn_fmed3f(z, -100.0f, 100.0f), q = h * h;
  const float s = act_sigmoid(z * __builtin_fmaf(kGeluB * kActLog2e, q, kGeluA * kActLog2e));
  return __builtin_fmaf(s * (1.0f - s), h * __builtin_fmaf(3.0f * kGeluB, q, kGeluA), s);
}

}  // namespace averis
