// The activations of a product's epilogue and of the way back through it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace averis {

// silu(z) = z s(z) and gelu(z) = z s(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3), with s(u) = 1 / (1 +
// e^-u): the tanh form of gelu, for (1 + tanh(v)) / 2 = s(2 v).  Both as z s(z (a + b z^2)).  e^-u and
// the reciprocal are single instructions (an error of 1 ulp each).
struct ActSigmoid {
  float a, b;   // of u in units of log 2
  float a1, b1;   // of du / dz
  __device__ __forceinline__ explicit ActSigmoid(int act) {
    const float k = 1.5957691216057308f, c = k * 0.044715f, log2e = 1.4426950408889634f;
    a1 = act == kActGelu ? k : 1.0f;
    b1 = act == kActGelu ? 3.0f * c : 0.0f;
    a = act == kActGelu ? k * log2e : log2e;
    b = act == kActGelu ? c * log2e : 0.0f;
  }
  // |z| past 100 changes nothing, and z^2 might overflow (a NaN z is not seen here: the products below
  // with z keep it)
  __device__ __forceinline__ float sigmoid(float z) const {
    z = __builtin_amdgcn_fmed3f(z, -100.0f, 100.0f);
    const float u = z * __builtin_fmaf(b, z * z, a);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-u));
  }
  __device__ __forceinline__ float value(float z) const { return z * sigmoid(z); }
  // s + z s (1 - s) du/dz, past |z| = 100 its limit, 1 or 0
  __device__ __forceinline__ float slope(float z) const {
    z = z > 100.0f ? 100.0f : z < -100.0f ? -100.0f : z;
    const float s = sigmoid(z);
    return __builtin_fmaf(z * s * (1.0f - s), __builtin_fmaf(b1, z * z, a1), s);
  }
};

}  // namespace averis
