// Rows in pieces, reductions over neighbouring lanes and launches of many
// tokens, for the mixture-of-experts kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "gemm_common.hpp"

namespace averis {

constexpr float kMasked = -__builtin_inff();   // a closed expert's logit

// ---------------------------------------------------------------------------
// 16-byte pieces at element alignment: gfx950 loads and stores them at any
// address, so one path serves every stride and offset
// ---------------------------------------------------------------------------
typedef u32x4_t piece_t __attribute__((aligned(2)));

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {   // bf16 bits
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float f32(uint16_t v) { return bf16_lo(v); }
  static __device__ __forceinline__ uint16_t from(float v) { return (uint16_t)bf16x2_rne(v, 0.0f); }
  static __device__ __forceinline__ void unpack(u32x4_t p, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(p[i]);
      f[2 * i + 1] = bf16_hi(p[i]);
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    return u32x4_t{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                   bf16x2_rne(f[6], f[7])};
  }
};
template <>
struct Elem<float> {
  static constexpr int kPer = 4;
  static __device__ __forceinline__ float f32(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
  static __device__ __forceinline__ void unpack(u32x4_t p, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(p[i]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    return u32x4_t{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                   __float_as_uint(f[3])};
  }
};

// ---------------------------------------------------------------------------
// reductions over groups of G neighbouring lanes (butterflies: every lane of
// the group gets the result).  The mirrors pair the halves of 8 and 16 lanes
// once those halves agree.
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
  else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
  else if constexpr (D == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);
  else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);
  else return (uint32_t)__shfl_xor((int)v, D, 64);
}
template <int G, typename F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F op) {
  if constexpr (G > 1) v = op(v, partner<1>(v));
  if constexpr (G > 2) v = op(v, partner<2>(v));
  if constexpr (G > 4) v = op(v, partner<4>(v));
  if constexpr (G > 8) v = op(v, partner<8>(v));
  if constexpr (G > 16) v = op(v, partner<16>(v));
  if constexpr (G > 32) v = op(v, partner<32>(v));
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<G>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int G>
__device__ __forceinline__ float group_fmax(float v) {
  return __uint_as_float(group_reduce<G>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__builtin_fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}

// A grid has fewer than 2^32 threads (workgroups of 256 here): f(first, many)
// for each launch of n tokens, `per` of them a workgroup.
template <typename F>
static void in_launches(int64_t n, int64_t per, F f) {
  const int64_t most = ((1 << 24) - 1) * per;
  for (int64_t i = 0; i < n; i += most) f(i, n - i < most ? n - i : most);
}

}  // namespace averis
