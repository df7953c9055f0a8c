// Eight consecutive elements of a row in registers, and their codes (fp8_common.hpp).
#pragma once

#include "fp8_common.hpp"

namespace averis {

// eight consecutive elements of a row, as loaded
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  u32x4_t w;
  __device__ __forceinline__ void zero() { w = u32x4_t{0u, 0u, 0u, 0u}; }
  // elements c .. c + 7 of a row of cols elements, 0 past its end
  __device__ __forceinline__ void load(const uint16_t* row, int64_t c, int64_t cols) {
    if (c + 8 <= cols) {
      w = *reinterpret_cast<const f8_piece_t*>(row + c);
      return;
    }
    zero();
    if (c >= cols) return;
    // all loads at once, those past the end of the last element (one by one, each
    // behind its own branch: 16384 x 3071 53.7 us instead of 47.0)
    uint16_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = row[c + i < cols ? c + i : cols - 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 2] |= (c + i < cols ? (uint32_t)e[i] : 0u) << (16 * (i & 1));
  }
  // bits of the largest magnitude, as fp32
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t k = 0x7FFF7FFFu;
    const uint32_t m = pk_max_u16(pk_max_u16(w[0] & k, w[1] & k), pk_max_u16(w[2] & k, w[3] & k));
    const uint32_t lo = m << 16, hi = m & 0xFFFF0000u;
    return lo > hi ? lo : hi;
  }
  __device__ __forceinline__ u32x2_t codes(uint32_t byte) const {
    return u32x2_t{f8_codes4_bf16(w[0], w[1], byte), f8_codes4_bf16(w[2], w[3], byte)};
  }
  __device__ __forceinline__ void f32(float* f) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  // rounded to nearest, ties to even
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16x2_rne(f[2 * i], f[2 * i + 1]);
  }
  // to elements c .. c + 7 of a row, those past its end left out
  __device__ __forceinline__ void store(uint16_t* row, int64_t c, int64_t cols) const {
    if (c + 8 <= cols) {
      *reinterpret_cast<f8_piece_t*>(row + c) = w;
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
};
template <>
struct Eight<float> {
  u32x4_t w[2];
  __device__ __forceinline__ void zero() { w[0] = w[1] = u32x4_t{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void load(const float* row, int64_t c, int64_t cols) {
    if (c + 8 <= cols) {
      w[0] = *reinterpret_cast<const f8_piece_t*>(row + c);
      w[1] = *reinterpret_cast<const f8_piece_t*>(row + c + 4);
      return;
    }
    zero();
    if (c >= cols) return;
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = row[c + i < cols ? c + i : cols - 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4][i % 4] = c + i < cols ? __float_as_uint(e[i]) : 0u;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t a = w[i / 4][i % 4] & 0x7FFFFFFFu;
      m = a > m ? a : m;
    }
    return m;
  }
  __device__ __forceinline__ u32x2_t codes(uint32_t byte) const {
    auto f = [&](int i) { return __uint_as_float(w[i / 4][i % 4]); };
    return u32x2_t{f8_codes4(f(0), f(1), f(2), f(3), byte), f8_codes4(f(4), f(5), f(6), f(7), byte)};
  }
  __device__ __forceinline__ void f32(float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i / 4][i % 4]);
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4][i % 4] = __float_as_uint(f[i]);
  }
  __device__ __forceinline__ void store(float* row, int64_t c, int64_t cols) const {
    if (c + 8 <= cols) {
      *reinterpret_cast<f8_piece_t*>(row + c) = w[0];
      *reinterpret_cast<f8_piece_t*>(row + c + 4) = w[1];
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = __uint_as_float(w[i / 4][i % 4]);
  }
};

// elements c .. c + 7 of a vector in F32 or BF16, as fp32 (0 past its end)
__device__ __forceinline__ void load_vector(const void* p, bool bf16, int64_t c, int64_t n, float* f) {
  if (bf16) {
    Eight<uint16_t> v;
    v.load(static_cast<const uint16_t*>(p), c, n);
    v.f32(f);
  } else {
    Eight<float> v;
    v.load(static_cast<const float*>(p), c, n);
    v.f32(f);
  }
}

template <typename T>
__device__ __forceinline__ u32x2_t eight_codes(const Eight<T>& v, uint32_t amax, uint32_t& byte) {
  byte = f8_scale_byte(amax);
  if (__builtin_expect(f8_not_finite(amax), 0)) {
    byte = kF8One;
    return u32x2_t{kF8NanCodes, kF8NanCodes};
  }
  return v.codes(byte);
}

// the codes of eight elements from column c on, those past the row's end 0
__device__ __forceinline__ u32x2_t without_pad(u32x2_t q, int64_t c, int64_t cols) {
  const int left = (int)(cols - c < 8 ? cols - c : 8);
  return u32x2_t{f8_without_pad(q[0], left), f8_without_pad(q[1], left - 4)};
}

}  // namespace averis
