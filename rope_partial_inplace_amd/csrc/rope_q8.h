// rope_q8.h -- 8-bit codes and their scales in device code (library-internal, gfx950).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "rope_plan.h"

namespace ropeamd {
namespace {

__device__ inline uint32_t div_by(const FastDiv &f, uint32_t n) {
  const uint32_t t = __umulhi(f.m, n);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}

// Size of x as a number that orders floats by it; infinities and NaN are the largest.
__device__ inline uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kNonFinite = 0x7f800000u;

// The scale that elements of size `top` need.  e4m3: the power of two 2^k with top <= 448 * 2^k, read off
// top's exponent and whether its fraction passes that of 448 = 1.75 * 2^8.
template <bool E4M3>
__device__ inline float needed_scale(float top) {
  if constexpr (E4M3) {
    const uint32_t u = __float_as_uint(top);
    const int32_t k = int32_t(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(uint32_t(max(k, -120) + 127) << 23);
  } else {
    return fmaxf(top * (1.0f / 127), 0x1p-120f);
  }
}

// Four floats within the codes' range to codes, to nearest even.  A NaN or infinity (CHECK: there may be
// some) becomes NaN in e4m3 and any code in int8, whose scale is then NaN.
//
// int8: added to 1.5 * 2^23 a float is rounded to an integer, whose low byte is the code.
template <bool E4M3, bool CHECK>
__device__ inline uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    if constexpr (CHECK) {
      auto one = [](float x) { return size_bits(x) < kNonFinite ? x : __builtin_nanf(""); };
      a = one(a), b = one(b), c = one(c), d = one(d);
    }
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
  } else {
    auto one = [](float x) { return __float_as_uint(x + 0x1.8p23f); };
    const uint32_t lo = __builtin_amdgcn_perm(one(b), one(a), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(one(d), one(c), 0x04000c0cu);
    return lo | hi;
  }
}

template <bool E4M3>
__device__ inline void decode4(uint32_t w, float *f) {
  if constexpr (E4M3) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    f[0] = lo[0];
    f[1] = lo[1];
    f[2] = hi[0];
    f[3] = hi[1];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = float(int8_t(w >> (8 * i)));
  }
}

// Four codes under a scale that is 1 / ratio times the old one.
template <bool E4M3>
__device__ inline uint32_t recode(uint32_t w, float ratio) {
  float f[4];
  decode4<E4M3>(w, f);
  return encode4<E4M3, true>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// V = 1, 4 or 8 codes of f * inv.
template <bool E4M3, bool CHECK, int V>
__device__ inline void store_codes(uint8_t *to, const float *f, float inv) {
  if constexpr (V == 1) {
    *to = uint8_t(encode4<E4M3, CHECK>(f[0] * inv, 0.0f, 0.0f, 0.0f));
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      w[i] = encode4<E4M3, CHECK>(f[4 * i] * inv, f[4 * i + 1] * inv, f[4 * i + 2] * inv,
                                  f[4 * i + 3] * inv);
    if constexpr (V == 4)
      *reinterpret_cast<uint32_t *>(to) = w[0];
    else
      *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
  }
}

}  // namespace
}  // namespace ropeamd
