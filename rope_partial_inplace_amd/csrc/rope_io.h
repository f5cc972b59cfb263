// rope_io.h -- storage types of the device code of librope_amd.so (library-internal).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ropeamd {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// ---- storage types <-> float32 ------------------------------------------------------------
// Decoding is exact; encoding rounds to nearest even (gfx950's v_cvt_pk_bf16_f32 and
// v_cvt_f16_f32 under the default round-to-nearest-even mode).

template <typename T>
struct Io;

template <>
struct Io<float> {
  static constexpr int kPer16 = 4;
  static constexpr int kPerWord = 1;
  using raw = uint32_t;
  __device__ static void word_to_floats(uint32_t w, float *f) { f[0] = __uint_as_float(w); }
  __device__ static uint32_t floats_to_word(const float *f) { return __float_as_uint(f[0]); }
  __device__ static void unpack(const uint4 &v, float *f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ static uint4 pack(const float *f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  __device__ static float from_raw(raw r) { return __uint_as_float(r); }
  __device__ static float load1(const void *p, int64_t i) {
    return static_cast<const float *>(p)[i];
  }
  __device__ static void store1(void *p, int64_t i, float v) { static_cast<float *>(p)[i] = v; }
};

template <>
struct Io<__bf16> {
  static constexpr int kPer16 = 8;
  static constexpr int kPerWord = 2;
  using raw = uint16_t;
  __device__ static void word_to_floats(uint32_t w, float *f) { unpack_word(w, f); }
  __device__ static uint32_t floats_to_word(const float *f) { return pack_word(f[0], f[1]); }
  __device__ static void unpack_word(uint32_t w, float *f) {
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
  }
  __device__ static uint32_t pack_word(float a, float b) {
    f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
  __device__ static void unpack(const uint4 &v, float *f) {
    unpack_word(v.x, f);
    unpack_word(v.y, f + 2);
    unpack_word(v.z, f + 4);
    unpack_word(v.w, f + 6);
  }
  __device__ static uint4 pack(const float *f) {
    return make_uint4(pack_word(f[0], f[1]), pack_word(f[2], f[3]), pack_word(f[4], f[5]),
                      pack_word(f[6], f[7]));
  }
  __device__ static float from_raw(raw r) { return __uint_as_float(uint32_t(r) << 16); }
  __device__ static float load1(const void *p, int64_t i) {
    return from_raw(static_cast<const uint16_t *>(p)[i]);
  }
  __device__ static void store1(void *p, int64_t i, float v) {
    static_cast<uint16_t *>(p)[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
};

template <>
struct Io<_Float16> {
  static constexpr int kPer16 = 8;
  static constexpr int kPerWord = 2;
  using raw = uint16_t;
  __device__ static void word_to_floats(uint32_t w, float *f) { unpack_word(w, f); }
  __device__ static uint32_t floats_to_word(const float *f) { return pack_word(f[0], f[1]); }
  __device__ static void unpack_word(uint32_t w, float *f) {
    f16x2 h = __builtin_bit_cast(f16x2, w);
    f[0] = static_cast<float>(h.x);
    f[1] = static_cast<float>(h.y);
  }
  __device__ static uint32_t pack_word(float a, float b) {
    f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  }
  __device__ static void unpack(const uint4 &v, float *f) {
    unpack_word(v.x, f);
    unpack_word(v.y, f + 2);
    unpack_word(v.z, f + 4);
    unpack_word(v.w, f + 6);
  }
  __device__ static uint4 pack(const float *f) {
    return make_uint4(pack_word(f[0], f[1]), pack_word(f[2], f[3]), pack_word(f[4], f[5]),
                      pack_word(f[6], f[7]));
  }
  __device__ static float from_raw(raw r) {
    return static_cast<float>(__builtin_bit_cast(_Float16, r));
  }
  __device__ static float load1(const void *p, int64_t i) {
    return static_cast<float>(static_cast<const _Float16 *>(p)[i]);
  }
  __device__ static void store1(void *p, int64_t i, float v) {
    static_cast<_Float16 *>(p)[i] = static_cast<_Float16>(v);
  }
};

}  // namespace
}  // namespace ropeamd
