// rope_mfma.h -- matrix instructions, transposed LDS reads and LDS tiles of the attention kernels
// (library-internal, gfx950).
//
// Products are written transposed, so that a lane always owns one column (one query row, or in
// the key gradients one key row) of the result of a 32x32 tile:
//   C[i][j] += sum_k A[i][k] B[k][j]
//   A: lane l holds A[l % 32][8 (l / 32) .. + 7];  B: B[8 (l / 32) .. + 7][l % 32]
//   C: register r of lane l holds C[8 (r / 4) + 4 (l / 32) + r % 4][l % 32]
// (16x16 tiles: l % 16 and l / 16 in their place, 4 registers of C, rows 4 (l / 16) + r.)
// A product's C then serves, rounded to 16 bits, as the B of the next one without leaving the
// lane: registers 0..7 are one step of 16 k values, 8..15 the next, if the A operand takes its
// k values in the order of those rows -- 4 (l / 32) + {0..3, 8..11} -- which is what two
// transposed LDS reads of four rows deliver.
//
// An LDS tile is cut into panels of 64 elements (128 bytes) a row.  The eight 16-byte chunks of
// a row are permuted by the bit-reversed row number, so that neither 32 rows' reads of one chunk
// nor a transposed read of four rows meets in the same banks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ropeamd {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr float kNegInf = -__builtin_huge_valf();

template <typename T>
struct Mfma;

template <>
struct Mfma<__bf16> {
  __device__ static f32x16 mul(s16x8 a, s16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  __device__ static f32x4 mul16(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  __device__ static uint32_t pack(float x, float y) {
    f32x2_t v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
  }
  __device__ static float low(uint32_t w) { return __uint_as_float(w << 16); }
  __device__ static float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  // all exponent bits set in either half of a word: an infinity or a NaN
  __device__ static bool non_finite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
  }
};

template <>
struct Mfma<_Float16> {
  __device__ static f32x16 mul(s16x8 a, s16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  __device__ static f32x4 mul16(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  __device__ static uint32_t pack(float x, float y) {
    f32x2_t v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
  }
  __device__ static float low(uint32_t w) {
    return static_cast<float>(__builtin_bit_cast(f16x2_t, w).x);
  }
  __device__ static float high(uint32_t w) {
    return static_cast<float>(__builtin_bit_cast(f16x2_t, w).y);
  }
  __device__ static bool non_finite(uint32_t w) {
    return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
  }
};

__device__ inline s16x8 as_operand(uint4 v) { return __builtin_bit_cast(s16x8, v); }

// Eight floats of consecutive C registers, rounded to the operand type.
template <typename T>
__device__ inline s16x8 round8(const float *f) {
  return as_operand(make_uint4(Mfma<T>::pack(f[0], f[1]), Mfma<T>::pack(f[2], f[3]),
                               Mfma<T>::pack(f[4], f[5]), Mfma<T>::pack(f[6], f[7])));
}

// Permutation of a row's eight 16-byte chunks: chunk c of row r lies at c ^ chunk_key(r).
__device__ inline uint32_t chunk_key(uint32_t row) {
  return ((row & 1u) << 2) | (row & 2u) | ((row >> 2) & 1u);
}

// 16 bytes per lane from global memory straight into LDS: lane l's bytes land at lds + 16 l.
// `lds` is the same for all lanes of the wavefront.
__device__ inline void load_lds16(const void *g, void *lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)g,
                                   (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// Four rows of a 16-column block, transposed: lane i of each group of 16 points at row i / 4,
// columns 4 (i % 4) .. + 3, and receives column i of the four rows.
__device__ inline s16x4 read_transposed(const char *lds) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4 *)const_cast<char *>(lds));
}

__device__ inline s16x8 join(s16x4 a, s16x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Byte offset, inside a panel, of the 16-byte operand chunk `c` of row `row`.
__device__ inline uint32_t panel_chunk(uint32_t row, uint32_t c) {
  return row * 128u + ((c ^ chunk_key(row)) << 4);
}

// Byte offset, inside a panel, that a lane supplies for a transposed read of rows
// 4 (lane / 32) + {0..3} (+8, +16, ... rows: + 1024 bytes each) of the 32 columns of half
// `e` (0 or 1) of the panel.
__device__ inline uint32_t panel_transposed(uint32_t lane, uint32_t e) {
  const uint32_t i = lane & 15u;
  const uint32_t row = 4u * (lane >> 5) + (i >> 2);
  const uint32_t c = 4u * e + 2u * ((lane >> 4) & 1u) + ((i & 3u) >> 1);
  return row * 128u + ((c ^ chunk_key(row)) << 4) + (i & 1u) * 8u;
}

// Value held by the lane 32 away.
__device__ inline float other_half(float x) { return __shfl_xor(x, 32, 64); }

__device__ inline void wait_loads_all() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// Workgroup barrier that orders LDS accesses (direct-to-LDS loads are waited for separately).
__device__ inline void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace
}  // namespace ropeamd
