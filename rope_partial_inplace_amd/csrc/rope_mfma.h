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
// An LDS tile is cut into panels of 64 elements (128 bytes) a row: two rows are one pass over the
// 64 banks.  The eight 16-byte chunks of a row are permuted by a key so that no access meets
// itself in a bank (conflicts: none, or below 1% of the cycles): it takes all eight values over 16
// rows, which keeps 32 rows' reads of one chunk apart; it moves rows 0 and 2 (1 and 3) of four to
// different halves of a row, for the transposed reads; and it differs by 1 only between rows 12
// apart, for 16 rows' reads of two neighbouring chunks.
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

// kNarrow: the type's exponents end far inside float32's.  What is rounded to it between two products
// is multiplied by a power of two first, which a sum's store takes off again: exact, and neither
// small values become subnormal nor large ones infinite.
//
// kSlack, kLift: the weights of a row's softmax are 2^(s - top + kLift), and top, a maximum of
// earlier scores, is raised when one passes it by more than kSlack.  With 4 and 11 float16 (2^15 at
// most) keeps half a step down to 2^-25 of the largest weight.
template <typename T>
struct Mfma;

template <>
struct Mfma<__bf16> {
  static constexpr bool kNarrow = false;
  static constexpr float kSlack = 8.0f, kLift = 0.0f;
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
};

template <>
struct Mfma<_Float16> {
  static constexpr bool kNarrow = true;
  static constexpr float kSlack = 4.0f, kLift = 11.0f;
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
};

// Natural logarithm of the sum of a row's weights 2^(s - top + kLift).
template <typename T>
__device__ inline float natural(float top, float sum) {
  return (top - Mfma<T>::kLift) * 0.693147180559945f + logf(sum);
}

__device__ inline s16x8 as_operand(uint4 v) { return __builtin_bit_cast(s16x8, v); }

// Eight floats of consecutive C registers, rounded to the operand type.
template <typename T>
__device__ inline s16x8 round8(const float *f) {
  return as_operand(make_uint4(Mfma<T>::pack(f[0], f[1]), Mfma<T>::pack(f[2], f[3]),
                               Mfma<T>::pack(f[4], f[5]), Mfma<T>::pack(f[6], f[7])));
}

// Permutation of a row's eight 16-byte chunks: chunk c of row r lies at c ^ chunk_key(r).  Rows
// 16 apart share a key.
__device__ inline uint32_t chunk_key(uint32_t row) {
  return ((row & 2u) << 1) ^ ((row >> 1) & 2u) ^ (3u & (0u - ((row >> 3) & 1u)));
}

// Memory from `base` (the same for all lanes) on, addressed by 32-bit byte offsets.
__device__ inline __amdgpu_buffer_rsrc_t buffer_at(const void *base) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint64_t u = uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(b >> 32))))) << 32 |
                     uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(b))));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(u), 0, int(0xffffffff),
                                           0x00027000);
}

// 16 bytes per lane from global memory straight into LDS, from offset + uniform of the buffer:
// lane l's bytes land at lds + 16 l.  `lds` and `uniform` are the same for all lanes of the
// wavefront.  (Buffer loads: after the flat form, global_load_lds, the compiler cannot count LDS
// reads and waits for all of them before each use.)
__device__ inline void load_lds16(__amdgpu_buffer_rsrc_t buffer, uint32_t offset, int uniform,
                                  void *lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (__attribute__((address_space(3))) void *)lds,
                                           16, int(offset), uniform, 0, 0);
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
// 4 (lane / 32) + {0..3} + 8 `up` (+ 16, 32, ... rows: + 2048 bytes each) of the 32 columns of
// half `e` (0 or 1) of the panel.
__device__ inline uint32_t panel_transposed(uint32_t lane, uint32_t e, uint32_t up) {
  const uint32_t i = lane & 15u;
  const uint32_t row = 4u * (lane >> 5) + (i >> 2) + 8u * up;
  const uint32_t c = 4u * e + 2u * ((lane >> 4) & 1u) + ((i & 3u) >> 1);
  return row * 128u + ((c ^ chunk_key(row)) << 4) + (i & 1u) * 8u;
}

// What the place of row + 8 differs by from that of a row whose number has the bit 8 clear.
constexpr uint32_t kEightRows = 8u * 128u | 3u << 4;

// The operand of 16 rows (from a multiple of 16) of 32 columns, transposed: k values in the order
// 4 (lane / 32) + {0..3, 8..11}.
__device__ inline s16x8 transposed_operand(const char *panel, uint32_t lane, uint32_t e) {
  return join(read_transposed(panel + panel_transposed(lane, e, 0)),
              read_transposed(panel + panel_transposed(lane, e, 1)));
}

// Maximum and sum over the two lanes 32 apart, and (max16) over the four 16 apart.
__device__ inline float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ inline float max_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ inline float sum_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Inclusive sum over the wavefront: shifts within 16 lanes, then each row's last lane to the
// rows behind it.
__device__ inline int32_t wave_scan(int32_t x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

__device__ inline void wait_loads_all() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// Workgroup barrier that orders LDS accesses.  Direct-to-LDS loads are waited for separately:
// written as waits and a barrier, since a fence would wait for those under way as well.
__device__ inline void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace
}  // namespace ropeamd
