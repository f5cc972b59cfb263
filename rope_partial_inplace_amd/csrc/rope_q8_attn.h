// rope_q8_attn.h -- grouped-query attention over a paged cache of 8-bit codes (gfx950): the kernel,
// instantiated for bfloat16 and float16 queries by two sources (library-internal).
//
//   s_j = scale ks_j <q, kc_j>,   p = softmax(s),   out = sum_j p_j vs_j vc_j
// with codes kc, vc and a float32 scale ks, vs for each block of tokens and head.  A query head reads
// the tokens of its key head; the heads of a group share them, so a token's 2 D bytes are read from
// HBM once for up to 32 (token, head) rows: 4 D operations a row and token leave decoding bound by HBM.
//
// One pass, running maximum and sum in float32.  Codes go from HBM straight to registers, in the
// layout in which the matrix instructions take them, and are made operands there: exact in bfloat16
// and float16 both, so the scales can wait -- ks multiplies the finished scores, vs the weights,
// before those are rounded for the second product.  No LDS and no barrier stand between a load and its use: a
// wavefront takes 32 tokens at a time and has the next 32 under way (8 KB at D 128).  The four wavefronts
// of a workgroup take up to four key heads of the same tokens; those of one head, each of which
// takes every n-th 32 tokens, join their sums at the end.
//
// Measured with 8 key heads of 128: 64 sequences of 200-9000 tokens 63 us (284 MB), of 9000 201 us
// (5.9 TB/s), six of 60-131k tokens and a scale for each 255 us (5.6 TB/s).
//
// Layout (16x16x32 products, lane l = 16 g + c):
//   S^T = K Q^T: A[key c][8 d], lane's d = g D / 4 + 16 i + 8 e + 0..7 for product (i, e): 16 bytes a load
//   and two products, and each load touches whole 128-byte lines; register r of S^T: key 4 g + r of query row c.
//   O^T = V^T P^T: the lane's eight keys are those of its two S^T registers sets, 4 g + r and
//   16 + 4 g + r, so P stays where it was computed; it loads D / 16 neighbouring bytes of each of the
//   eight tokens (16 lanes: a whole row) and turns them: column t of the eight is the A operand of
//   output d = c D / 16 + t.  A lane of O^T holds d = (4 g + r) D / 16 + t of query row c.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "rope.h"
#include "rope_launch.h"
#include "rope_mfma.h"
#include "rope_q8.h"
#include "rope_q8_plan.h"

namespace ropeamd {
namespace {

constexpr int kAttnBlock = 256;
constexpr int kAttnWaves = kAttnBlock / 64;
constexpr int kTile = 32;  // tokens of a wavefront at a time
static_assert(kTile * kAttnWaves == 1 << q8_step_log2(16, 64, 0), "a step is a tile of every wavefront");

// What beginning an item costs, in steps: the shares of the workgroups are cut by steps and this.
constexpr int32_t kQ8ItemCost = 2;

// Codes to operands of type T.
template <typename T, bool E4M3>
struct Operand;

template <typename T>
struct Operand<T, true> {
  // two codes, bytes 2 `high` and 2 `high` + 1 of w
  template <bool HIGH>
  __device__ static uint32_t pair(uint32_t w) {
    if constexpr (Mfma<T>::kNarrow)
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(int(w), 1.0f, HIGH));
    else
      return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(int(w), 1.0f, HIGH));
  }
  __device__ static s16x8 row(uint32_t w0, uint32_t w1) {
    return as_operand(make_uint4(pair<false>(w0), pair<true>(w0), pair<false>(w1), pair<true>(w1)));
  }
  // bytes 2 `HIGH` and 2 `HIGH` + 1 of eight words, as two operands
  template <bool HIGH>
  __device__ static void columns(const uint32_t (&w)[8], s16x8 *a, s16x8 *b) {
    uint32_t c[8], x[4], y[4];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = pair<HIGH>(w[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = __builtin_amdgcn_perm(c[2 * j + 1], c[2 * j], 0x05040100u);
      y[j] = __builtin_amdgcn_perm(c[2 * j + 1], c[2 * j], 0x07060302u);
    }
    *a = as_operand(make_uint4(x[0], x[1], x[2], x[3]));
    *b = as_operand(make_uint4(y[0], y[1], y[2], y[3]));
  }
};

template <typename T>
struct Operand<T, false> {
  // the byte B of w0 and w1
  template <int B0, int B1>
  __device__ static uint32_t two(uint32_t w0, uint32_t w1) {
    if constexpr (Mfma<T>::kNarrow) {
      // 1024 + 128 + code in float16: the code, its sign bit turned, are the low bits of 1024 + ..
      constexpr uint32_t sel = 0x0c000c00u | uint32_t(4 + B1) << 16 | uint32_t(B0);
      const uint32_t u = __builtin_amdgcn_perm(w1, w0, sel) ^ 0x64806480u;
      const f16x2_t v = __builtin_bit_cast(f16x2_t, u) + f16x2_t{_Float16(-1152), _Float16(-1152)};
      return __builtin_bit_cast(uint32_t, v);
    } else {  // a code has at most 8 significant bits: a float's upper half holds it
      const float a = float(int8_t(w0 >> (8 * B0))), b = float(int8_t(w1 >> (8 * B1)));
      return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    }
  }
  __device__ static s16x8 row(uint32_t w0, uint32_t w1) {
    return as_operand(make_uint4(two<0, 1>(w0, w0), two<2, 3>(w0, w0), two<0, 1>(w1, w1),
                                 two<2, 3>(w1, w1)));
  }
  template <bool HIGH>
  __device__ static void columns(const uint32_t (&w)[8], s16x8 *a, s16x8 *b) {
    constexpr int B = HIGH ? 2 : 0;
    *a = as_operand(make_uint4(two<B, B>(w[0], w[1]), two<B, B>(w[2], w[3]),
                               two<B, B>(w[4], w[5]), two<B, B>(w[6], w[7])));
    *b = as_operand(make_uint4(two<B + 1, B + 1>(w[0], w[1]), two<B + 1, B + 1>(w[2], w[3]),
                               two<B + 1, B + 1>(w[4], w[5]), two<B + 1, B + 1>(w[6], w[7])));
  }
};

// Values that are NaN.  A product makes a NaN of 0 times one, and a token's codes are an operand for all rows.  So
// that a NaN stays with the rows that see its token, in tiles that some rows see in part its code becomes that
// of -0 (and -0 that of 0, which no sum tells apart) before the product, and outputs become NaN by a
// product that counts, for each of them, the NaN that its row sees.

// Four e4m3 codes so; not 0 where one was a NaN (a size of 127).
__device__ inline uint32_t mark_nans(uint32_t *w) {
  const uint32_t size = *w & 0x7f7f7f7fu;
  const uint32_t nans = (size + 0x01010101u) & 0x80808080u, some = (size + 0x7f7f7f7fu) & 0x80808080u;
  *w = ((size | (*w & some)) & ~((nans >> 7) * 0xffu)) | nans;
  return nans;
}

// An operand with 1 for each -0 of another and 0 elsewhere.
template <typename T>
__device__ inline s16x8 marked(s16x8 x) {
  auto ones = [](uint32_t w) {
    const uint32_t turned = w ^ 0x80008000u;
    const uint32_t other = ((turned & 0x7fff7fffu) + 0x7fff7fffu) | turned;  // top bits: not a -0
    return ((~other & 0x80008000u) >> 15) * (Mfma<T>::kNarrow ? 0x3c00u : 0x3f80u);
  };
  const uint4 w = __builtin_bit_cast(uint4, x);
  return as_operand(make_uint4(ones(w.x), ones(w.y), ones(w.z), ones(w.w)));
}

// What a sequence asks for: its query rows (token by token, the heads of a group one after the other) in
// tiles.  A tile's steps end with the last token that one of its rows sees, so of causal rows a later
// tile has more steps; the k-th tile from the end and the k-th from the front make a pair, and all
// pairs, of every key head, cost alike.
struct SequenceQ8 {
  int32_t len, first, count;  // cached tokens; first query token, query tokens (below 0: descending)
  int32_t tiles;
  int32_t cost;               // of a pair
  __device__ int32_t pairs() const { return (tiles + 1) / 2; }
};

template <int ROWS>
struct WorkQ8 {
  const AttnQ8Plan &p;

  // Tokens that the last row of a tile sees, and its steps.
  __device__ int32_t visible(const SequenceQ8 &s, int32_t tile) const {
    const int32_t rows = s.count * p.group;
    const int32_t tok = int32_t(div_by(p.div_group, uint32_t(min((tile + 1) * ROWS, rows) - 1)));
    return max(0, s.len - s.count + 1 + tok);
  }
  __device__ int32_t steps(const SequenceQ8 &s, int32_t tile) const {
    return max(1, (visible(s, tile) + (1 << p.step_log2) - 1) >> p.step_log2);
  }
  // Lengths and offsets are device data: values outside their ranges are clamped.
  __device__ SequenceQ8 sequence(int32_t b) const {
    const Sequences &q = p.seq;
    SequenceQ8 s;
    s.len = int32_t(min(max(q.lens[b * q.len_stride], int64_t(0)), q.max_pages * q.page_size));
    if (q.offsets != nullptr) {
      const int64_t o0 = min(max(q.offsets[b * q.off_stride], int64_t(0)), q.T);
      const int64_t o1 = min(max(q.offsets[(b + 1) * q.off_stride], int64_t(0)), q.T);
      s.first = int32_t(o0);
      s.count = int32_t(o1 - o0);
    } else {
      s.first = int32_t(b * q.each);
      s.count = int32_t(q.each);
    }
    s.tiles = (max(s.count, 0) * p.group + ROWS - 1) / ROWS;
    s.cost = 0;
    if (s.tiles > 0) {
      s.cost = steps(s, s.tiles - 1) + kQ8ItemCost;
      // the first tile beside the last; other pairs see up to ROWS rows' tokens more than this one
      if (s.tiles > 1) s.cost += steps(s, 0) + kQ8ItemCost + (ROWS >> p.step_log2) + 2;
    }
    return s;
  }
  __device__ int64_t cost(const SequenceQ8 &s) const {
    return int64_t(s.pairs()) * p.head_sets * s.cost;
  }
};

// How a tile's tokens are found.  kCoarse: pages of whole runs of 16 tokens and scales of whole runs of 4: a
// half tile lies in one page, whose number is the same for all lanes, and a lane's four neighbouring
// tokens under one scale.  kFine: such pages, any scales: a lane reads those of one token, and the others'
// come from its neighbours.  kAny: pages of any size, too.
enum { kAny = 0, kFine = 1, kCoarse = 2 };

// Keys, or values, of 32 tokens: a lane's codes, and its tokens' scales.
template <int D, int MODE>
struct KeysQ8 {
  uint4 code[2][D / 64];
  float scale[MODE == kCoarse ? 2 : 1];
};
template <int D, int MODE>
struct ValuesQ8 {
  uint32_t code[8][D / 64];
  float scale[MODE == kCoarse ? 2 : 1];
};

// Scale of the lane's token j of eight: 16 (j / 4) + 4 g + j % 4 of the tile.
template <int MODE>
__device__ __forceinline__ float scale_of(const float *s, int j, int lane) {
  if constexpr (MODE == kCoarse) return s[j / 4];
  return __shfl(s[0], 16 * (j / 4) + 4 * (lane >> 4) + j % 4);
}

// Where a tile lies: the pages of its halves, or the page and row of a token a lane.
template <int MODE>
struct WhereQ8 {
  int64_t page[2];
};
template <>
struct WhereQ8<kAny> {
  int32_t page, row;
};

__device__ inline int64_t page_of(const Sequences &s, int32_t b, int32_t index) {
  const int64_t id = s.table[b * s.table_seq + index * s.table_page];
  return min(max(id, int64_t(0)), s.num_pages - 1);
}

// Tokens past the last one (`last`) repeat it.
template <int MODE>
__device__ __forceinline__ WhereQ8<MODE> locate(const Sequences &s, int32_t b, int32_t t0,
                                                int32_t last, int lane) {
  WhereQ8<MODE> w;
  if constexpr (MODE != kAny) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w.page[h] = page_of(s, b, int32_t(div_by(s.div_page, uint32_t(min(t0 + 16 * h, last)))));
  } else {
    const uint32_t t = uint32_t(min(t0 + (lane & 31), last));
    const uint32_t i = div_by(s.div_page, t);
    w.page = int32_t(page_of(s, b, int32_t(i)));
    w.row = int32_t(t - i * uint32_t(s.page_size));
  }
  return w;
}

// W words of a row that 16 lanes load whole.  Whole lines are loaded past the caches, which no other load
// wants them from: 64 sequences 66.8 -> 62.5 us, six of 60-131k tokens 275 -> 254 (plain loads of dense memory
// end at 6.2 TB/s on this card, such ones at 7.0).  Half lines (heads of 64) are not, and neither are keys, two
// loads of which share a line: they came twice (254 -> 270).
template <int W>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = *reinterpret_cast<const uint32_t *>(p);
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    const words x = __builtin_nontemporal_load(reinterpret_cast<const words *>(p));
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = x[i];
  }
}

// Half h of a tile in one page: its first row there, and how many tokens follow that row's.
struct HalfQ8 {
  int32_t row, more;
};
__device__ __forceinline__ HalfQ8 half_of(const Sequences &s, int32_t t0, int h, int32_t last) {
  const int32_t begin = min(t0 + 16 * h, last);
  return {begin - int32_t(div_by(s.div_page, uint32_t(begin)) * uint32_t(s.page_size)), last - begin};
}

// The scales of a tile whose halves lie in one page each.
template <int MODE>
__device__ __forceinline__ void load_scales(const AttnQ8Plan &p, const Q8Cache &c,
                                            const WhereQ8<MODE> &w, int32_t t0, int32_t last,
                                            int64_t head, int lane, float *scale) {
  if constexpr (MODE == kCoarse) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const HalfQ8 x = half_of(p.seq, t0, h, last);
      const int64_t block = div_by(p.div_block, uint32_t(x.row + min(4 * (lane >> 4), x.more)));
      scale[h] = c.scales[w.page[h] * c.s_page + head * c.s_head + block * c.s_block];
    }
  } else if constexpr (MODE == kFine) {
    const HalfQ8 a = half_of(p.seq, t0, 0, last), b = half_of(p.seq, t0, 1, last);
    const bool up = (lane & 16) != 0;
    const int32_t row = (up ? b.row : a.row) + min(lane & 15, up ? b.more : a.more);
    const int64_t block = div_by(p.div_block, uint32_t(row));
    scale[0] = c.scales[(up ? w.page[1] : w.page[0]) * c.s_page + head * c.s_head + block * c.s_block];
  } else {
    const int64_t block = div_by(p.div_block, uint32_t(w.row));
    scale[0] = c.scales[w.page * c.s_page + head * c.s_head + block * c.s_block];
  }
}

template <int D, int MODE>
__device__ __forceinline__ void load_keys(const AttnQ8Plan &p, const WhereQ8<MODE> &w, int32_t t0,
                                          int32_t last, int64_t head, int lane,
                                          KeysQ8<D, MODE> &k) {
  const int c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t *from;
    uint32_t at = 0;
    if constexpr (MODE != kAny) {
      const HalfQ8 x = half_of(p.seq, t0, h, last);
      from = p.k.codes + w.page[h] * p.k.page + head * p.k.head + int64_t(x.row) * p.k.row;
      at = uint32_t(min(c, x.more) * p.k.row + D / 4 * g);
    } else {
      const int64_t page = __shfl(w.page, 16 * h + c), row = __shfl(w.row, 16 * h + c);
      from = p.k.codes + page * p.k.page + head * p.k.head + row * p.k.row + D / 4 * g;
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
      k.code[h][i] = *reinterpret_cast<const uint4 *>(from + (at + 16 * i));
  }
  load_scales<MODE>(p, p.k, w, t0, last, head, lane, k.scale);
}

template <int D, int MODE>
__device__ __forceinline__ void load_values(const AttnQ8Plan &p, const WhereQ8<MODE> &w, int32_t t0,
                                            int32_t last, int64_t head, int lane,
                                            ValuesQ8<D, MODE> &v) {
  const int c = lane & 15, g = lane >> 4;
  if constexpr (MODE != kAny) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const HalfQ8 x = half_of(p.seq, t0, h, last);
      const uint8_t *from =
          p.v.codes + w.page[h] * p.v.page + head * p.v.head + int64_t(x.row) * p.v.row;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        load_words(from + uint32_t(min(4 * g + j, x.more) * p.v.row + c * (D / 16)),
                   v.code[4 * h + j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int key = 16 * (j / 4) + 4 * g + j % 4;
      const int64_t page = __shfl(w.page, key), row = __shfl(w.row, key);
      load_words(p.v.codes + page * p.v.page + head * p.v.head + row * p.v.row + c * (D / 16),
                 v.code[j]);
    }
  }
  load_scales<MODE>(p, p.v, w, t0, last, head, lane, v.scale);
}

// The power of two above x >= 0, within those whose reciprocal is one, too; and that of such a power.
__device__ inline float reach_above(float x) {
  return __uint_as_float((min(max(__float_as_uint(x) >> 23, 1u), 252u) + 1u) << 23);
}
__device__ inline float inverse_power(float x) {
  return __uint_as_float((254u << 23) - __float_as_uint(x));
}

// A wavefront's running state for R tiles of 16 query rows; the lane's row of a tile is row c.
template <typename T, int D, int R>
struct StateQ8 {
  s16x8 q[R][D / 32];
  f32x4 o[R][D / 16];
  float top[R], sum[R];
  int32_t limit[R];  // tokens that the lane's row may see
  // float16: the weights p vs have to stay in its range, so a row takes vs relative to a power of two above the
  // largest one that it has seen, its reach; this is the reciprocal
  float by_reach[R];
};
constexpr float kFirstByReach = 0x1p120f;  // of the smallest scale

// Scores of a tile in powers of two, masked where not every row sees all of it (t0 + 32 above `floor`).
template <typename T, int D, int R, bool E4M3, int MODE>
__device__ __forceinline__ void score_tile(const KeysQ8<D, MODE> &k, const StateQ8<T, D, R> &s,
                                           int32_t t0, int32_t floor, float scale_log2, int lane,
                                           f32x4 (&x)[R][2]) {
  const int g = lane >> 4;
  using Op = Operand<T, E4M3>;
#pragma unroll
  for (int r = 0; r < R; ++r) x[r][0] = x[r][1] = f32x4{};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint4 w = k.code[h][i];
      const s16x8 a = Op::row(w.x, w.y), b = Op::row(w.z, w.w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[r][h] = Mfma<T>::mul16(a, s.q[r][2 * i], x[r][h]);
        x[r][h] = Mfma<T>::mul16(b, s.q[r][2 * i + 1], x[r][h]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = scale_of<MODE>(k.scale, j, lane) * scale_log2;
#pragma unroll
    for (int r = 0; r < R; ++r) x[r][j / 4][j % 4] *= f;
  }
  if (t0 + kTile > floor) {
    asm volatile("");  // a branch: most tiles need no masks
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (t0 + 16 * (j / 4) + 4 * g + j % 4 >= s.limit[r]) x[r][j / 4][j % 4] = kNegInf;
  }
}

// Marks NaN among a tile's values; outputs of rows that see one become NaN.
template <typename T, int D, int R, int MODE>
__device__ __forceinline__ void part_nans(ValuesQ8<D, MODE> &v, StateQ8<T, D, R> &s, int32_t t0, int lane) {
  uint32_t found = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < D / 64; ++i) found |= mark_nans(&v.code[j][i]);
  if (!__any(found != 0)) return;
  s16x8 seen[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float one[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      one[j] = t0 + 16 * (j / 4) + 4 * (lane >> 4) + j % 4 < s.limit[r] ? 1.0f : 0.0f;
    seen[r] = round8<T>(one);
  }
  auto count = [&](int n, const s16x8 &a) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const f32x4 nans = Mfma<T>::mul16(marked<T>(a), seen[r], f32x4{});
#pragma unroll
      for (int k = 0; k < 4; ++k) s.o[r][n][k] = nans[k] > 0.0f ? __builtin_nanf("") : s.o[r][n][k];
    }
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = v.code[j][i];
    s16x8 a, b;
    Operand<T, true>::template columns<false>(c, &a, &b);
    count(4 * i, a);
    count(4 * i + 1, b);
    Operand<T, true>::template columns<true>(c, &a, &b);
    count(4 * i + 2, a);
    count(4 * i + 3, b);
  }
}

// The weights of a tile, at maxima that are raised where a score passes one by more than kSlack (until
// then larger weights are carried, which changes no result beyond its rounding), and
// O^T += V^T P^T.
template <typename T, int D, int R, bool E4M3, int MODE>
__device__ __forceinline__ void weigh_tile(const ValuesQ8<D, MODE> &v, StateQ8<T, D, R> &s,
                                           int32_t t0, int32_t floor, int lane,
                                           const f32x4 (&x)[R][2]) {
  const int g = lane >> 4;
  const bool masked = t0 + kTile > floor;
  float best[R];
  bool raise = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float m = x[r][0][0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, x[r][j / 4][j % 4]);
    best[r] = max_quarters(m);
    raise |= best[r] > s.top[r] + Mfma<T>::kSlack;
  }
  constexpr int SC = MODE == kCoarse ? 2 : 1;
  float most[R];  // float16: the largest vs of the lane's tokens, of those that its rows see where some do not
  if constexpr (Mfma<T>::kNarrow) {
#pragma unroll
    for (int r = 0; r < R; ++r) most[r] = fmaxf(fabsf(v.scale[0]), fabsf(v.scale[SC - 1]));
    if (masked) {
      asm volatile("");
#pragma unroll
      for (int r = 0; r < R; ++r) most[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float vs = fabsf(scale_of<MODE>(v.scale, j, lane));
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (t0 + 16 * (j / 4) + 4 * g + j % 4 < s.limit[r]) most[r] = fmaxf(most[r], vs);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) raise |= most[r] * s.by_reach[r] > 1.0f;
  }
  if (__any(raise)) {
    float all = 0.0f;  // of the tile, which every row sees
    if constexpr (Mfma<T>::kNarrow) {
      if (!masked) {
        all = most[0];
        for (int d = 1; d < 64; d *= 2) all = fmaxf(all, __shfl_xor(all, d));
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f = 1.0f;
      if (best[r] > s.top[r] + Mfma<T>::kSlack) {
        f = __builtin_amdgcn_exp2f(s.top[r] - best[r]);
        s.top[r] = best[r];
      }
      s.sum[r] *= f;
      if constexpr (Mfma<T>::kNarrow) {
        const float seen = masked ? max_quarters(most[r]) : all;
        const float by = seen * s.by_reach[r] > 1.0f ? inverse_power(reach_above(seen)) : s.by_reach[r];
        f *= by * inverse_power(s.by_reach[r]);
        s.by_reach[r] = by;
      }
#pragma unroll
      for (int n = 0; n < D / 16; ++n) s.o[r][n] *= f;
    }
  }
  float e[R][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float scale = scale_of<MODE>(v.scale, j, lane);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float vs = Mfma<T>::kNarrow ? scale * s.by_reach[r] : scale;
      const float ref = s.top[r] == kNegInf ? 0.0f : s.top[r] - Mfma<T>::kLift;
      const float y = __builtin_amdgcn_exp2f(x[r][j / 4][j % 4] - ref);
      s.sum[r] += y;
      e[r][j] = y * vs;
    }
  }
  if (masked) {
    asm volatile("");
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j)  // whatever the scale of a token that the row does not see
        if (t0 + 16 * (j / 4) + 4 * g + j % 4 >= s.limit[r]) e[r][j] = 0.0f;
  }
  s16x8 w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = round8<T>(e[r]);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = v.code[j][i];
    auto multiply = [&](int n, const s16x8 &a, const s16x8 &b) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s.o[r][n] = Mfma<T>::mul16(a, w[r], s.o[r][n]);
        s.o[r][n + 1] = Mfma<T>::mul16(b, w[r], s.o[r][n + 1]);
      }
      __builtin_amdgcn_sched_barrier(0);  // or the compiler converts everything first, and spills
    };
    s16x8 a, b;
    Operand<T, E4M3>::template columns<false>(c, &a, &b);
    multiply(4 * i, a, b);
    Operand<T, E4M3>::template columns<true>(c, &a, &b);
    multiply(4 * i + 2, a, b);
  }
}

// Sum over the workgroup's threads before this one, and of all (in `total`).  SMALL: sums fit 31 bits.
template <bool SMALL>
__device__ inline int64_t block_scan(int64_t x, int64_t *lds, int64_t *total) {
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  int64_t incl = x;
  if constexpr (SMALL) {
    incl = wave_scan(int32_t(x));
  } else {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int64_t y = __shfl_up(incl, d);
      if (lane >= d) incl += y;
    }
  }
  if (lane == 63) lds[wave] = incl;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int v = 0; v < kAttnWaves; ++v) {
    if (v < wave) base += lds[v];
    all += lds[v];
  }
  *total = all;
  return base + incl - x;
}

__device__ inline int64_t uniform64(int64_t x) {
  return int64_t(uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(uint64_t(x) >> 32))))) << 32 |
                 uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(uint64_t(x))))));
}

// A piece of a workgroup's share: steps [st0, st1) of one tile of rows of one key head.
struct SegmentQ8 {
  int32_t set, row0, live;    // of key heads; the tile's first row, and rows in it
  int32_t steps, st0, st1;
  int32_t hidden;             // + a row's token: cached tokens that the row sees
  int32_t most;               // tokens that the last row sees
  int64_t begin;              // where the tile's cost begins
  int32_t part;               // 0: the first piece of the share
  __device__ bool whole() const { return st0 == 0 && st1 == steps; }
};

struct ShareLds {
  int64_t scan[2][kAttnWaves];
  int64_t place;
  SequenceQ8 found;
  int32_t b, descends[kAttnWaves];
};

// A workgroup's share of the cost of all pairs, which it goes through piece by piece.  All members are the
// same for all lanes.
template <int ROWS>
struct ShareQ8 {
  WorkQ8<ROWS> work;
  int64_t per, w0, w1, w;   // the share [w0, w1), and where in it
  int64_t *rec;
  int32_t b, item, x;       // sequence, pair and key head, place in their cost
  SequenceQ8 sq;
  uint32_t partial = 0;     // bit s: part s of this workgroup is one of a tile's several

  __device__ static int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

  // Finds the share; false where there is none.
  __device__ bool begin(ShareLds &lds) {
    const AttnQ8Plan &p = work.p;
    const int tid = int(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    const int32_t B = int32_t(p.seq.B);
    const int64_t me = blockIdx.x;
    // The first 256 sequences' sums say which one the share begins in, if it is one of them; later ones
    // are gone through again.
    SequenceQ8 s = {};
    int64_t rest = 0, total, n = 0;
    bool down = false;
    if (tid < B) {
      s = work.sequence(tid);
      n = work.cost(s);
      down = s.count < 0;
    }
    for (int32_t i = tid + kAttnBlock; i < B; i += kAttnBlock) {
      const SequenceQ8 y = work.sequence(i);
      rest += work.cost(y);
      down |= y.count < 0;
    }
    down = __any(down);
    if (lane == 0) lds.descends[wave] = down;
    int64_t place = p.small ? block_scan<true>(n, lds.scan[0], &total)
                            : block_scan<false>(n, lds.scan[0], &total);
    int64_t before = total;  // of the sequences so far
    if (B > kAttnBlock) {
      int64_t all;
      block_scan<false>(rest, lds.scan[1], &all);
      total += all;
    }
#pragma unroll
    for (int v = 0; v < kAttnWaves; ++v) down |= lds.descends[v] != 0;
    total = uniform64(total);
    per = p.small ? int64_t((uint32_t(total) + uint32_t(p.groups) - 1) / uint32_t(p.groups))
                  : (total + p.groups - 1) / p.groups;
    w = w0 = me * per;
    w1 = min(total, w0 + per);
    rec = p.joins + me * 2 * kQ8JoinWords;
    if (down || w0 >= total) {
      if (tid < 2) rec[tid * kQ8JoinWords] = 0;
      return false;
    }
    for (int32_t b0 = 0;; b0 += kAttnBlock) {  // ends: w0 < total
      if (b0 > 0) {
        n = 0;
        if (b0 + tid < B) {
          s = work.sequence(b0 + tid);
          n = work.cost(s);
        }
        int64_t all;
        __syncthreads();  // the last round's sums have been read
        place = before + block_scan<false>(n, lds.scan[0], &all);
        before += all;
      }
      if (place <= w0 && w0 < place + n) {
        lds.b = b0 + tid;
        lds.place = place;
        lds.found = s;
      }
      if (w0 < before) break;
    }
    __syncthreads();
    b = uniform(lds.b);
    sq = {uniform(lds.found.len), uniform(lds.found.first), uniform(lds.found.count),
          uniform(lds.found.tiles), uniform(lds.found.cost)};
    const int64_t into = w0 - uniform64(lds.place);
    item = int32_t(p.small ? int64_t(uint32_t(into) / uint32_t(sq.cost)) : into / sq.cost);
    x = int32_t(into - int64_t(item) * sq.cost);
    return true;
  }

  // The piece that begins at w.
  __device__ SegmentQ8 segment() {
    const AttnQ8Plan &p = work.p;
    const int32_t pair = int32_t(uint32_t(item) / uint32_t(p.head_sets));
    SegmentQ8 g;
    g.set = item - pair * p.head_sets;
    int32_t tile = sq.tiles - 1 - pair, at = 0, end = sq.cost;
    if (tile != pair) {  // two tiles: the longer one first
      const int32_t border = work.steps(sq, tile) + kQ8ItemCost;
      if (x < border) {
        end = border;
      } else {
        at = border;
        tile = pair;
      }
    }
    g.row0 = tile * ROWS;
    g.live = min(ROWS, sq.count * p.group - g.row0);
    g.steps = work.steps(sq, tile);
    g.most = work.visible(sq, tile);
    g.hidden = sq.len - sq.count + 1;
    g.begin = w - (x - at);
    const int32_t x1 = int32_t(min(int64_t(end), x + (w1 - w)));
    g.st0 = min(max(0, x - at - kQ8ItemCost), g.steps);
    g.st1 = min(max(0, x1 - at - kQ8ItemCost), g.steps);
    g.part = w == w0 ? 0 : 1;
    w += x1 - x;
    x = x1;
    return g;
  }

  // Notes a piece that is not a whole tile, for the joining kernel: the tile's parts are those of n
  // workgroups from `first` on.
  __device__ void note(const SegmentQ8 &g) {
    if (g.whole()) return;
    partial |= 1u << g.part;
    if (threadIdx.x == 0) {
      const int64_t from = g.begin + kQ8ItemCost, first = from / per;
      int64_t *to = rec + g.part * kQ8JoinWords;
      to[0] = (from + g.steps - 1) / per - first + 1;
      to[1] = first;
      to[2] = g.begin <= first * per ? 0 : 1;
      to[3] = sq.first;
      to[4] = g.set;
      to[5] = g.row0;
      to[6] = g.live;
    }
  }

  // On to the next piece; false at the end of the share.
  __device__ bool next() {
    if (w >= w1) {
      if (threadIdx.x < 2 && (partial >> threadIdx.x & 1u) == 0) rec[threadIdx.x * kQ8JoinWords] = 0;
      return false;
    }
    if (x >= sq.cost) {
      x = 0;
      if (++item >= sq.pairs() * work.p.head_sets) {
        item = 0;
        do {  // ends: w < w1 <= total, so a later sequence has tiles
          sq = work.sequence(++b);
        } while (sq.tiles == 0);
      }
    }
    return true;
  }
};

// Where row `m` of a tile of key head `head` lies in the output, in rows of D.
__device__ inline int64_t output_row(const AttnQ8Plan &p, const SegmentQ8 &g, int32_t head,
                                     int32_t first, int32_t m) {
  const int32_t r = g.row0 + m, tok = int32_t(div_by(p.div_group, uint32_t(r)));
  return int64_t(first + tok) * p.heads + head * p.group + r - tok * p.group;
}

template <typename T, int D, int R, bool E4M3, int MODE>
__global__ __launch_bounds__(kAttnBlock) __attribute__((amdgpu_waves_per_eu(q8_waves(D, R)))) void
attention_q8_kernel(AttnQ8Plan p) {
  constexpr int ROWS = 16 * R, N = D / 16;
  constexpr int LANE = 4 * N + 4;  // floats of a lane's outputs, kept apart by a chunk of 16 bytes
  __shared__ __attribute__((aligned(16))) float join_o[kAttnWaves][64 * LANE];
  __shared__ float join_top[kAttnWaves][16], join_sum[kAttnWaves][16];
  __shared__ ShareLds share_lds;

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the wavefront's key head of a set, and its turn among those of the same head
  const int32_t own = wave & (p.abreast - 1), turn = wave >> p.abreast_log2;
  ShareQ8<ROWS> share = {{p}};
  if (!share.begin(share_lds)) return;
  do {
    const SegmentQ8 g = share.segment();
    if (g.st0 >= g.st1) continue;
    const SequenceQ8 &sq = share.sq;
    const int32_t key_head = g.set * p.abreast + own;
    // fewest tokens that a row sees
    const int32_t floor = g.hidden + int32_t(div_by(p.div_group, uint32_t(g.row0)));
    // where rows may differ in the tokens that they see
    const int32_t apart = floor < g.most ? floor : 0x7fffffff;

    StateQ8<T, D, R> s;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s.by_reach[r] = kFirstByReach;
      const int32_t m = r * 16 + (lane & 15);
      const bool some = m < g.live;
      const int32_t tok = int32_t(div_by(p.div_group, uint32_t(g.row0 + (some ? m : 0))));
      const int32_t h = key_head * p.group + g.row0 + (some ? m : 0) - tok * p.group;
      s.limit[r] = some ? g.hidden + tok : 0;
      s.top[r] = kNegInf;
      s.sum[r] = 0.0f;
      const T *q = static_cast<const T *>(p.q) + int64_t(sq.first + tok) * p.q_tok +
                   int64_t(h) * p.q_head + D / 4 * (lane >> 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        s.q[r][i] = some ? as_operand(*reinterpret_cast<const uint4 *>(q + 8 * i)) : s16x8{};
#pragma unroll
      for (int n = 0; n < N; ++n) s.o[r][n] = f32x4{};
    }
    {
      const int32_t last = sq.len - 1, step = 1 << p.step_log2, b = share.b;
      const int64_t head = key_head;
      int32_t t0 = g.st0 * step + turn * kTile;
      const int32_t end = min(g.st1 * step, g.most);
      auto at = [&](int32_t t) { return locate<MODE>(p.seq, b, t, last, lane); };
      if (t0 < end) {
        // A tile's keys are asked for once the tile before is scored, its values once that is weighed.
        // The loads are made whether or not there is another tile (the present one again, from the
        // caches): behind a branch the compiler would wait for all loads at each use.
        KeysQ8<D, MODE> k;
        ValuesQ8<D, MODE> v;
        WhereQ8<MODE> next = at(t0);
        load_keys<D, MODE>(p, next, t0, last, head, lane, k);
        load_values<D, MODE>(p, next, t0, last, head, lane, v);
        while (true) {  // ends: t0 grows
          const int32_t t1 = t0 + step < end ? t0 + step : t0;
          next = at(t1);
          if constexpr (E4M3) {
            if (t0 + kTile > apart) {
              asm volatile("");
              part_nans<T, D, R>(v, s, t0, lane);
            }
          }
          f32x4 x[R][2];
          score_tile<T, D, R, E4M3, MODE>(k, s, t0, floor, p.scale_log2, lane, x);
          load_keys<D, MODE>(p, next, t1, last, head, lane, k);
          weigh_tile<T, D, R, E4M3, MODE>(v, s, t0, floor, lane, x);
          if (t1 == t0) break;
          load_values<D, MODE>(p, next, t1, last, head, lane, v);
          t0 = t1;
        }
      }
    }

    // ---- the sums of a head's wavefronts, joined 16 rows at a time; 16 threads a row, as many threads
    // for each head ----
    const int heads_log2 = p.abreast_log2, gr = tid & 15;
    const int mine = tid >> (8 - heads_log2), m0 = tid >> 4 & ((16 >> heads_log2) - 1);
    const int64_t slot = (int64_t(blockIdx.x) * 2 + g.part) * p.abreast + mine;
    const int32_t to_head = g.set * p.abreast + mine;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float sum = sum_quarters(s.sum[r]);
      const float unit = Mfma<T>::kNarrow ? inverse_power(s.by_reach[r]) : 1.0f;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int n = 0; n < N; n += 4)
          *reinterpret_cast<f32x4 *>(&join_o[wave][lane * LANE + k * N + n]) =
              f32x4{s.o[r][n][k], s.o[r][n + 1][k], s.o[r][n + 2][k], s.o[r][n + 3][k]} * unit;
      if (lane < 16) {
        join_top[wave][lane] = s.top[r];
        join_sum[wave][lane] = sum;
      }
      __syncthreads();
      for (int m = m0; m < min(16, g.live - r * 16); m += 16 >> heads_log2) {
        const int row = r * 16 + m;
        float top = kNegInf;
        for (int v = mine; v < kAttnWaves; v += p.abreast) top = fmaxf(top, join_top[v][m]);
        float l = 0.0f, o[N];
#pragma unroll
        for (int n = 0; n < N; ++n) o[n] = 0.0f;
        for (int v = mine; v < kAttnWaves; v += p.abreast) {
          const float f = __builtin_amdgcn_exp2f(join_top[v][m] - (top == kNegInf ? 0.0f : top));
          l += f * join_sum[v][m];
          const float *from = &join_o[v][((gr >> 2) * 16 + m) * LANE + (gr & 3) * N];
#pragma unroll
          for (int n = 0; n < N; n += 4) {
            const f32x4 y = *reinterpret_cast<const f32x4 *>(from + n);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n + e] += f * y[e];
          }
        }
        if (g.whole()) {
          const int64_t at = output_row(p, g, to_head, sq.first, row);
          const bool some = l > 0.0f || l != l;  // a row that sees nothing gets zeros
          const float inv = some ? 1.0f / l : 0.0f;
          uint32_t y[N / 2];
#pragma unroll
          for (int n = 0; n < N / 2; ++n) y[n] = Mfma<T>::pack(o[2 * n] * inv, o[2 * n + 1] * inv);
          char *out = static_cast<char *>(p.out) + at * (2 * D) + gr * (2 * N);
#pragma unroll
          for (int n = 0; n < N / 2; n += 2)
            *reinterpret_cast<uint2 *>(out + 4 * n) = make_uint2(y[n], y[n + 1]);
          if (gr == 0 && p.lse != nullptr) p.lse[at] = some ? natural<T>(top, l) : kNegInf;
        } else {
          float *to = p.parts + (slot * ROWS + row) * D + gr * N;
#pragma unroll
          for (int n = 0; n < N; n += 4)
            *reinterpret_cast<f32x4 *>(to + n) = f32x4{o[n], o[n + 1], o[n + 2], o[n + 3]};
          if (gr == 0)
            *reinterpret_cast<float2 *>(p.stats + (slot * ROWS + row) * 2) = make_float2(top, l);
        }
      }
    }
    share.note(g);
  } while (share.next());
}

// Joins the parts of items that several workgroups had a share of: with unnormalised outputs o_k at
// maximum m_k and weight sum l_k,  out = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k,  m = max m_k.
// One workgroup for each of an item's n parts takes the n-th of its lines (rows of its key heads), several
// lines at a time, head_size / 4 threads each.  Of more than four parts several threads share an element's,
// so that the 43 parts of an item of long contexts take two rounds of loads, not eleven (11.8 -> 6.8 us).
template <typename T>
__global__ __launch_bounds__(kAttnBlock) void attention_q8_join_kernel(AttnQ8Plan p) {
  __shared__ f32x4 join_o[kAttnBlock];
  __shared__ float2 join_stat[kAttnBlock];
  const int64_t *rec = p.joins + int64_t(blockIdx.x) * kQ8JoinWords;
  const int32_t n = int32_t(rec[0]);
  if (n <= 1) return;
  const int64_t g0 = rec[1], first = rec[2];
  const int32_t k0 = int32_t(int64_t(blockIdx.x >> 1) - g0);
  const int32_t live = int32_t(rec[6]), lines = live * p.abreast;
  const int32_t l0 = int32_t(int64_t(lines) * k0 / n), l1 = int32_t(int64_t(lines) * (k0 + 1) / n);
  const int32_t tid = int32_t(threadIdx.x), wide = p.head_size / 4;  // 16, 32 or 64
  const int32_t d = tid & (wide - 1), turn = tid / wide, turns = kAttnBlock / wide;
  constexpr int AHEAD = 4;  // parts that a thread reads at a time
  int32_t ways = 1;         // threads of an element
  while (ways < turns && ways * AHEAD < n) ways *= 2;
  const int32_t way = turn & (ways - 1);
  for (int32_t l = l0; l < l1; l += turns / ways) {
    const int32_t line = l + turn / ways, own = line / live, m = line - own * live;
    const bool some = line < l1;
    float top = kNegInf, sum = 0.0f;
    f32x4 o = {};
    for (int32_t k = way; k < n; k += AHEAD * ways) {
      float2 stat[AHEAD];
      f32x4 x[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int32_t part = k + u * ways;
        stat[u] = make_float2(kNegInf, 0.0f);
        x[u] = f32x4{};
        if (some && part < n) {
          const int64_t at = (((g0 + part) * 2 + (part == 0 ? first : 0)) * p.abreast + own) * p.rows + m;
          stat[u] = *reinterpret_cast<const float2 *>(p.stats + at * 2);
          x[u] = *reinterpret_cast<const f32x4 *>(p.parts + at * p.head_size + d * 4);
        }
      }
      float next = top;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) next = fmaxf(next, stat[u].x);
      const float ref = next == kNegInf ? 0.0f : next;
      const float f = __builtin_amdgcn_exp2f(top - ref);
      top = next;
      sum *= f;
      o *= f;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const float y = __builtin_amdgcn_exp2f(stat[u].x - ref);
        sum += stat[u].y * y;
        o += x[u] * y;
      }
    }
    if (ways > 1) {
      __syncthreads();
      join_o[tid] = o;
      join_stat[tid] = make_float2(top, sum);
      __syncthreads();
      if (way != 0) continue;
      for (int32_t v = 1; v < ways; ++v) top = fmaxf(top, join_stat[tid + v * wide].x);
      const float ref = top == kNegInf ? 0.0f : top;
      sum = 0.0f;
      o = f32x4{};
      for (int32_t v = 0; v < ways; ++v) {
        const float y = __builtin_amdgcn_exp2f(join_stat[tid + v * wide].x - ref);
        sum += join_stat[tid + v * wide].y * y;
        o += join_o[tid + v * wide] * y;
      }
    }
    if (!some) continue;
    const bool any = sum > 0.0f || sum != sum;
    const float inv = any ? 1.0f / sum : 0.0f;
    const int32_t row = int32_t(rec[5]) + m, tok = int32_t(div_by(p.div_group, uint32_t(row)));
    const int64_t at = (rec[3] + tok) * p.heads + (rec[4] * p.abreast + own) * p.group + row - tok * p.group;
    *reinterpret_cast<uint2 *>(static_cast<char *>(p.out) + (at * p.head_size + d * 4) * 2) =
        make_uint2(Mfma<T>::pack(o[0] * inv, o[1] * inv), Mfma<T>::pack(o[2] * inv, o[3] * inv));
    if (d == 0 && p.lse != nullptr) p.lse[at] = any ? natural<T>(top, sum) : kNegInf;
  }
}

}  // namespace
}  // namespace ropeamd
