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
// wavefront takes 32 tokens at a time, has the next 32 under way (8 KB at D 128), and four
// wavefronts of a workgroup, which take every fourth 32 tokens each, join their sums at the end.
//
// Layout (16x16x32 products, lane l = 16 g + c):
//   S^T = K Q^T: A[key c][8 d], lane's d = 64 i + 16 g + 8 e + 0..7 for product (i, e): 16 bytes a load
//   and two products; register r of S^T: key 4 g + r of query row c.
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
static_assert(kTile * kAttnWaves == kQ8Step, "a step is a tile of every wavefront");

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

// What a sequence asks for.
struct SequenceQ8 {
  int32_t len, first, count;  // cached tokens; first query token, query tokens (below 0: descending)
  int32_t items, steps;       // items of a key head; steps of an item
  __device__ int64_t cost(int kv_heads) const {
    return int64_t(items) * kv_heads * (steps + kQ8ItemCost);
  }
};

// Lengths and offsets are device data: values outside their ranges are clamped.
__device__ inline SequenceQ8 sequence_q8(const AttnQ8Plan &p, int32_t b, int rows) {
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
  s.items = (max(s.count, 0) * p.group + rows - 1) / rows;
  s.steps = max(1, (s.len + int32_t(kQ8Step) - 1) / int32_t(kQ8Step));
  return s;
}

// 32 tokens of a key head: codes, and the scales of the lane's keys in S^T.
template <int D, bool RUNS>
struct TileQ8 {
  static constexpr int W = D / 64;
  static constexpr int SC = RUNS ? 2 : 8;
  uint4 k[2][W];
  uint32_t v[8][W];
  float ks[SC], vs[SC];
  __device__ float key_scale(int j) const { return ks[RUNS ? j / 4 : j]; }
  __device__ float value_scale(int j) const { return vs[RUNS ? j / 4 : j]; }
};

// Where a tile lies: runs of 16 tokens in one page each, the same for all lanes; or a token a lane.
template <bool RUNS>
struct WhereQ8;
template <>
struct WhereQ8<true> {
  int64_t page[2];
};
template <>
struct WhereQ8<false> {
  int32_t page, row;
};

__device__ inline int64_t page_of(const Sequences &s, int32_t b, int32_t index) {
  const int64_t id = s.table[b * s.table_seq + index * s.table_page];
  return min(max(id, int64_t(0)), s.num_pages - 1);
}

// Tokens past the last one (`last`) repeat it.
template <bool RUNS>
__device__ __forceinline__ WhereQ8<RUNS> locate(const Sequences &s, int32_t b, int32_t t0,
                                                int32_t last, int lane) {
  WhereQ8<RUNS> w;
  if constexpr (RUNS) {
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

template <int W>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    v[0] = x.x;
    v[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    v[0] = x.x;
    v[1] = x.y;
    v[2] = x.z;
    v[3] = x.w;
  }
}

template <int D, bool RUNS>
__device__ __forceinline__ void load_tile(const AttnQ8Plan &p, const WhereQ8<RUNS> &w, int32_t t0,
                                          int32_t last, int64_t head, int lane,
                                          TileQ8<D, RUNS> &t) {
  constexpr int W = D / 64;
  const int c = lane & 15, g = lane >> 4;
  if constexpr (RUNS) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int32_t begin = min(t0 + 16 * h, last), more = last - begin;
      const int32_t row = begin - int32_t(div_by(p.seq.div_page, uint32_t(begin)) *
                                          uint32_t(p.seq.page_size));
      const uint8_t *k = p.k.codes + w.page[h] * p.k.page + head * p.k.head + int64_t(row) * p.k.row;
      const uint32_t at = uint32_t(min(c, more) * p.k.row + 16 * g);
#pragma unroll
      for (int i = 0; i < W; ++i)
        t.k[h][i] = *reinterpret_cast<const uint4 *>(k + (at + 64 * i));
      const uint8_t *v = p.v.codes + w.page[h] * p.v.page + head * p.v.head + int64_t(row) * p.v.row;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        load_words<W>(v + uint32_t(min(4 * g + j, more) * p.v.row + c * (D / 16)), t.v[4 * h + j]);
      const int64_t block = div_by(p.div_block, uint32_t(row + min(4 * g, more)));
      t.ks[h] = p.k.scales[w.page[h] * p.k.s_page + head * p.k.s_head + block * p.k.s_block];
      t.vs[h] = p.v.scales[w.page[h] * p.v.s_page + head * p.v.s_head + block * p.v.s_block];
    }
  } else {
    const int64_t block = div_by(p.div_block, uint32_t(w.row));
    const float ks = p.k.scales[w.page * p.k.s_page + head * p.k.s_head + block * p.k.s_block];
    const float vs = p.v.scales[w.page * p.v.s_page + head * p.v.s_head + block * p.v.s_block];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t page = __shfl(w.page, 16 * h + c), row = __shfl(w.row, 16 * h + c);
      const uint8_t *k = p.k.codes + page * p.k.page + head * p.k.head + row * p.k.row + 16 * g;
#pragma unroll
      for (int i = 0; i < W; ++i) t.k[h][i] = *reinterpret_cast<const uint4 *>(k + 64 * i);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int key = 16 * (j / 4) + 4 * g + j % 4;
      const int64_t page = __shfl(w.page, key), row = __shfl(w.row, key);
      load_words<W>(p.v.codes + page * p.v.page + head * p.v.head + row * p.v.row + c * (D / 16),
                    t.v[j]);
      t.ks[j] = __shfl(ks, key);
      t.vs[j] = __shfl(vs, key);
    }
  }
}

// A wavefront's running state for R tiles of 16 query rows; the lane's row of a tile is row c.
template <typename T, int D, int R>
struct StateQ8 {
  s16x8 q[R][D / 32];
  f32x4 o[R][D / 16];
  float top[R], sum[R];
  int32_t limit[R];  // tokens that the lane's row may see
  // float16: the weights p vs have to stay in its range, so vs is taken relative to a power of two not
  // below the largest one so far
  float reach, by_reach;
};

template <typename T, int D, int R, bool E4M3, bool RUNS>
__device__ __forceinline__ void attend_tile(const TileQ8<D, RUNS> &t, StateQ8<T, D, R> &s,
                                            int32_t t0, int32_t floor, float scale_log2, int lane) {
  constexpr int W = D / 64;
  const int g = lane >> 4;
  using Op = Operand<T, E4M3>;
  f32x4 x[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) x[r][0] = x[r][1] = f32x4{};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const s16x8 a = Op::row(t.k[h][i].x, t.k[h][i].y), b = Op::row(t.k[h][i].z, t.k[h][i].w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[r][h] = Mfma<T>::mul16(a, s.q[r][2 * i], x[r][h]);
        x[r][h] = Mfma<T>::mul16(b, s.q[r][2 * i + 1], x[r][h]);
      }
    }
  // scores in powers of two
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < 8; ++j) x[r][j / 4][j % 4] *= t.key_scale(j) * scale_log2;
  const bool masked = t0 + kTile > floor;
  if (masked) {
    asm volatile("");  // a branch: most tiles need no masks
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (t0 + 16 * (j / 4) + 4 * g + j % 4 >= s.limit[r]) x[r][j / 4][j % 4] = kNegInf;
  }
  // A row's maximum is raised only when a tile passes it by more than kSlack; until then larger weights
  // are carried, which changes no result beyond its rounding.
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
  float vs[RUNS ? 2 : 8];
#pragma unroll
  for (int j = 0; j < (RUNS ? 2 : 8); ++j) {
    vs[j] = t.vs[j];
    if constexpr (Mfma<T>::kNarrow) raise |= fabsf(vs[j]) > s.reach;
  }
  if (__any(raise)) {
    float reach = s.reach;
    if constexpr (Mfma<T>::kNarrow) {
      float most = 0.0f;
#pragma unroll
      for (int j = 0; j < (RUNS ? 2 : 8); ++j) most = fmaxf(most, fabsf(vs[j]));
      for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
      // the power of two above it, within those whose reciprocal is one, too
      const uint32_t e = min(max(__float_as_uint(most) >> 23, 1u), 252u) + 1u;
      if (most > reach) reach = __uint_as_float(e << 23);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f = 1.0f;
      if (best[r] > s.top[r] + Mfma<T>::kSlack) {
        f = __builtin_amdgcn_exp2f(s.top[r] - best[r]);
        s.top[r] = best[r];
      }
      s.sum[r] *= f;
      if constexpr (Mfma<T>::kNarrow) f *= s.reach * __uint_as_float((254u << 23) - __float_as_uint(reach));
#pragma unroll
      for (int n = 0; n < D / 16; ++n) s.o[r][n] *= f;
    }
    if constexpr (Mfma<T>::kNarrow) {
      s.reach = reach;
      s.by_reach = __uint_as_float((254u << 23) - __float_as_uint(reach));
    }
  }
  if constexpr (Mfma<T>::kNarrow) {
#pragma unroll
    for (int j = 0; j < (RUNS ? 2 : 8); ++j) vs[j] *= s.by_reach;
  }
  s16x8 w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float ref = s.top[r] == kNegInf ? 0.0f : s.top[r] - Mfma<T>::kLift;
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = __builtin_amdgcn_exp2f(x[r][j / 4][j % 4] - ref);
      s.sum[r] += y;
      e[j] = y * vs[RUNS ? j / 4 : j];
    }
    if (masked) {
      asm volatile("");
#pragma unroll
      for (int j = 0; j < 8; ++j)  // whatever the scale of a token that the row does not see
        if (t0 + 16 * (j / 4) + 4 * g + j % 4 >= s.limit[r]) e[j] = 0.0f;
    }
    w[r] = round8<T>(e);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = t.v[j][i];
    s16x8 a[4];
    Op::template columns<false>(v, &a[0], &a[1]);
    Op::template columns<true>(v, &a[2], &a[3]);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int r = 0; r < R; ++r) s.o[r][4 * i + n] = Mfma<T>::mul16(a[n], w[r], s.o[r][4 * i + n]);
  }
}

// Sum over the workgroup's threads before this one, and of all (in `total`).
__device__ inline int64_t block_scan(int64_t x, int64_t *lds, int64_t *total) {
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  int64_t incl = x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  __syncthreads();
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

template <typename T, int D, int R, bool E4M3, bool RUNS>
__global__ __launch_bounds__(kAttnBlock) void attention_q8_kernel(AttnQ8Plan p) {
  constexpr int ROWS = 16 * R, N = D / 16;
  constexpr int LANE = 4 * N + 4;  // floats of a lane's outputs, kept apart by a chunk of 16 bytes
  __shared__ __attribute__((aligned(16))) float join_o[kAttnWaves][64 * LANE];
  __shared__ float join_top[kAttnWaves][16], join_sum[kAttnWaves][16];
  __shared__ int64_t scan[kAttnWaves];
  __shared__ int64_t found_at;
  __shared__ int32_t found_b, descends;

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  auto uniform = [](int32_t x) { return __builtin_amdgcn_readfirstlane(x); };
  const int32_t B = int32_t(p.seq.B);
  const int64_t me = blockIdx.x;

  // ---- this workgroup's share [w0, w1) of all items' cost ----
  if (tid == 0) descends = 0;
  __syncthreads();
  int64_t mine = 0, total;
  for (int32_t b = tid; b < B; b += kAttnBlock) {
    const SequenceQ8 s = sequence_q8(p, b, ROWS);
    mine += s.cost(p.kv_heads);
    if (s.count < 0) descends = 1;
  }
  block_scan(mine, scan, &total);
  const int64_t per = (total + p.groups - 1) / p.groups;
  const int64_t w0 = me * per, w1 = min(total, w0 + per);
  int64_t *rec = p.joins + me * 2 * kQ8JoinWords;
  if (descends || w0 >= total) {
    if (tid < 2) rec[tid * kQ8JoinWords] = 0;
    return;
  }
  int64_t before = 0;
  for (int32_t b0 = 0;; b0 += kAttnBlock) {  // ends: w0 < total
    int64_t n = 0, all;
    if (b0 + tid < B) n = sequence_q8(p, b0 + tid, ROWS).cost(p.kv_heads);
    const int64_t at = before + block_scan(n, scan, &all);
    if (at <= w0 && w0 < at + n) {
      found_b = b0 + tid;
      found_at = at;
    }
    before += all;
    if (w0 < before) break;
  }
  __syncthreads();
  int32_t b = uniform(found_b);
  SequenceQ8 sq = sequence_q8(p, b, ROWS);
  int64_t w = w0;
  int32_t item, x0;
  {
    const int64_t into = w0 - uniform64(found_at);
    const int64_t cost = sq.steps + kQ8ItemCost;
    item = int32_t(into / cost);
    x0 = int32_t(into - item * cost);
  }
  uint32_t partial = 0;  // bit s: part s of this workgroup is one of an item's several

  while (true) {
    const int32_t cost = sq.steps + kQ8ItemCost;
    const int32_t x1 = int32_t(min(int64_t(cost), x0 + (w1 - w)));
    const int32_t st0 = max(0, x0 - kQ8ItemCost), st1 = max(0, x1 - kQ8ItemCost);
    if (st0 < st1) {
      const int32_t head = int32_t(uint32_t(item) % uint32_t(p.kv_heads));
      const int32_t row0 = int32_t(uint32_t(item) / uint32_t(p.kv_heads)) * ROWS;
      const int32_t rows = sq.count * p.group, live = min(ROWS, rows - row0);
      const int32_t hidden = sq.len - sq.count + 1;  // + token: tokens that it sees
      // fewest and most tokens that a row sees
      const int32_t floor = hidden + int32_t(div_by(p.div_group, uint32_t(row0)));
      const int32_t most = min(sq.len, hidden + int32_t(div_by(p.div_group, uint32_t(row0 + live - 1))));

      StateQ8<T, D, R> s;
      s.reach = 0x1p-120f;
      s.by_reach = 0x1p120f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int32_t m = r * 16 + (lane & 15);
        const bool some = m < live;
        const int32_t tok = int32_t(div_by(p.div_group, uint32_t(row0 + (some ? m : 0))));
        const int32_t h = head * p.group + row0 + (some ? m : 0) - tok * p.group;
        s.limit[r] = some ? hidden + tok : 0;
        s.top[r] = kNegInf;
        s.sum[r] = 0.0f;
        const T *q = static_cast<const T *>(p.q) + int64_t(sq.first + tok) * p.q_tok +
                     int64_t(h) * p.q_head + 16 * (lane >> 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          s.q[r][i] = some ? as_operand(*reinterpret_cast<const uint4 *>(q + 64 * (i / 2) + 8 * (i % 2)))
                           : s16x8{};
#pragma unroll
        for (int n = 0; n < N; ++n) s.o[r][n] = f32x4{};
      }
      {
        const int32_t last = sq.len - 1;
        int32_t t0 = st0 * int32_t(kQ8Step) + wave * kTile;
        const int32_t end = min(st1 * int32_t(kQ8Step), most);
        auto at = [&](int32_t t) { return locate<RUNS>(p.seq, b, t, last, lane); };
        if (t0 < end) {
          TileQ8<D, RUNS> a, c;
          load_tile<D, RUNS>(p, at(t0), t0, last, head, lane, a);
          WhereQ8<RUNS> next = at(t0 + int32_t(kQ8Step));
          while (true) {  // ends: t0 grows
            int32_t t1 = t0 + int32_t(kQ8Step);
            if (t1 < end) {
              load_tile<D, RUNS>(p, next, t1, last, head, lane, c);
              next = at(t1 + int32_t(kQ8Step));
            }
            attend_tile<T, D, R, E4M3, RUNS>(a, s, t0, floor, p.scale_log2, lane);
            if (t1 >= end) break;
            t0 = t1 + int32_t(kQ8Step);
            if (t0 < end) {
              load_tile<D, RUNS>(p, next, t0, last, head, lane, a);
              next = at(t0 + int32_t(kQ8Step));
            }
            attend_tile<T, D, R, E4M3, RUNS>(c, s, t1, floor, p.scale_log2, lane);
            if (t0 >= end) break;
          }
        }
      }

      // ---- the wavefronts' sums, joined 16 rows at a time; 16 threads a row ----
      const bool whole = st0 == 0 && st1 == sq.steps;
      const int part = w == w0 ? 0 : 1;
      const int64_t slot = me * 2 + part;
      const int m = tid >> 4, gr = tid & 15;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float sum = sum_quarters(s.sum[r]);
        const float unit = Mfma<T>::kNarrow ? s.reach : 1.0f;
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
        const int row = r * 16 + m;
        if (row >= live) continue;
        float top = join_top[0][m];
#pragma unroll
        for (int v = 1; v < kAttnWaves; ++v) top = fmaxf(top, join_top[v][m]);
        float l = 0.0f, o[N];
#pragma unroll
        for (int n = 0; n < N; ++n) o[n] = 0.0f;
#pragma unroll
        for (int v = 0; v < kAttnWaves; ++v) {
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
        if (whole) {
          const int32_t tok = int32_t(div_by(p.div_group, uint32_t(row0 + row)));
          const int64_t at = int64_t(sq.first + tok) * p.heads + head * p.group + row0 + row -
                             tok * p.group;
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
      if (!whole) {
        partial |= 1u << part;
        if (tid == 0) {  // the item's parts: `n` workgroups from `first` on
          const int64_t begin = w - x0, first = (begin + kQ8ItemCost) / per;
          int64_t *to = rec + part * kQ8JoinWords;
          to[0] = (begin + cost - 1) / per - first + 1;
          to[1] = first;
          to[2] = begin <= first * per ? 0 : 1;
          to[3] = sq.first;
          to[4] = head;
          to[5] = row0;
          to[6] = live;
        }
      }
    }
    w += x1 - x0;
    if (w >= w1) break;
    x0 = 0;
    if (++item >= sq.items * p.kv_heads) {
      item = 0;
      do {  // ends: w < w1 <= total, so a later sequence has items
        ++b;
        sq = sequence_q8(p, b, ROWS);
      } while (sq.items == 0);
    }
  }
  if (tid < 2 && (partial >> tid & 1u) == 0) rec[tid * kQ8JoinWords] = 0;
}

// Joins the parts of items that several workgroups had a share of: with unnormalised outputs o_k at
// maximum m_k and weight sum l_k,  out = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k,  m = max m_k.
// One workgroup for each part takes its n-th of the item's rows and columns.
template <typename T>
__global__ __launch_bounds__(kAttnBlock) void attention_q8_join_kernel(AttnQ8Plan p) {
  const int64_t *rec = p.joins + int64_t(blockIdx.x) * kQ8JoinWords;
  const int32_t n = int32_t(rec[0]);
  if (n <= 1) return;
  const int64_t g0 = rec[1], first = rec[2];
  const int32_t k0 = int32_t(int64_t(blockIdx.x >> 1) - g0);
  const int32_t rows = 16 * p.tiles, wide = p.head_size / 4;
  const int32_t cells = int32_t(rec[6]) * wide;
  const int32_t c0 = int32_t(int64_t(cells) * k0 / n), c1 = int32_t(int64_t(cells) * (k0 + 1) / n);
  for (int32_t cell = c0 + int32_t(threadIdx.x); cell < c1; cell += kAttnBlock) {
    const int32_t m = cell / wide, d = cell - m * wide;
    float top = kNegInf, l = 0.0f;
    f32x4 o = {};
    constexpr int AHEAD = 4;
    for (int32_t k = 0; k < n; k += AHEAD) {
      float2 stat[AHEAD];
      f32x4 x[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        stat[u] = make_float2(kNegInf, 0.0f);
        x[u] = f32x4{};
        if (k + u < n) {
          const int64_t at = ((g0 + k + u) * 2 + (k + u == 0 ? first : 0)) * rows + m;
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
      l *= f;
      o *= f;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const float y = __builtin_amdgcn_exp2f(stat[u].x - ref);
        l += stat[u].y * y;
        o += x[u] * y;
      }
    }
    const bool some = l > 0.0f || l != l;
    const float inv = some ? 1.0f / l : 0.0f;
    const int32_t r = int32_t(rec[5]) + m, tok = int32_t(div_by(p.div_group, uint32_t(r)));
    const int64_t at = (rec[3] + tok) * p.heads + rec[4] * p.group + r - tok * p.group;
    *reinterpret_cast<uint2 *>(static_cast<char *>(p.out) + (at * p.head_size + d * 4) * 2) =
        make_uint2(Mfma<T>::pack(o[0] * inv, o[1] * inv), Mfma<T>::pack(o[2] * inv, o[3] * inv));
    if (d == 0 && p.lse != nullptr) p.lse[at] = some ? natural<T>(top, l) : kNegInf;
  }
}

template <typename T, int D, int R>
const void *pick_attention_q8(const AttnQ8Plan &p) {
#define ROPE_KQ(E, RU) reinterpret_cast<const void *>(&attention_q8_kernel<T, D, R, E, RU>)
  if (p.e4m3) return p.runs ? ROPE_KQ(true, true) : ROPE_KQ(true, false);
  return p.runs ? ROPE_KQ(false, true) : ROPE_KQ(false, false);
#undef ROPE_KQ
}

template <typename T, int D>
const void *pick_attention_q8(const AttnQ8Plan &p) {
  return p.tiles == 1 ? pick_attention_q8<T, D, 1>(p) : pick_attention_q8<T, D, 2>(p);
}

template <typename T>
int run_attention_q8(AttnQ8Plan &p, void *stream) {
  const void *fn = p.head_size == 64    ? pick_attention_q8<T, 64>(p)
                   : p.head_size == 128 ? pick_attention_q8<T, 128>(p)
                                        : pick_attention_q8<T, 256>(p);
  const int st = launch_kernel(fn, dim3(uint32_t(p.groups)), kAttnBlock, 0, stream, &p);
  if (st != ROPE_OK) return st;
  return launch_kernel(reinterpret_cast<const void *>(&attention_q8_join_kernel<T>),
                       dim3(uint32_t(p.groups) * 2), kAttnBlock, 0, stream, &p);
}

}  // namespace
}  // namespace ropeamd
