// rope_q8_rows.h -- attention over a paged cache of 8-bit codes for many query rows of a key head: pieces of
// prompts, drafts of many heads (gfx950; library-internal, instantiated beside rope_q8_attn.h).
//
// With some 40 rows and more a call is bound by its products and what lies between them, and a tile's
// codes are worth turning into operands once for all rows: a workgroup has 128 rows, 32 of each
// wavefront.  Codes come to registers a tile ahead, are made 16-bit operands and go to LDS, into the
// second of two buffers, in the panels of rope_mfma.h; S^T = K Q^T and O^T = V^T P^T are 32x32x16
// products, so that a lane owns a query row and P goes from one to the other in registers.
// Scales wait, as in the other kernel: keys' multiply the scores, values' the weights.
//
// 4 x 4096 prompt tokens of 32 heads of 128, 8 key heads: 762 us a launch (725-790), 719 a call back to back,
// 0.72-0.77 PFLOP/s.  The vector units work 0.61 of the cycles (of 327 instructions a step 96 turn codes into
// operands, 161 are the softmax's), the matrix units 0.33: the two wavefronts of a SIMD rarely need them at the same
// time, and what is left is not idle.
#pragma once

#include "rope_q8_attn.h"

namespace ropeamd {
namespace {

template <int D>
struct RowsShape {
  static constexpr int TILE = D == 256 ? 32 : 64;  // tokens of a step
  static_assert(TILE == 1 << q8_step_log2(kQ8ManyRows, D, 0), "a step is a tile");
  static constexpr int PANELS = D / 64;
  static constexpr int PANEL = TILE * 128;          // bytes
  static constexpr int THREADS = kAttnBlock / TILE;  // of a token's codes
  static constexpr int BYTES = D / THREADS;          // of one thread: pieces of 16
  // A wavefront takes tokens of 16 from run(wave) on (8 where a tile has 32); a lane one of them, and
  // every THREADS-th 16 codes from 16 piece() on.  Eight lanes write operands to LDS at a time: two tokens 8
  // apart, whose chunks of half a row of a panel lie in different banks.  (With neighbouring tokens, and a lane's
  // codes side by side, four met in a bank: 0.22 of the cycles were such conflicts, and 4 x 4096 tokens of 32
  // heads took 1.82 M cycles, not 1.60 M.)
  __device__ static int run(int wave) { return D == 256 ? wave / 2 * 16 : wave * 16; }
  __device__ static int token(int wave, int lane) {
    const int x = lane >> 2;
    return D == 256 ? (x & 1) << 3 | wave % 2 * 4 | lane >> 4
                    : (x & 1) << 3 | (x & 2) >> 1 | (x & 12) >> 1;
  }
  __device__ static int piece(int lane) { return D == 256 ? (lane & 3) | (lane >> 1 & 4) : lane & 3; }
};

// Scales of a tile.  kCoarse: one for each 4 tokens, those of the lanes below 32 first: of tokens
// 8 c + 4 (l / 32) and on at 8 (l / 32) + c, c up to 8; else one for each token.
template <int D, int MODE>
struct ScalesOf {
  static constexpr int RUN = MODE == kCoarse ? 4 : 1, COUNT = RowsShape<D>::TILE / RUN;
  static constexpr int EACH = COUNT / kAttnWaves;  // of a wavefront's own tokens
  // the token of a wavefront's run of 16 whose scale a lane loads
  __device__ static int token(int wave, int lane) { return (wave * EACH % (16 / RUN) + lane % EACH) * RUN; }
  __device__ static int place(int i) { return MODE == kCoarse ? (i & 1) * (COUNT / 2) + (i >> 1) : i; }
};

// What a thread has of a tile: some of a token's key and value codes, and a scale (of its wavefront's keys in
// the first lanes, of their values in the next).
template <int D>
struct StageQ8 {
  uint4 k[RowsShape<D>::BYTES / 16], v[RowsShape<D>::BYTES / 16];
  float scale;
};

template <int D>
struct RowsLds {
  struct Buffer {
    char k[RowsShape<D>::PANELS * RowsShape<D>::PANEL], v[RowsShape<D>::PANELS * RowsShape<D>::PANEL];
    float k_scale[RowsShape<D>::TILE], v_scale[RowsShape<D>::TILE];
  };
  Buffer buffer[2];
  ShareLds share;
  int32_t nans[2][kAttnWaves];  // of each buffer: whether a wavefront's tokens have NaN values (e4m3, `look` of put)
};

// Where a wavefront's tokens of a tile lie; tokens past the last one repeat it.  Pages of whole runs of 16
// tokens: all in one page, whose number and first row are the same for all lanes.
template <int MODE>
struct TokensQ8 {
  int64_t page;
  int32_t row, more;  // the first token's row; tokens that follow it in the sequence
};
template <>
struct TokensQ8<kAny> {
  int32_t page, row;  // of the thread's token, and of the one whose scale it loads
  int32_t scale_page, scale_row;
};

template <int D, int MODE>
__device__ __forceinline__ TokensQ8<MODE> tokens_at(const Sequences &s, int32_t b, int32_t t, int32_t last,
                                                    int wave, int lane) {
  using S = RowsShape<D>;
  const int32_t t0 = t + S::run(wave);
  TokensQ8<MODE> x;
  if constexpr (MODE != kAny) {
    const int32_t begin = min(t0, last);
    const uint32_t i = div_by(s.div_page, uint32_t(begin));
    x.page = page_of(s, b, int32_t(i));
    x.row = begin - int32_t(i * uint32_t(s.page_size));
    x.more = last - begin;
  } else {
    auto one = [&](int32_t token, int32_t &page, int32_t &row) {
      const uint32_t i = div_by(s.div_page, uint32_t(token));
      page = int32_t(page_of(s, b, int32_t(i)));
      row = token - int32_t(i * uint32_t(s.page_size));
    };
    one(min(t0 + S::token(wave, lane), last), x.page, x.row);
    one(min(t0 + ScalesOf<D, MODE>::token(wave, lane), last), x.scale_page, x.scale_row);
  }
  return x;
}

template <int D, int MODE>
__device__ __forceinline__ void fetch(const AttnQ8Plan &p, const TokensQ8<MODE> &x, int64_t head, int wave,
                                      int lane, StageQ8<D> &stage) {
  using S = RowsShape<D>;
  using Sc = ScalesOf<D, MODE>;
  const uint8_t *k, *v;
  uint32_t k_at, v_at;
  const float *scale;
  const bool keys = lane < Sc::EACH;
  if constexpr (MODE != kAny) {
    const int64_t page = uniform64(x.page), row = x.row;
    k = p.k.codes + page * p.k.page + head * p.k.head + row * p.k.row;
    v = p.v.codes + page * p.v.page + head * p.v.head + row * p.v.row;
    const int32_t token = min(S::token(wave, lane), x.more);
    k_at = uint32_t(token * p.k.row + S::piece(lane) * 16);
    v_at = uint32_t(token * p.v.row + S::piece(lane) * 16);
    const float *ks = p.k.scales + page * p.k.s_page + head * p.k.s_head;
    const float *vs = p.v.scales + page * p.v.s_page + head * p.v.s_head;
    const int32_t at = x.row + min(Sc::token(wave, lane), x.more);
    scale = (keys ? ks : vs) +
            int64_t(div_by(p.div_block, uint32_t(at))) * (keys ? p.k.s_block : p.v.s_block);
  } else {
    k = p.k.codes + x.page * p.k.page + head * p.k.head + int64_t(x.row) * p.k.row;
    v = p.v.codes + x.page * p.v.page + head * p.v.head + int64_t(x.row) * p.v.row;
    k_at = v_at = uint32_t(S::piece(lane) * 16);
    const Q8Cache &c = keys ? p.k : p.v;
    scale = c.scales + x.scale_page * c.s_page + head * c.s_head +
            int64_t(div_by(p.div_block, uint32_t(x.scale_row))) * c.s_block;
  }
#pragma unroll
  for (int i = 0; i < S::BYTES / 16; ++i) {
    stage.k[i] = *reinterpret_cast<const uint4 *>(k + (k_at + 16 * S::THREADS * i));
    stage.v[i] = *reinterpret_cast<const uint4 *>(v + (v_at + 16 * S::THREADS * i));
  }
  stage.scale = *scale;
}

// Into a buffer, as operands.  look: some rows see the tile in part, so that NaN among its values are marked.
template <typename T, int D, bool E4M3, int MODE>
__device__ __forceinline__ void put(StageQ8<D> &x, int tid, float scale_log2, bool look,
                                    typename RowsLds<D>::Buffer &to, int32_t *nans) {
  using S = RowsShape<D>;
  using Op = Operand<T, E4M3>;
  const int wave = tid / 64, lane = tid & 63;
  const uint32_t row = uint32_t(S::run(wave) + S::token(wave, lane));
  const uint32_t piece = uint32_t(S::piece(lane));  // four to a panel's row, two chunks each
  if constexpr (E4M3) {
    if (look) {
      asm volatile("");
      uint32_t found = 0;
#pragma unroll
      for (int i = 0; i < S::BYTES / 16; ++i)
        found |= mark_nans(&x.v[i].x) | mark_nans(&x.v[i].y) | mark_nans(&x.v[i].z) | mark_nans(&x.v[i].w);
      const bool any = __any(found != 0);
      if (lane == 0) nans[wave] = any;
    }
  }
#pragma unroll
  for (int i = 0; i < S::BYTES / 16; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t at = (piece / 4 + uint32_t(S::THREADS / 4 * i)) * S::PANEL +
                          (panel_chunk(row, piece % 4 * 2) ^ uint32_t(16 * e));
      const s16x8 k = e == 0 ? Op::row(x.k[i].x, x.k[i].y) : Op::row(x.k[i].z, x.k[i].w);
      const s16x8 v = e == 0 ? Op::row(x.v[i].x, x.v[i].y) : Op::row(x.v[i].z, x.v[i].w);
      *reinterpret_cast<s16x8 *>(to.k + at) = k;
      *reinterpret_cast<s16x8 *>(to.v + at) = v;
    }
  using Sc = ScalesOf<D, MODE>;
  const int at = Sc::place(wave * Sc::EACH + lane % Sc::EACH);
  if (lane < 2 * Sc::EACH)
    (lane < Sc::EACH ? to.k_scale : to.v_scale)[at] = lane < Sc::EACH ? x.scale * scale_log2 : x.scale;
}

// The scales of the lane's tokens of block kb of 32 in S^T: four by four.
template <int D, int MODE>
__device__ __forceinline__ void scales_at(const float *s, int kb, int lane, f32x4 (&f)[4]) {
  if constexpr (MODE == kCoarse) {
    const f32x4 y = *reinterpret_cast<const f32x4 *>(s + (lane >> 5) * (RowsShape<D>::TILE / 8) + kb * 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) f[c] = f32x4{y[c], y[c], y[c], y[c]};
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      f[c] = *reinterpret_cast<const f32x4 *>(s + kb * 32 + c * 8 + 4 * (lane >> 5));
  }
}

template <typename T, int D, bool E4M3, int MODE>
__global__ __launch_bounds__(kAttnBlock) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2))) void
attention_q8_rows_kernel(AttnQ8Plan p) {
  using S = RowsShape<D>;
  constexpr int TILE = S::TILE, KB = TILE / 32, ROWS = int(kQ8ManyRows), DB = D / 32;
  __shared__ __attribute__((aligned(16))) RowsLds<D> lds;
  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  ShareQ8<ROWS> share = {{p}};
  if (!share.begin(lds.share)) return;
  do {
    const SegmentQ8 g = share.segment();
    if (g.st0 >= g.st1) continue;
    const SequenceQ8 &sq = share.sq;
    const int32_t b = share.b, last = sq.len - 1;
    const int64_t head = g.set;

    // ---- the lane's query row ----
    const int32_t m = wave * 32 + (lane & 31);
    const bool some = m < g.live;
    const int32_t tok = int32_t(div_by(p.div_group, uint32_t(g.row0 + (some ? m : 0))));
    const int32_t limit = some ? g.hidden + tok : 0;
    const int32_t floor = g.hidden + int32_t(div_by(p.div_group, uint32_t(g.row0 + min(wave * 32, g.live - 1))));
    const int32_t lowest = g.hidden + int32_t(div_by(p.div_group, uint32_t(g.row0)));  // of all wavefronts
    s16x8 q[D / 16];
    {
      const int32_t h = g.set * p.group + g.row0 + (some ? m : 0) - tok * p.group;
      const T *from = static_cast<const T *>(p.q) + int64_t(sq.first + tok) * p.q_tok +
                      int64_t(h) * p.q_head + 8 * (lane >> 5);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        q[i] = some ? as_operand(*reinterpret_cast<const uint4 *>(from + 16 * i)) : s16x8{};
    }
    float top = kNegInf, sum = 0.0f;
    float by_reach = kFirstByReach;  // as in StateQ8
    f32x16 o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] = f32x16{};

    uint32_t keys_at = panel_chunk(uint32_t(lane & 31), uint32_t(lane >> 5));
    uint32_t values_at = panel_transposed(uint32_t(lane), 0, 0);

    // ---- the steps that a row of the tile sees ----
    const int32_t end = min(g.st1 * TILE, g.most);
    int32_t t0 = g.st0 * TILE;
    if (t0 < end) {
      auto at_tile = [&](int32_t t) { return tokens_at<D, MODE>(p.seq, b, t, last, wave, lane); };
      StageQ8<D> stage;
      fetch<D, MODE>(p, at_tile(t0), head, wave, lane, stage);
      lds_barrier();  // what the last piece read of the buffers
      put<T, D, E4M3, MODE>(stage, tid, p.scale_log2, t0 + TILE > lowest, lds.buffer[0], lds.nans[0]);
      int32_t t1 = t0 + TILE < end ? t0 + TILE : t0;
      TokensQ8<MODE> tokens = at_tile(t1);
      for (int32_t n = 0;; ++n) {  // ends: t0 grows
        lds_barrier();
        // the next tile's codes on their way (the present one's again behind the last: no branch)
        fetch<D, MODE>(p, tokens, head, wave, lane, stage);
        const int32_t t2 = t1 + TILE < end ? t1 + TILE : t1;
        tokens = at_tile(t2);
        const typename RowsLds<D>::Buffer &at = lds.buffer[n & 1];

        // Opaque: the places that follow from these are worked out again in every step.  Kept from step to
        // step they would take registers that the products need.
        asm volatile("" : "+v"(keys_at), "+v"(values_at));
        // S^T
        f32x16 x[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) x[kb] = f32x16{};
        constexpr int AHEAD = 2;  // products whose operands are read ahead
        s16x8 kf[AHEAD + 1][KB];
        auto load_keys = [&](int i) {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            kf[i % (AHEAD + 1)][kb] = *reinterpret_cast<const s16x8 *>(
                at.k + i / 4 * S::PANEL + kb * 4096 + (keys_at ^ (i % 4 * 32u)));
        };
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) load_keys(i);
        __builtin_amdgcn_s_setprio(1);  // the other wavefront's exponentials fill the pauses
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if (i + AHEAD < D / 16) load_keys(i + AHEAD);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) x[kb] = Mfma<T>::mul(kf[i % (AHEAD + 1)][kb], q[i], x[kb]);
          __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
        // scores in powers of two, masked where not every row of the wavefront sees all of the tile
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          f32x4 f[4];
          scales_at<D, MODE>(at.k_scale, kb, lane, f);
#pragma unroll
          for (int r = 0; r < 16; ++r) x[kb][r] *= f[r / 4][r % 4];
        }
        const bool masked = t0 + TILE > floor;
        if (masked) {
          asm volatile("");
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (t0 + kb * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4 >= limit) x[kb][r] = kNegInf;
        }
        float best = kNegInf;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int r = 0; r < 16; ++r) best = fmaxf(best, x[kb][r]);
        best = max_halves(best);
        bool raise = best > top + Mfma<T>::kSlack;
        float most = 0.0f;
        if constexpr (Mfma<T>::kNarrow) {
          most = fabsf(at.v_scale[lane % ScalesOf<D, MODE>::COUNT]);
          if (masked) {  // of the lane's tokens that its row sees
            asm volatile("");
            most = 0.0f;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
              f32x4 f[4];
              scales_at<D, MODE>(at.v_scale, kb, lane, f);
#pragma unroll
              for (int r = 0; r < 16; ++r)
                if (t0 + kb * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4 < limit)
                  most = fmaxf(most, fabsf(f[r / 4][r % 4]));
            }
          }
          raise |= most * by_reach > 1.0f;
        }
        if (__any(raise)) {
          float f = 1.0f;
          if (best > top + Mfma<T>::kSlack) {
            f = __builtin_amdgcn_exp2f(top - best);
            top = best;
          }
          sum *= f;
          if constexpr (Mfma<T>::kNarrow) {
            if (masked)
              most = max_halves(most);
            else
              for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
            const float by = most * by_reach > 1.0f ? inverse_power(reach_above(most)) : by_reach;
            f *= by * inverse_power(by_reach);
            by_reach = by;
          }
#pragma unroll
          for (int d = 0; d < DB; ++d) o[d] *= f;
        }
        const float ref = top == kNegInf ? 0.0f : top - Mfma<T>::kLift;
        s16x8 w[KB][2];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          float e[16];
          f32x4 f[4];
          scales_at<D, MODE>(at.v_scale, kb, lane, f);
          if constexpr (Mfma<T>::kNarrow) {
#pragma unroll
            for (int c = 0; c < 4; ++c) f[c] *= by_reach;
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float y = __builtin_amdgcn_exp2f(x[kb][r] - ref);
            sum += y;
            e[r] = y * f[r / 4][r % 4];
          }
          if (masked) {
            asm volatile("");
#pragma unroll
            for (int r = 0; r < 16; ++r)  // whatever the scale of a token that the row does not see
              if (t0 + kb * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4 >= limit) e[r] = 0.0f;
          }
          w[kb][0] = round8<T>(e);
          w[kb][1] = round8<T>(e + 8);
        }
        // O^T += V^T P^T
        constexpr int V_AHEAD = 3, PRODUCTS = KB * 2 * DB;
        s16x8 vf[V_AHEAD + 1];
        auto load_values = [&](int n) {  // 16 tokens n / DB, columns 32 (n % DB) and on
          const char *from = at.v + n % DB / 2 * S::PANEL + n / DB * 2048;
          const uint32_t v = values_at ^ (n % DB % 2 * 64u);
          vf[n % (V_AHEAD + 1)] = join(read_transposed(from + v), read_transposed(from + (v ^ kEightRows)));
        };
#pragma unroll
        for (int n = 0; n < V_AHEAD; ++n) load_values(n);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int n = 0; n < PRODUCTS; ++n) {
          if (n + V_AHEAD < PRODUCTS) load_values(n + V_AHEAD);
          __builtin_amdgcn_sched_barrier(0);
          o[n % DB] = Mfma<T>::mul(vf[n % (V_AHEAD + 1)], w[n / DB / 2][n / DB % 2], o[n % DB]);
          __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
        if constexpr (E4M3) {
          if (t0 + TILE > lowest) {  // put has looked
            asm volatile("");
            if (__any(lds.nans[n & 1][lane % kAttnWaves])) {  // outputs of rows that see a token with a NaN
#pragma unroll
              for (int d = 0; d < DB; ++d) {
                f32x16 nans = {};
#pragma unroll
                for (int k = 0; k < 2 * KB; ++k) {
                  const char *from = at.v + d / 2 * S::PANEL + k * 2048;
                  const uint32_t v = values_at ^ (d % 2 * 64u);
                  const s16x8 a = join(read_transposed(from + v), read_transposed(from + (v ^ kEightRows)));
                  float one[8];
#pragma unroll
                  for (int r = 0; r < 8; ++r)
                    one[r] = t0 + k * 16 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4 < limit ? 1.0f : 0.0f;
                  nans = Mfma<T>::mul(marked<T>(a), round8<T>(one), nans);
                  __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) o[d][r] = nans[r] > 0.0f ? __builtin_nanf("") : o[d][r];
              }
            }
          }
        }
        if (t1 == t0) break;
        put<T, D, E4M3, MODE>(stage, tid, p.scale_log2, t1 + TILE > lowest, lds.buffer[~n & 1],
                              lds.nans[~n & 1]);
        t0 = t1;
        t1 = t2;
      }
    }
    sum = sum_halves(sum);

    // ---- the piece's result ----
    if (some) {
      const float unit = Mfma<T>::kNarrow ? inverse_power(by_reach) : 1.0f;
      if (g.whole()) {
        const int64_t row = output_row(p, g, g.set, sq.first, m);
        const bool any = sum > 0.0f || sum != sum;  // a row that sees nothing gets zeros
        const float inv = any ? unit / sum : 0.0f;
        char *out = static_cast<char *>(p.out) + row * (2 * D) + 8 * (lane >> 5);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint2 *>(out + d * 64 + c * 16) =
                make_uint2(Mfma<T>::pack(o[d][4 * c] * inv, o[d][4 * c + 1] * inv),
                           Mfma<T>::pack(o[d][4 * c + 2] * inv, o[d][4 * c + 3] * inv));
        if (lane < 32 && p.lse != nullptr) p.lse[row] = any ? natural<T>(top, sum) : kNegInf;
      } else {
        const int64_t row = (int64_t(blockIdx.x) * 2 + g.part) * ROWS + m;
        float *to = p.parts + row * D + 4 * (lane >> 5);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<f32x4 *>(to + d * 32 + c * 8) =
                f32x4{o[d][4 * c], o[d][4 * c + 1], o[d][4 * c + 2], o[d][4 * c + 3]} * unit;
        if (lane < 32) *reinterpret_cast<float2 *>(p.stats + row * 2) = make_float2(top, sum);
      }
    }
    share.note(g);
  } while (share.next());
}

template <typename T, int D, int R>
const void *pick_attention_q8(const AttnQ8Plan &p) {
#define ROPE_KQ(E, MO) reinterpret_cast<const void *>(&attention_q8_kernel<T, D, R, E, MO>)
#define ROPE_KM(E) (p.mode == kCoarse ? ROPE_KQ(E, kCoarse) : p.mode == kFine ? ROPE_KQ(E, kFine) : ROPE_KQ(E, kAny))
  return p.e4m3 ? ROPE_KM(true) : ROPE_KM(false);
#undef ROPE_KM
#undef ROPE_KQ
}

template <typename T, int D>
const void *pick_attention_q8(const AttnQ8Plan &p) {
  if (p.rows == kQ8ManyRows) {
#define ROPE_KR(E, MO) reinterpret_cast<const void *>(&attention_q8_rows_kernel<T, D, E, MO>)
#define ROPE_KM(E) (p.mode == kCoarse ? ROPE_KR(E, kCoarse) : p.mode == kFine ? ROPE_KR(E, kFine) : ROPE_KR(E, kAny))
    return p.e4m3 ? ROPE_KM(true) : ROPE_KM(false);
#undef ROPE_KM
#undef ROPE_KR
  }
  return p.rows == 16 ? pick_attention_q8<T, D, 1>(p) : pick_attention_q8<T, D, 2>(p);
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
