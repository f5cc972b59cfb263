// rope_latent_paged.hip -- latent attention over a paged cache, absorbed form (gfx950).
//
// Every head h of query token i of a sequence attends to the sequence's cached latent rows c_j
// (latent_dim elements and a rotated tail of 64), the last query seeing all of them and each
// earlier one a row less:
//   s_j = scale <q_ih, c_j>,   p = softmax(s),   out_ih = sum_j p_j c_j[0 : latent_dim]
// The cache row is key and value at once and is shared by all heads, so a row is read from HBM
// once for up to 128 (token, head) pairs: 2 (latent_dim + 64 + latent_dim) operations a pair and
// a row of 1152 bytes (latent_dim 512) leave the call bound by HBM up to about 128 heads, if the
// loads never pause.
//
// One pass, running maximum and sum in float32.  A workgroup is four wavefronts and 32 or 64
// query rows.  Cache rows pass through LDS, 64 at a time in two buffers that direct-to-LDS loads
// fill one step ahead.  S^T = K Q^T is split between the wavefronts by cache rows (and query
// rows), so that Q stays in registers as the second operand (144 of them at latent_dim 512);
// O^T = V^T P^T is split by columns of V, so that a wavefront accumulates a quarter of the
// latent for all rows (64 or 128 registers) and every byte of the tile is read for it once, by
// transposed LDS reads.  In between P goes through LDS, rounded to the storage type: a relative
// error of at most half a step on each weight, as on the output itself.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "rope.h"
#include "rope_latent_plan.h"
#include "rope_launch.h"
#include "rope_mfma.h"

namespace ropeamd {
namespace {

constexpr int kPagedBlock = 256;
constexpr int kPageIds = 1024;  // page numbers held in LDS at a time

__device__ inline uint32_t div_by(const FastDiv &f, uint32_t n) {
  const uint32_t t = __umulhi(f.m, n);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}

// What a sequence asks for.
struct Sequence {
  int32_t len;     // cached tokens
  int32_t first;   // first query token
  int32_t count;   // query tokens
  int32_t items;
  int32_t steps;   // of one item
};

// Lengths and offsets are device data: values outside their ranges are clamped, so that no
// access leaves the tensors.
__device__ inline Sequence sequence(const PagedPlan &p, int32_t b, int rows, int step) {
  Sequence s;
  const int64_t cap = p.max_pages * p.page_size;
  s.len = int32_t(min(max(p.lens[b * p.len_stride], int64_t(0)), cap));
  if (p.offsets != nullptr) {
    const int64_t o0 = min(max(p.offsets[b * p.off_stride], int64_t(0)), p.T);
    const int64_t o1 = min(max(p.offsets[(b + 1) * p.off_stride], o0), p.T);
    s.first = int32_t(o0);
    s.count = int32_t(o1 - o0);
  } else {
    s.first = int32_t(b * p.queries);
    s.count = int32_t(p.queries);
  }
  s.items = (s.count * p.heads + rows - 1) / rows;
  s.steps = max(1, (s.len + step - 1) / step);
  return s;
}

// Inclusive sum over the wavefront.
__device__ inline int64_t wave_scan(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}

// A wavefront's quarter of a tile of 64 cache rows (tokens tile0 .. tile0 + 63, the last one
// repeated past `len`) into LDS: 16 rows of each 64-element panel.
template <typename T, int PANELS>
__device__ __forceinline__ void fetch_tile(const PagedPlan &p, const int32_t *ids, int32_t page0,
                                           int32_t tile0, int32_t len, int wave, int lane,
                                           char *__restrict__ tile) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int rb = wave * 2 + i;  // 8-row block
    const int32_t tok = min(tile0 + 8 * rb + (lane >> 3), len - 1);
    const int32_t page = int32_t(div_by(p.div_page, uint32_t(tok)));
    const int64_t off = int64_t(ids[page - page0]) * p.c_page +
                        int64_t(tok - page * int32_t(p.page_size)) * p.c_row;
    const char *row = static_cast<const char *>(p.cache) + off * int64_t(sizeof(T)) +
                      ((uint32_t(lane & 7) ^ chunk_key(uint32_t(lane >> 3))) << 4);
#pragma unroll
    for (int n = 0; n < PANELS; ++n) load_lds16(row + n * 128, tile + n * 8192 + rb * 1024);
  }
}

// Running maximum of a row: raised (and what was summed at the old one rescaled by the returned
// factor) only when the tile's maximum passes it by more than 8, so that rescaling is rare.
// Until then weights of up to 2^8 are carried, which changes no result beyond its rounding.
__device__ inline float raise(float &top, float best) {
  float f = 1.0f;
  if (best > top + 8.0f) {
    f = __builtin_amdgcn_exp2f(top - best);
    top = best;
  }
  return f;
}

// One tile.  seen: cache rows of the tile that a query row may see (per lane and row block);
// whole: whether every row sees all of it.
template <typename T, int DB, int RB>
struct Step {
  static constexpr int PANELS = DB / 2 + 1;
  static constexpr int ROWS = 32 * RB;
  static constexpr int SB = RB == 1 ? 2 : 1;    // row blocks of a wavefront in S
  static constexpr int PARTS = RB == 1 ? 4 : 2;  // wavefronts that share a row's cache rows in S
  static constexpr int QF = RB == 1 ? PANELS * 2 : PANELS * 4;
  static constexpr int COLS = DB / 4;            // 32-column blocks of a wavefront in O

  // Row of the workgroup that this lane owns in S (block i), and in O (block i).
  __device__ static int s_row(int wave, int lane, int i) {
    return RB == 1 ? i * 16 + (lane & 15) : (wave >> 1) * 32 + (lane & 31);
  }
  __device__ static int s_part(int wave) { return RB == 1 ? wave : wave & 1; }

  // S^T of the wavefront's cache rows; scaled, masked; returns the rows' maxima.
  __device__ __forceinline__ static void scores(const char *__restrict__ tile,
                                                const s16x8 (&qf)[SB][QF], int wave, int lane,
                                                const int32_t (&seen)[SB], bool whole,
                                                float scale_log2, float (&e)[SB][RB == 1 ? 4 : 16],
                                                float (&best)[SB]) {
    if constexpr (RB == 1) {
      f32x4 s[SB] = {};
      const uint32_t row = uint32_t(wave * 16 + (lane & 15));
#pragma unroll
      for (int n = 0; n < PANELS; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const s16x8 kf = as_operand(*reinterpret_cast<const uint4 *>(
              tile + n * 8192 + panel_chunk(row, 4u * c + (uint32_t(lane) >> 4))));
#pragma unroll
          for (int i = 0; i < SB; ++i) s[i] = Mfma<T>::mul16(kf, qf[i][n * 2 + c], s[i]);
        }
#pragma unroll
      for (int i = 0; i < SB; ++i) {
        best[i] = kNegInf;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = s[i][r] * scale_log2;
          if (!whole) x = wave * 16 + 4 * (lane >> 4) + r < seen[i] ? x : kNegInf;
          e[i][r] = x;
          best[i] = fmaxf(best[i], x);
        }
        best[i] = fmaxf(best[i], __shfl_xor(best[i], 16, 64));
        best[i] = fmaxf(best[i], other_half(best[i]));
      }
    } else {
      f32x16 s = {};
      const uint32_t row = uint32_t((wave & 1) * 32 + (lane & 31));
#pragma unroll
      for (int n = 0; n < PANELS; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const s16x8 kf = as_operand(*reinterpret_cast<const uint4 *>(
              tile + n * 8192 + panel_chunk(row, 2u * c + (uint32_t(lane) >> 5))));
          s = Mfma<T>::mul(kf, qf[0][n * 4 + c], s);
        }
      best[0] = kNegInf;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float x = s[r] * scale_log2;
        if (!whole)
          x = (wave & 1) * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4 < seen[0] ? x : kNegInf;
        e[0][r] = x;
        best[0] = fmaxf(best[0], x);
      }
      best[0] = fmaxf(best[0], other_half(best[0]));
    }
  }

  // Weights of four cache rows (4 g4 .. + 3 of the tile) of query row `row` into the P tile, in
  // the order the second product takes them: a 16-byte chunk 2 k + h holds cache rows
  // 16 k + 4 h + {0..3} and those 8 further on.
  __device__ static void put_weights(char *__restrict__ pt, int row, int g4, const float *e) {
    const uint32_t chunk = uint32_t(2 * (g4 >> 2) + (g4 & 1));
    *reinterpret_cast<uint2 *>(pt + panel_chunk(uint32_t(row), chunk) + ((g4 >> 1) & 1) * 8) =
        make_uint2(Mfma<T>::pack(e[0], e[1]), Mfma<T>::pack(e[2], e[3]));
  }

  // O^T += V^T P^T over the tile.
  __device__ __forceinline__ static void outputs(const char *__restrict__ tile,
                                                 const char *__restrict__ pt, int wave, int lane,
                                                 f32x16 (&acc)[RB][COLS]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s16x8 pf[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i)
        pf[i] = as_operand(*reinterpret_cast<const uint4 *>(
            pt + panel_chunk(uint32_t(i * 32 + (lane & 31)), uint32_t(2 * k + (lane >> 5)))));
#pragma unroll
      for (int d = 0; d < COLS; ++d) {
        const int block = wave * COLS + d;
        const char *at = tile + (block >> 1) * 8192 + k * 2048 +
                         panel_transposed(uint32_t(lane), uint32_t(block & 1));
        const s16x8 vf = join(read_transposed(at), read_transposed(at + 1024));
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[i][d] = Mfma<T>::mul(vf, pf[i], acc[i][d]);
      }
    }
  }
};

template <typename T, int DB, int RB>
__global__ __launch_bounds__(kPagedBlock) __attribute__((amdgpu_waves_per_eu(1, 1))) void
latent_paged_kernel(PagedPlan p) {
  using S = Step<T, DB, RB>;
  constexpr int PANELS = S::PANELS, ROWS = S::ROWS, SB = S::SB;
  constexpr int STEP = int(kPagedStep);
  constexpr int TILE = PANELS * 8192;  // bytes
  constexpr int SE = RB == 1 ? 4 : 16;
  __shared__ __attribute__((aligned(16))) char tiles[2 * TILE];
  __shared__ __attribute__((aligned(16))) char weights[ROWS * 128];
  __shared__ int32_t ids[kPageIds];
  __shared__ float row_max[S::PARTS][ROWS];
  __shared__ int64_t wave_total[4];
  __shared__ int64_t found_before;
  __shared__ int32_t found_seq;

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the workgroups of a cluster are kXcds apart: on one XCD, they share its L2
  const int32_t turn = int32_t(blockIdx.x / kXcds);
  const int32_t g = (turn / p.cluster) * int32_t(kXcds) + int32_t(blockIdx.x % kXcds);
  const int32_t member = turn % p.cluster;
  const int32_t item_rows = ROWS * p.cluster;

  // ---- the cluster's share [w0, w1) of all steps ----
  int64_t mine = 0;
  for (int32_t b = tid; b < p.B; b += kPagedBlock) {
    const Sequence s = sequence(p, b, item_rows, STEP);
    mine += int64_t(s.items) * s.steps;
  }
  const int64_t wave_sum = __shfl(wave_scan(mine, lane), 63, 64);
  if (lane == 0) wave_total[wave] = wave_sum;
  __syncthreads();
  const int64_t total = wave_total[0] + wave_total[1] + wave_total[2] + wave_total[3];
  const int64_t per = (total + p.clusters - 1) / p.clusters;
  const int64_t w0 = g * per, w1 = min(total, w0 + per);
  if (w0 >= w1) {
    if (tid == 0 && member == 0) p.joins[g * 4 + 3] = 0;
    return;
  }
  // the sequence that holds step w0
  int64_t before = 0;
  for (int32_t b0 = 0; b0 < p.B; b0 += kPagedBlock) {
    const int32_t b = b0 + tid;
    int64_t n = 0;
    if (b < p.B) {
      const Sequence s = sequence(p, b, item_rows, STEP);
      n = int64_t(s.items) * s.steps;
    }
    const int64_t incl = wave_scan(n, lane);
    __syncthreads();
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    int64_t base = before;
    for (int v = 0; v < wave; ++v) base += wave_total[v];
    const int64_t chunk = wave_total[0] + wave_total[1] + wave_total[2] + wave_total[3];
    if (n > 0 && base + incl - n <= w0 && w0 < base + incl) {
      found_seq = b;
      found_before = base + incl - n;
    }
    before += chunk;
    if (w0 < before) break;
  }
  __syncthreads();
  int32_t b = __builtin_amdgcn_readfirstlane(found_seq);
  Sequence sq = sequence(p, b, item_rows, STEP);
  const int64_t into = w0 - found_before;
  int32_t item = int32_t(into / sq.steps);
  int32_t st0 = int32_t(into - int64_t(item) * sq.steps);
  int64_t w = w0;
  bool joined = false;

  while (true) {
    const int32_t st1 = int32_t(min(int64_t(sq.steps), st0 + (w1 - w)));
    const int32_t rows = sq.count * p.heads;
    const int32_t row0 = item * item_rows + member * ROWS;
    if (row0 < rows) {
      // ---- this wavefront's query rows, and how much of the cache each may see ----
      s16x8 qf[SB][S::QF];
      int32_t limit[SB];
#pragma unroll
      for (int i = 0; i < SB; ++i) {
        const int32_t r = row0 + S::s_row(wave, lane, i);
        const bool live = r < rows;
        const int32_t qi = live ? int32_t(div_by(p.div_heads, uint32_t(r))) : 0;
        const int32_t head = live ? r - qi * p.heads : 0;
        limit[i] = live ? sq.len - sq.count + qi + 1 : 0;
        const T *q = static_cast<const T *>(p.q) + int64_t(sq.first + qi) * p.q_tok +
                     int64_t(head) * p.q_head + 8 * (RB == 1 ? lane >> 4 : lane >> 5);
#pragma unroll
        for (int k = 0; k < S::QF; ++k)
          qf[i][k] = live ? as_operand(*reinterpret_cast<const uint4 *>(q + k * (RB == 1 ? 32 : 16)))
                          : s16x8{};
      }
      // fewest cache rows that any row of the workgroup sees
      const int32_t floor = row0 + ROWS > rows
                                ? 0
                                : sq.len - sq.count + int32_t(div_by(p.div_heads, uint32_t(row0))) + 1;

      float s_top[SB], s_sum[SB], o_top[RB];
      f32x16 acc[RB][S::COLS];
#pragma unroll
      for (int i = 0; i < SB; ++i) s_top[i] = kNegInf, s_sum[i] = 0.0f;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        o_top[i] = kNegInf;
#pragma unroll
        for (int d = 0; d < S::COLS; ++d) acc[i][d] = f32x16{};
      }

      auto step = [&](const char *__restrict__ cur, char *__restrict__ other,
                      char *__restrict__ pt, int32_t tile0, int32_t next0, int32_t page0) {
        if (next0 >= 0) fetch_tile<T, PANELS>(p, ids, page0, next0, sq.len, wave, lane, other);
        int32_t seen[SB];
#pragma unroll
        for (int i = 0; i < SB; ++i) seen[i] = limit[i] - tile0;
        float e[SB][SE], best[SB];
        S::scores(cur, qf, wave, lane, seen, tile0 + STEP <= floor, p.scale_log2, e, best);
#pragma unroll
        for (int i = 0; i < SB; ++i)
          if (lane < (RB == 1 ? 16 : 32))
            row_max[S::s_part(wave)][S::s_row(wave, lane, i)] = best[i];
        lds_barrier();
#pragma unroll
        for (int i = 0; i < SB; ++i) {
          const int row = S::s_row(wave, lane, i);
          float high = row_max[0][row];
#pragma unroll
          for (int k = 1; k < S::PARTS; ++k) high = fmaxf(high, row_max[k][row]);
          s_sum[i] *= raise(s_top[i], high);
          const float ref = s_top[i] == kNegInf ? 0.0f : s_top[i];
#pragma unroll
          for (int r = 0; r < SE; ++r) {
            e[i][r] = __builtin_amdgcn_exp2f(e[i][r] - ref);
            s_sum[i] += e[i][r];
          }
          if constexpr (RB == 1) {
            S::put_weights(pt, row, wave * 4 + (lane >> 4), e[i]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              S::put_weights(pt, row, (wave & 1) * 8 + 2 * c + (lane >> 5), e[i] + 4 * c);
          }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const int row = i * 32 + (lane & 31);
          float high = row_max[0][row];
#pragma unroll
          for (int k = 1; k < S::PARTS; ++k) high = fmaxf(high, row_max[k][row]);
          const float f = raise(o_top[i], high);
          if (__any(f != 1.0f)) {
#pragma unroll
            for (int d = 0; d < S::COLS; ++d) acc[i][d] *= f;
          }
        }
        lds_barrier();
        S::outputs(cur, pt, wave, lane, acc);
      };

      if (sq.len > 0) {
        int32_t st = st0;
        while (st < st1) {
          // ---- page numbers of as many of the segment's steps as the table holds ----
          const int32_t page0 = int32_t(div_by(p.div_page, uint32_t(st * STEP)));
          const int32_t last_tok = min(st1 * STEP, sq.len) - 1;
          const int32_t pages = min(int32_t(kPageIds),
                                    int32_t(div_by(p.div_page, uint32_t(last_tok))) - page0 + 1);
          __syncthreads();
          for (int32_t i = tid; i < pages; i += kPagedBlock) {
            const int64_t id = p.table[b * p.table_seq + (page0 + i) * p.table_page];
            ids[i] = int32_t(min(max(id, int64_t(0)), p.num_pages - 1));
          }
          __syncthreads();
          int32_t end = st1;
          if (int64_t(page0 + pages) * p.page_size <= last_tok)
            end = int32_t((int64_t(page0 + pages) * p.page_size) / STEP);
          // ---- the steps: the next tile is on its way while one is multiplied ----
          fetch_tile<T, PANELS>(p, ids, page0, st * STEP, sq.len, wave, lane, tiles);
          for (int32_t n = 0; st < end; ++st, ++n) {
            wait_loads_all();
            lds_barrier();
            step(tiles + (n & 1) * TILE, tiles + (~n & 1) * TILE, weights, st * STEP,
                 st + 1 < end ? (st + 1) * STEP : -1, page0);
          }
        }
      }

      // ---- sums of the wavefronts that shared a row ----
      __syncthreads();
#pragma unroll
      for (int i = 0; i < SB; ++i) {
        if constexpr (RB == 1) s_sum[i] += __shfl_xor(s_sum[i], 16, 64);
        s_sum[i] += other_half(s_sum[i]);
        if (lane < (RB == 1 ? 16 : 32))
          row_max[S::s_part(wave)][S::s_row(wave, lane, i)] = s_sum[i];
      }
      __syncthreads();

      // ---- the segment's result: a whole item's output, or a part for the joining kernel ----
      const bool whole = st0 == 0 && st1 == sq.steps;
      const int64_t slot = (int64_t(g) * p.cluster + member) * 2 + (w == w0 ? 0 : 1);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const int m = i * 32 + (lane & 31);
        float sum = row_max[0][m];
#pragma unroll
        for (int k = 1; k < S::PARTS; ++k) sum += row_max[k][m];
        const int32_t r = row0 + m;
        const int64_t out_row = int64_t(sq.first) * p.heads + r;
        const bool some = sum > 0.0f || sum != sum;  // a row that sees nothing gets zeros
        if (whole) {
          if (r < rows) {
            const float inv = some ? 1.0f / sum : 0.0f;
            char *out = static_cast<char *>(p.out) + out_row * p.latent * int64_t(sizeof(T));
#pragma unroll
            for (int d = 0; d < S::COLS; ++d)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const f32x16 &a = acc[i][d];
                const int d4 = (wave * S::COLS + d) * 8 + c * 2 + (lane >> 5);
                *reinterpret_cast<uint2 *>(out + d4 * 8) =
                    make_uint2(Mfma<T>::pack(a[4 * c] * inv, a[4 * c + 1] * inv),
                               Mfma<T>::pack(a[4 * c + 2] * inv, a[4 * c + 3] * inv));
              }
            if (wave == 0 && lane < 32 && p.lse != nullptr)
              p.lse[out_row] = some ? o_top[i] * 0.693147180559945f + logf(sum) : kNegInf;
          }
        } else {
          float *part = p.parts + slot * ROWS * p.latent + m * 4;
#pragma unroll
          for (int d = 0; d < S::COLS; ++d)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const f32x16 &a = acc[i][d];
              const int d4 = (wave * S::COLS + d) * 8 + c * 2 + (lane >> 5);
              *reinterpret_cast<float4 *>(part + d4 * (ROWS * 4)) =
                  make_float4(a[4 * c], a[4 * c + 1], a[4 * c + 2], a[4 * c + 3]);
            }
          if (wave == 0 && lane < 32)
            *reinterpret_cast<float2 *>(p.stats + (slot * ROWS + m) * 2) =
                make_float2(o_top[i], sum);
        }
      }
    }
    // an item that began here and goes on in the next clusters is joined afterwards
    if (st0 == 0 && st1 < sq.steps) {
      joined = true;
      if (tid == 0 && member == 0) {
        p.joins[g * 4 + 0] = b;
        p.joins[g * 4 + 1] = item;
        p.joins[g * 4 + 2] = w == w0 ? 0 : 1;
        p.joins[g * 4 + 3] = int32_t((w + sq.steps - 1) / per - g + 1);
      }
    }
    w += st1 - st0;
    if (w >= w1) break;
    st0 = 0;
    if (++item >= sq.items) {
      item = 0;
      do {  // ends: w < w1 <= total, so a later sequence has items
        ++b;
        sq = sequence(p, b, item_rows, STEP);
      } while (sq.items == 0);
    }
  }
  if (!joined && tid == 0 && member == 0) p.joins[g * 4 + 3] = 0;
}

// Joins the parts of the item that began in a cluster's share: a part k holds
// unnormalised outputs o_k at maximum m_k with weight sum l_k, and
//   out = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k,   m = max_k m_k.
// Four wavefronts share the parts of one (4-column group, row) and add up through LDS in a fixed
// order, so results do not depend on timing.
template <typename T, int DB, int RB>
__global__ __launch_bounds__(kPagedBlock) void latent_paged_join_kernel(PagedPlan p) {
  constexpr int ROWS = 32 * RB;
  constexpr int CELLS = DB * 8 * ROWS;  // (4-column group, row) pairs
  __shared__ float4 add[4][64];
  __shared__ float add_l[4][64], add_top[4][64];
  const int32_t g = int32_t(blockIdx.x) / p.cluster, member = int32_t(blockIdx.x) % p.cluster;
  const int32_t n = p.joins[g * 4 + 3];
  if (n <= 1) return;
  const int32_t b = p.joins[g * 4], item = p.joins[g * 4 + 1], first = p.joins[g * 4 + 2];
  const Sequence sq = sequence(p, b, ROWS * p.cluster, int(kPagedStep));
  const int32_t rows = sq.count * p.heads, row0 = (item * p.cluster + member) * ROWS;
  if (row0 >= rows) return;
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  auto slot = [&](int32_t k) {
    return (int64_t(g + k) * p.cluster + member) * 2 + (k == 0 ? first : 0);
  };
  for (int c0 = int(blockIdx.y) * 64; c0 < CELLS; c0 += int(gridDim.y) * 64) {
    const int cell = c0 + lane;
    const int m = cell % ROWS;
    // every wavefront joins its share of the parts at a maximum of its own
    float top = kNegInf, l = 0.0f;
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int32_t k = wave; k < n; k += 4) {
      const float2 stat = *reinterpret_cast<const float2 *>(p.stats + (slot(k) * ROWS + m) * 2);
      const float4 o =
          *reinterpret_cast<const float4 *>(p.parts + slot(k) * ROWS * p.latent + int64_t(cell) * 4);
      const float next = fmaxf(top, stat.x), ref = next == kNegInf ? 0.0f : next;
      const float fa = __builtin_amdgcn_exp2f(top - ref), fb = __builtin_amdgcn_exp2f(stat.x - ref);
      top = next;
      l = l * fa + stat.y * fb;
      t.x = t.x * fa + o.x * fb;
      t.y = t.y * fa + o.y * fb;
      t.z = t.z * fa + o.z * fb;
      t.w = t.w * fa + o.w * fb;
    }
    add[wave][lane] = t;
    add_l[wave][lane] = l;
    add_top[wave][lane] = top;
    __syncthreads();
    const int32_t r = row0 + m;
    if (wave == 0 && r < rows) {
      float high = top;
#pragma unroll
      for (int k = 1; k < 4; ++k) high = fmaxf(high, add_top[k][lane]);
      const float ref = high == kNegInf ? 0.0f : high;
      l = 0.0f;
      t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f = __builtin_amdgcn_exp2f(add_top[k][lane] - ref);
        const float4 y = add[k][lane];
        t.x += f * y.x;
        t.y += f * y.y;
        t.z += f * y.z;
        t.w += f * y.w;
        l += f * add_l[k][lane];
      }
      const bool some = l > 0.0f || l != l;
      const float inv = some ? 1.0f / l : 0.0f;
      const int64_t row = int64_t(sq.first) * p.heads + r;
      *reinterpret_cast<uint2 *>(static_cast<char *>(p.out) +
                                 row * p.latent * int64_t(sizeof(T)) + (cell / ROWS) * 8) =
          make_uint2(Mfma<T>::pack(t.x * inv, t.y * inv), Mfma<T>::pack(t.z * inv, t.w * inv));
      if (cell < ROWS && p.lse != nullptr)
        p.lse[row] = some ? high * 0.693147180559945f + logf(l) : kNegInf;
    }
    __syncthreads();
  }
}

template <typename T, int DB>
int run_paged(PagedPlan &p, void *stream) {
  const uint32_t groups = uint32_t(p.clusters * p.cluster);
  const bool two = p.row_blocks == 2;
  const void *fn = two ? reinterpret_cast<const void *>(&latent_paged_kernel<T, DB, 2>)
                       : reinterpret_cast<const void *>(&latent_paged_kernel<T, DB, 1>);
  const void *join = two ? reinterpret_cast<const void *>(&latent_paged_join_kernel<T, DB, 2>)
                         : reinterpret_cast<const void *>(&latent_paged_join_kernel<T, DB, 1>);
  const int st = launch_kernel(fn, dim3(groups), kPagedBlock, 0, stream, &p);
  if (st != ROPE_OK) return st;
  return launch_kernel(join, dim3(groups, uint32_t(p.join_slices)), kPagedBlock, 0, stream, &p);
}

template <typename T>
int run_paged_width(PagedPlan &p, void *stream) {
  return p.latent == 512   ? run_paged<T, 16>(p, stream)
         : p.latent == 256 ? run_paged<T, 8>(p, stream)
                           : run_paged<T, 4>(p, stream);
}

}  // namespace
}  // namespace ropeamd

using namespace ropeamd;

ROPE_API int64_t rope_latent_attention_paged_workspace(int64_t num_tokens, int64_t num_heads,
                                                       int64_t latent_dim, int64_t num_sequences) {
  return paged_workspace(num_tokens, num_heads, latent_dim, num_sequences);
}

ROPE_API int rope_latent_attention_paged(const rope_tensor *query, const rope_tensor *latent_cache,
                                         const rope_tensor *page_table,
                                         const rope_tensor *seq_lens,
                                         const rope_tensor *query_offsets, int64_t latent_dim,
                                         double scale, const rope_tensor *out,
                                         const rope_tensor *lse, void *workspace,
                                         int64_t workspace_bytes, void *stream) {
  PagedPlan plan;
  std::string err;
  const int st = plan_paged(query, latent_cache, page_table, seq_lens, query_offsets, latent_dim,
                            scale, out, lse, workspace, workspace_bytes, &plan, &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
  if (plan.noop) return ROPE_OK;
  return plan.dt == ROPE_F16 ? run_paged_width<_Float16>(plan, stream)
                             : run_paged_width<__bf16>(plan, stream);
}
