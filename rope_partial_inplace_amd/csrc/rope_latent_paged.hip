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
// One pass, running maximum and sum in float32.  A workgroup is eight wavefronts, two on each
// SIMD, and 32 or 64 query rows.  Cache rows pass through LDS, 64 at a time in two buffers that
// direct-to-LDS loads fill one step ahead.  S^T = K Q^T is split between the wavefronts by blocks of
// 16 query rows and by cache rows, so that Q stays in registers as the second operand (72 of them
// at latent_dim 512; 32 rows a wavefront would halve the LDS reads of S, but with 144 registers
// for them the loop spills).  O^T = V^T P^T is split by columns of V, so that a wavefront
// accumulates an eighth of the latent for all rows (64 registers) and every byte of the tile is
// read for it once, by transposed LDS reads.  In between P goes through LDS, rounded to the
// storage type: a relative error of at most half a step on each weight, as on the output itself.
// (float16 has no exponents for weights far below the largest: they are taken times 2^11, which the
// division by their sum takes off, and keep half a step down to 2^-25 of the largest.  As they are, many
// small ones beside a large one would be lost; 24 sequences of 100 to 5000 tokens with 1 to 5 queries
// of 16 heads take 21.7 us for it in place of 20.9.)
//
// Measured, bfloat16, latent_dim 512, this kernel and the joining one, caches from HBM: 64 sequences
// of 200 to 9000 tokens, 32 heads, 53 + 8 us (213 MB: 4.0 TB/s in the first, where a dense copy of
// 1 GiB reaches 6.8: each workgroup's first tile and its last part's way out are not covered; back to
// back on one cache, which the Infinity Cache holds in part, 44 + 8), with latent_dim 256 34 + 6, with
// 128 24 + 6; 6 of 60000 to 131072 tokens, 128 heads, 161 - 205 + 13 us (0.55 - 0.69 PF/s: LDS reads
// of the tile, once for S and once for O, and the exponentials between, at 1.9 GHz); one of 1001
// tokens, 16 heads, 11.6 + 4.0 us (dependent reads: lengths, page, tile, part).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>
#include <type_traits>

#include "rope.h"
#include "rope_latent_plan.h"
#include "rope_launch.h"
#include "rope_mfma.h"

namespace ropeamd {
namespace {

constexpr int kPagedBlock = 512;
constexpr int kPagedWaves = kPagedBlock / 64;
constexpr int kPageIds = 512;  // pages whose places LDS holds at a time

__device__ inline uint32_t div_by(const FastDiv &f, uint32_t n) {
  const uint32_t t = __umulhi(f.m, n);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}

// Beginning an item (its page numbers, its queries, a first tile that nothing hides) costs about
// as much as two steps: the shares of the clusters are cut by steps and this.
//
// Every cluster gets an even share however small: shares of at least some steps, for fewer parts
// to join, made the first kernel slower by what the second gained (24 sequences of 100 to 5000
// tokens with 1 to 5 queries of 16 heads: 21.0 + 18.7 us, and 24.7 + 14.6 with half as many parts).
constexpr int32_t kItemCost = 2;
// What a sequence asks for.
struct Sequence {
  int32_t len;     // cached tokens
  int32_t first;   // first query token
  int32_t count;   // query tokens (below 0: the offsets descend here)
  int32_t items;
  int32_t steps;   // of one item
  __device__ int32_t cost() const { return steps + kItemCost; }
};

// Lengths and offsets are device data: values outside their ranges are clamped, so that no
// access leaves the tensors.
__device__ inline Sequence sequence(const PagedPlan &p, int32_t b, int rows, int step) {
  Sequence s;
  const int64_t cap = p.max_pages * p.page_size;
  s.len = int32_t(min(max(p.lens[b * p.len_stride], int64_t(0)), cap));
  if (p.offsets != nullptr) {
    const int64_t o0 = min(max(p.offsets[b * p.off_stride], int64_t(0)), p.T);
    const int64_t o1 = min(max(p.offsets[(b + 1) * p.off_stride], int64_t(0)), p.T);
    s.first = int32_t(o0);
    s.count = int32_t(o1 - o0);
  } else {
    s.first = int32_t(b * p.queries);
    s.count = int32_t(p.queries);
  }
  s.items = (max(s.count, 0) * p.heads + rows - 1) / rows;
  s.steps = max(1, (s.len + step - 1) / step);
  return s;
}

// A wavefront's eighth of a tile of 64 cache rows is 8 of them (tokens tile0 .. tile0 + 63 of the
// sequence, the last one repeated past `len`).  This lane's piece: where in the cache its 16-byte
// chunk of the row's first 128 bytes lies.  places: byte offsets of the sequence's pages from page0 on.
template <typename T>
__device__ __forceinline__ int64_t tile_piece(const PagedPlan &p, const int64_t *places,
                                              int32_t page0, int32_t tile0, int32_t len, int wave,
                                              int lane) {
  const uint32_t tok = uint32_t(min(tile0 + 8 * wave + (lane >> 3), len - 1));
  const uint32_t page = div_by(p.div_page, tok);
  return places[int32_t(page) - page0] +
         int64_t(uint64_t(tok - page * uint32_t(p.page_size)) * uint64_t(p.c_row * sizeof(T)) +
                 ((uint32_t(lane & 7) ^ chunk_key(uint32_t(8 * wave + (lane >> 3)))) << 4));
}

// The pieces' way into LDS, 128 bytes of every row at a time.  A buffer reaches 4 GiB, a cache may
// be larger: rows are fetched by 2 GiB blocks, nearly always all of them in one.
template <int PANELS>
__device__ __forceinline__ void fetch_tile(const char *cache, int64_t piece, int wave,
                                           char *__restrict__ tile) {
  const int32_t block = int32_t(piece >> 31);
  const uint32_t offset = uint32_t(piece) & 0x7fffffffu;
  uint64_t left = __ballot(true);
  while (left != 0) {  // ends: every turn serves the first lane left
    const int32_t first = __builtin_amdgcn_readlane(block, __builtin_ctzll(left));
    // opaque, or the compiler would take the lanes' own `block` for the address in the branch
    int32_t now = first;
    asm volatile("" : "+s"(now));
    left &= ~__ballot(block == first);
    if (block == first) {
      const auto buffer = buffer_at(cache + (int64_t(now) << 31));
#pragma unroll
      for (int n = 0; n < PANELS; ++n)
        load_lds16(buffer, offset, n * 128, tile + n * 8192 + wave * 1024);
    }
  }
}

// How the wavefronts share a tile of 64 cache rows, DB 32-column blocks of the latent and RB
// 32-row blocks of queries.
template <typename T, int DB, int RB>
struct Step {
  static constexpr int PANELS = DB / 2 + 1;
  static constexpr int ROWS = 32 * RB;
  // S: a wavefront multiplies ST strips of 16 cache rows by one block of 16 query rows, WR of them
  // side by side over the query rows, PARTS over the cache rows
  static constexpr int WR = 2 * RB, PARTS = kPagedWaves / WR, ST = 4 / PARTS;
  static constexpr int QF = PANELS * 2;
  // O: COLS column blocks and OB row blocks of a wavefront
  static constexpr bool SPLIT = DB < kPagedWaves;  // fewer column blocks than wavefronts
  static constexpr int COLS = SPLIT ? 1 : DB / kPagedWaves;
  static constexpr int OB = SPLIT ? 1 : RB;
  static_assert(!SPLIT || DB == kPagedWaves / 2, "column blocks");

  __device__ static int part(int wave) { return wave / WR; }
  // Row of the workgroup that this lane owns in its S, and in block i of its O.
  __device__ static int s_row(int wave, int lane) { return wave % WR * 16 + (lane & 15); }
  __device__ static int o_row(int wave, int lane, int i) {
    return (SPLIT ? wave / DB : i) * 32 + (lane & 31);
  }
  __device__ static int column(int wave, int d) { return SPLIT ? wave % DB : wave * COLS + d; }
  // wavefronts without a share of O (one row block, four column blocks)
  __device__ static bool has_output(int wave) { return !SPLIT || wave / DB < RB; }

  // A lane's places in the tiles' panels, from which its other chunks differ by an exclusive or:
  // of its key row, of its transposed values, and of the weights it writes and reads.
  struct Lanes {
    uint32_t keys, values, put, get;
    __device__ Lanes(int wave, int lane)
        : keys(panel_chunk(uint32_t(part(wave) * ST * 16 + (lane & 15)), uint32_t(lane) >> 4)),
          values(panel_transposed(uint32_t(lane), 0, 0)),
          put(panel_chunk(uint32_t(s_row(wave, lane)), (uint32_t(lane) >> 4) & 1u) +
              (uint32_t(lane) >> 5) * 8u),
          get(panel_chunk(uint32_t(o_row(wave, lane, 0)), uint32_t(lane) >> 5)) {}
    // Opaque: what follows from these is worked out again in every step.  Kept from step to step
    // it would take the registers that Q and the accumulators need.
    __device__ void fresh() {
      asm volatile("" : "+v"(keys), "+v"(values), "+v"(put), "+v"(get));
    }
  };

  // Operands out of LDS: panel n of the strips' rows; P of the 16 cache rows of step k; and for
  // product n (step n / COLS, column block n % COLS) the values.  The tile goes in as an argument
  // everywhere, never captured: only so does the compiler see that these reads and the loads
  // into the other buffer do not meet, and does not wait for those loads here.
  __device__ __forceinline__ static void load_keys(const char *tile, const Lanes &at, int n,
                                                   s16x8 (&f)[ST][2]) {
#pragma unroll
    for (int j = 0; j < ST; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        f[j][c] = as_operand(*reinterpret_cast<const uint4 *>(tile + n * 8192 + j * 2048 +
                                                              (at.keys ^ (c * 64u))));
  }
  __device__ __forceinline__ static void load_weights(const char *pt, const Lanes &at, int k,
                                                      s16x8 *f) {
#pragma unroll
    for (int i = 0; i < OB; ++i)
      f[i] = as_operand(*reinterpret_cast<const uint4 *>(pt + i * 4096 + (at.get ^ (k * 32u))));
  }
  __device__ __forceinline__ static s16x8 load_values(const char *tile, const Lanes &at, int wave,
                                                      int n) {
    const int block = column(wave, n % COLS);
    const char *from = tile + (block >> 1) * 8192 + n / COLS * 2048;
    const uint32_t v = at.values ^ (uint32_t(block & 1) * 64u);
    return join(read_transposed(from + v), read_transposed(from + (v ^ kEightRows)));
  }

  // S^T of the wavefront's strips and rows, masked where not every query row sees all of the tile
  // (seen: rows of the tile that this lane's query row may see); returns the row's maximum.
  __device__ __forceinline__ static float scores(const char *__restrict__ tile,
                                                 const Lanes &at, const s16x8 (&qf)[QF], int wave,
                                                 int lane, int32_t seen, bool whole,
                                                 f32x4 (&s)[ST]) {
    constexpr int AHEAD = 2;  // panels read ahead
    s16x8 kf[AHEAD + 1][ST][2];
#pragma unroll
    for (int j = 0; j < ST; ++j) s[j] = f32x4{};
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) load_keys(tile, at, n, kf[n]);
#pragma unroll
    for (int n = 0; n < PANELS; ++n) {
      if (n + AHEAD < PANELS)
        load_keys(tile, at, n + AHEAD, kf[(n + AHEAD) % (AHEAD + 1)]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < ST; ++j)
          s[j] = Mfma<T>::mul16(kf[n % (AHEAD + 1)][j][c], qf[n * 2 + c], s[j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!whole) {
      asm volatile("");  // a branch: most tiles need no masks
#pragma unroll
      for (int j = 0; j < ST; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if ((part(wave) * ST + j) * 16 + 4 * (lane >> 4) + r >= seen) s[j][r] = kNegInf;
    }
    float best = kNegInf;
#pragma unroll
    for (int j = 0; j < ST; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) best = fmaxf(best, s[j][r]);
    return max_quarters(best);
  }

  // The weights of the wavefront's strips at maximum `top`, into the P tile; returns this lane's
  // share of their sum.  P lies in the order the second product takes it: a 16-byte chunk 2 k + h
  // holds the weights of cache rows 16 k + 4 h + {0..3} and of those 8 further on.
  __device__ __forceinline__ static float weights(char *__restrict__ pt, const Lanes &at,
                                                  const f32x4 (&s)[ST], int wave,
                                                  float scale_log2, float top) {
    const float ref = top == kNegInf ? 0.0f : top - Mfma<T>::kLift;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < ST; ++j) {
      float e[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][r], scale_log2, -ref));
        sum += e[r];
      }
      *reinterpret_cast<uint2 *>(pt + (at.put ^ (uint32_t(part(wave) * ST + j) * 32u))) =
          make_uint2(Mfma<T>::pack(e[0], e[1]), Mfma<T>::pack(e[2], e[3]));
    }
    return sum;
  }

  // O^T += V^T P^T over the tile.
  __device__ __forceinline__ static void outputs(const char *__restrict__ tile,
                                                 const char *__restrict__ pt, const Lanes &at,
                                                 int wave, f32x16 (&acc)[OB][COLS]) {
    s16x8 pf[2][OB], vf[2];  // read one product ahead
    load_weights(pt, at, 0, pf[0]);
    vf[0] = load_values(tile, at, wave, 0);
#pragma unroll
    for (int n = 0; n < 4 * COLS; ++n) {
      const int k = n / COLS;
      if (n + 1 < 4 * COLS) vf[(n + 1) % 2] = load_values(tile, at, wave, n + 1);
      if (n % COLS == 0 && k < 3) load_weights(pt, at, k + 1, pf[(k + 1) % 2]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < OB; ++i)
        acc[i][n % COLS] = Mfma<T>::mul(vf[n % 2], pf[k % 2][i], acc[i][n % COLS]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

template <typename T, int DB, int RB>
__global__ __launch_bounds__(kPagedBlock) __attribute__((amdgpu_waves_per_eu(2, 2))) void
latent_paged_kernel(PagedPlan p) {
  using S = Step<T, DB, RB>;
  constexpr int PANELS = S::PANELS, ROWS = S::ROWS, OB = S::OB, COLS = S::COLS;
  constexpr int STEP = int(kPagedStep);
  constexpr int TILE = PANELS * 8192;  // bytes
  // One LDS variable: with several the compiler would mark accesses by variable, and lose what it
  // knows about the two halves of `tiles`.
  struct Lds {
    char tiles[2 * TILE];
    char weights[ROWS * 128];
    int64_t places[kPageIds];
    float row_max[S::PARTS][ROWS];
    int32_t raised;  // some wavefront's row passed its maximum
    int32_t wave_total[kPagedWaves];
    int32_t found[7];
  };
  __shared__ __attribute__((aligned(16))) Lds lds;
  char *tiles = lds.tiles, *weights = lds.weights;
  int64_t *places = lds.places;
  int32_t *found = lds.found;
  auto &row_max = lds.row_max;
  int32_t *wave_total = lds.wave_total;

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the workgroups of a cluster are kXcds apart: on one XCD, they share its L2
  const int32_t turn = int32_t(blockIdx.x / kXcds);
  const int32_t g = (turn / p.cluster) * int32_t(kXcds) + int32_t(blockIdx.x % kXcds);
  const int32_t member = turn % p.cluster;
  const int32_t item_rows = ROWS * p.cluster;

  // ---- the cluster's share [w0, w1) of all items' cost (it fits 31 bits: plan) ----
  Sequence sq = {};
  int32_t mine = 0, n = 0;
  bool descends = false;
  if (tid < p.B) {
    sq = sequence(p, tid, item_rows, STEP);
    n = sq.items * sq.cost();
    descends = sq.count < 0;
  }
  for (int32_t b = tid + kPagedBlock; b < p.B; b += kPagedBlock) {
    const Sequence s = sequence(p, b, item_rows, STEP);
    mine += s.items * s.cost();
    descends |= s.count < 0;
  }
  int32_t incl = wave_scan(n);
  const int32_t rest = p.B > kPagedBlock ? wave_scan(mine) : 0;
  // Offsets that descend could let the sequences' rows add up to more than the plan's 31 bits
  // hold: then there is no work.  (The flag goes with the sums: a barrier that combines one brings
  // an LDS variable of its own, and the steps wait for their loads again.)
  descends = __any(descends);
  if (lane == 63) wave_total[wave] = descends ? -1 : incl + rest;
  __syncthreads();
  int32_t total = 0;
#pragma unroll
  for (int v = 0; v < kPagedWaves; ++v) {
    descends |= wave_total[v] < 0;
    total += wave_total[v];
  }
  auto uniform = [](int32_t x) { return __builtin_amdgcn_readfirstlane(x); };
  total = uniform(total);
  const int32_t per = uniform(int32_t((uint32_t(total) + p.clusters - 1) / uint32_t(p.clusters)));
  const int64_t start = int64_t(g) * per;
  if (descends || start >= total) {
    if (tid < 2 && member == 0) p.joins[(g * 2 + tid) * kJoinWords] = 0;
    return;
  }
  const int32_t w0 = int32_t(start), w1 = int32_t(min(int64_t(total), start + per));
  // the sequence that w0 falls into
  int32_t before = 0;
  for (int32_t b0 = 0; b0 < p.B; b0 += kPagedBlock) {
    if (b0 > 0) {
      n = 0;
      if (b0 + tid < p.B) {
        sq = sequence(p, b0 + tid, item_rows, STEP);
        n = sq.items * sq.cost();
      }
      incl = wave_scan(n);
    }
    if (p.B > kPagedBlock) {  // else wave_total holds the first (only) round's sums already
      __syncthreads();
      if (lane == 63) wave_total[wave] = incl;
      __syncthreads();
    }
    int32_t base = before;
    for (int v = 0; v < kPagedWaves; ++v) {
      if (v < wave) base += wave_total[v];
      before += wave_total[v];
    }
    if (n > 0 && base + incl - n <= w0 && w0 < base + incl) {
      found[0] = b0 + tid;
      found[1] = sq.len;
      found[2] = sq.first;
      found[3] = sq.count;
      found[4] = sq.items;
      found[5] = sq.steps;
      found[6] = base + incl - n;
    }
    if (w0 < before) break;  // the same for all threads
  }
  __syncthreads();
  int32_t b = uniform(found[0]);
  sq = {uniform(found[1]), uniform(found[2]), uniform(found[3]), uniform(found[4]),
        uniform(found[5])};
  const int32_t into = w0 - uniform(found[6]);
  int32_t item = uniform(int32_t(uint32_t(into) / uint32_t(sq.cost())));
  int32_t x0 = into - item * sq.cost();  // where in the item
  int32_t w = w0;
  typename S::Lanes at(wave, lane);
  uint32_t partial = 0;  // bit s: part s of this cluster is one of an item's several

  while (true) {
    const int32_t x1 = min(sq.cost(), x0 + (w1 - w));
    const int32_t st0 = max(0, x0 - kItemCost), st1 = max(0, x1 - kItemCost);  // steps
    const int32_t rows = sq.count * p.heads;
    const int32_t row0 = item * item_rows + member * ROWS;
    if (row0 < rows && st0 < st1) {
      // places of the pages of as many of the steps from `st` on as LDS holds; returns the step that
      // they end before
      int32_t page0 = 0;
      auto load_places = [&](int32_t st) {
        page0 = int32_t(div_by(p.div_page, uint32_t(st * STEP)));
        const int32_t last_tok = min(st1 * STEP, sq.len) - 1;
        const int32_t pages = min(int32_t(kPageIds),
                                  int32_t(div_by(p.div_page, uint32_t(last_tok))) - page0 + 1);
        for (int32_t i = tid; i < pages; i += kPagedBlock) {
          const int64_t id = p.table[b * p.table_seq + (page0 + i) * p.table_page];
          places[i] = min(max(id, int64_t(0)), p.num_pages - 1) * p.c_page * int64_t(sizeof(T));
        }
        return int64_t(page0 + pages) * p.page_size <= last_tok
                   ? int32_t((int64_t(page0 + pages) * p.page_size) / STEP)
                   : st1;
      };
      lds_barrier();  // what the last segment read of places, tiles and row_max
      if (tid == 0) lds.raised = 0;
      int32_t end = st1;
      if (sq.len > 0) end = load_places(st0);

      // ---- this wavefront's query rows, and how much of the cache each may see ----
      s16x8 qf[S::QF];
      const int32_t s_r = row0 + S::s_row(wave, lane);
      const bool live = s_r < rows;
      const int32_t qi = live ? int32_t(div_by(p.div_heads, uint32_t(s_r))) : 0;
      const int32_t limit = live ? sq.len - sq.count + qi + 1 : 0;
      {
        const int32_t head = live ? s_r - qi * p.heads : 0;
        const T *q = static_cast<const T *>(p.q) + int64_t(sq.first + qi) * p.q_tok +
                     int64_t(head) * p.q_head + 8 * (lane >> 4);
#pragma unroll
        for (int k = 0; k < S::QF; ++k)
          qf[k] = live ? as_operand(*reinterpret_cast<const uint4 *>(q + k * 32)) : s16x8{};
        if (p.negative) {  // a negative scale becomes the queries' sign: maxima stay maxima
#pragma unroll
          for (int k = 0; k < S::QF; ++k) qf[k] ^= short(0x8000);
        }
      }
      // fewest cache rows that any row of the workgroup sees
      const int32_t floor = row0 + ROWS > rows
                                ? 0
                                : sq.len - sq.count + int32_t(div_by(p.div_heads, uint32_t(row0))) + 1;

      const char *cache = static_cast<const char *>(p.cache);
      float s_top = kNegInf, s_sum = 0.0f;
      f32x16 acc[OB][COLS];
#pragma unroll
      for (int i = 0; i < OB; ++i)
#pragma unroll
        for (int d = 0; d < COLS; ++d) acc[i][d] = f32x16{};

      // A row's maximum is raised only when a tile passes it by more than kSlack; until then larger
      // weights are carried, which changes no result beyond its rounding.  So the wavefronts that
      // share a row need not agree on a maximum in every tile: each takes the weights at the old
      // one, and all of them see at the barrier before the second product whether any had to pass
      // it, which is rare.  Then the maxima are exchanged, accumulators and sums rescaled and the
      // weights taken again.
      //
      // LDS pointers are arguments, restrict, of what runs between two barriers and of nothing
      // longer: so the compiler does not wait for the loads into the other buffer at each use, and
      // moves no access over a barrier.
      const int s_row = S::s_row(wave, lane), s_part = S::part(wave);
      f32x4 s[S::ST];
      float best = 0.0f, sum = 0.0f;
      // the tile's scores, and weights at the present maxima; returns where the tile after the
      // next one comes from
      auto first_half = [&](const char *__restrict__ cur, char *__restrict__ other,
                            char *__restrict__ pt, int32_t *__restrict__ raised,
                            const int64_t *__restrict__ pages, const char *cache, int64_t piece,
                            int32_t st) {
        if (st + 1 < end) fetch_tile<PANELS>(cache, piece, wave, other);
        const int32_t tile0 = st * STEP;
        at.fresh();
        best = S::scores(cur, at, qf, wave, lane, limit - tile0, tile0 + STEP <= floor, s) *
               p.scale_log2;
        sum = S::weights(pt, at, s, wave, p.scale_log2, s_top);
        if (__any(best > s_top + Mfma<T>::kSlack) && lane == 0) *raised = 1;
        return st + 2 < end
                   ? tile_piece<T>(p, pages, page0, (st + 2) * STEP, sq.len, wave, lane)
                   : 0;
      };
      auto any_raised = [&](const int32_t *__restrict__ raised) { return uniform(*raised) != 0; };
      auto put_row = [&](float *__restrict__ rm, int slot, float x) {
        if (lane < 16) rm[slot * ROWS + s_row] = x;
      };
      // new maxima and weights; returns the factor that what was summed before is rescaled by
      auto raise = [&](const float *__restrict__ rm, char *__restrict__ pt,
                       int32_t *__restrict__ raised) {
        if (tid == 0) *raised = 0;
        float high = rm[s_row];
#pragma unroll
        for (int k = 1; k < S::PARTS; ++k) high = fmaxf(high, rm[k * ROWS + s_row]);
        float f = 1.0f;
        if (high > s_top + Mfma<T>::kSlack) {
          f = __builtin_amdgcn_exp2f(s_top - high);
          s_top = high;
        }
        s_sum *= f;
        sum = S::weights(pt, at, s, wave, p.scale_log2, s_top);
        return f;
      };
      auto rescale = [&](const float *__restrict__ rm) {
#pragma unroll
        for (int i = 0; i < OB; ++i) {
          const float f = rm[S::o_row(wave, lane, i) % ROWS];
#pragma unroll
          for (int d = 0; d < COLS; ++d) acc[i][d] *= f;
        }
      };
      auto second_half = [&](const char *__restrict__ cur, const char *__restrict__ pt) {
        if (S::has_output(wave)) S::outputs(cur, pt, at, wave, acc);
      };
      auto step = [&](const char *cur, char *other, int64_t piece, int32_t st) {
        float *rm = &row_max[0][0];
        const int64_t after = first_half(cur, other, weights, &lds.raised, places, cache, piece, st);
        lds_barrier();
        if (any_raised(&lds.raised)) {
          put_row(rm, s_part, best);
          lds_barrier();
          const float f = raise(rm, weights, &lds.raised);
          lds_barrier();
          if (s_part == 0) put_row(rm, 0, f);
          lds_barrier();
          rescale(rm);
        }
        s_sum += sum;
        second_half(cur, weights);
        return after;
      };

      if (sq.len > 0) {
        int32_t st = st0;
        while (true) {
          // ---- the steps: the next tile is on its way while one is multiplied ----
          lds_barrier();
          fetch_tile<PANELS>(cache, tile_piece<T>(p, places, page0, st * STEP, sq.len, wave, lane),
                             wave, tiles);
          int64_t next = st + 1 < end ? tile_piece<T>(p, places, page0, (st + 1) * STEP, sq.len,
                                                      wave, lane)
                                      : 0;
          for (int32_t i = 0; st < end; ++st, ++i) {
            wait_loads_all();
            lds_barrier();
            next = step(tiles + (i & 1) * TILE, tiles + (~i & 1) * TILE, next, st);
          }
          if (st >= st1) break;
          lds_barrier();
          end = load_places(st);
        }
      }

      // ---- maxima, and sums of the wavefronts that shared a row, to those that hold outputs ----
      s_sum = sum_quarters(s_sum);
      float o_top[OB];
      lds_barrier();
      if (s_part == 0) put_row(&row_max[0][0], 0, s_top);
      lds_barrier();
#pragma unroll
      for (int i = 0; i < OB; ++i) o_top[i] = row_max[0][S::o_row(wave, lane, i) % ROWS];
      lds_barrier();
      put_row(&row_max[0][0], s_part, s_sum);
      lds_barrier();

      // ---- the segment's result: a whole item's output, or a part for the joining kernel ----
      const bool whole = st0 == 0 && st1 == sq.steps;
      const int64_t slot = (int64_t(g) * p.cluster + member) * 2 + (w == w0 ? 0 : 1);
      if (S::has_output(wave)) {
#pragma unroll
        for (int i = 0; i < OB; ++i) {
          const int m = S::o_row(wave, lane, i);
          float sum = row_max[0][m];
#pragma unroll
          for (int k = 1; k < S::PARTS; ++k) sum += row_max[k][m];
          const int32_t r = row0 + m;
          const int64_t out_row = int64_t(sq.first) * p.heads + r;
          const bool some = sum > 0.0f || sum != sum;  // a row that sees nothing gets zeros
          const bool first_column = S::column(wave, 0) == 0;
          if (whole) {
            if (r < rows) {
              const float inv = some ? 1.0f / sum : 0.0f;
              char *out = static_cast<char *>(p.out) + out_row * p.latent * int64_t(sizeof(T));
#pragma unroll
              for (int d = 0; d < COLS; ++d)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const f32x16 &a = acc[i][d];
                  const int d4 = S::column(wave, d) * 8 + c * 2 + (lane >> 5);
                  *reinterpret_cast<uint2 *>(out + d4 * 8) =
                      make_uint2(Mfma<T>::pack(a[4 * c] * inv, a[4 * c + 1] * inv),
                                 Mfma<T>::pack(a[4 * c + 2] * inv, a[4 * c + 3] * inv));
                }
              if (first_column && lane < 32 && p.lse != nullptr)
                p.lse[out_row] = some ? natural<T>(o_top[i], sum) : kNegInf;
            }
          } else if (r < rows) {
            float *part = p.parts + slot * ROWS * p.latent + m * 4;
#pragma unroll
            for (int d = 0; d < COLS; ++d)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const f32x16 &a = acc[i][d];
                const int d4 = S::column(wave, d) * 8 + c * 2 + (lane >> 5);
                const f32x4 v = {a[4 * c], a[4 * c + 1], a[4 * c + 2], a[4 * c + 3]};
                *reinterpret_cast<f32x4 *>(part + d4 * (ROWS * 4)) = v;
              }
            if (first_column && lane < 32)
              *reinterpret_cast<float2 *>(p.stats + (slot * ROWS + m) * 2) =
                  make_float2(o_top[i], sum);
          }
        }
      }
    }
    if (st0 < st1 && (st0 != 0 || st1 != sq.steps)) {
      const int part = w == w0 ? 0 : 1;
      partial |= 1u << part;
      if (tid == 0 && member == 0) {
        const uint32_t begin = uint32_t(w - x0), u_per = uint32_t(per);
        const uint32_t first_g = (begin + kItemCost) / u_per;
        int32_t *rec = p.joins + (g * 2 + part) * kJoinWords;
        rec[0] = int32_t((begin + uint32_t(sq.cost()) - 1) / u_per - first_g + 1);
        rec[1] = int32_t(first_g);
        rec[2] = begin <= first_g * u_per ? 0 : 1;
        rec[3] = sq.first * p.heads + item * item_rows;
        rec[4] = rows - item * item_rows;
      }
    }
    w += x1 - x0;
    if (w >= w1) break;
    x0 = 0;
    if (++item >= sq.items) {
      item = 0;
      do {  // ends: w < w1 <= total, so a later sequence has items
        ++b;
        sq = sequence(p, b, item_rows, STEP);
      } while (sq.items == 0);
    }
  }
  if (tid < 2 && member == 0 && (partial >> tid & 1u) == 0)
    p.joins[(g * 2 + tid) * kJoinWords] = 0;
}

// Joins the parts of items that several clusters had a share of: a part k holds unnormalised
// outputs o_k at maximum m_k with weight sum l_k, and
//   out = sum_k 2^(m_k - m) o_k / sum_k 2^(m_k - m) l_k,   m = max_k m_k.
// One workgroup for each part joins the n-th part of the item's (4-column group, row) cells, so
// that all workgroups have about one part's bytes to read.  It is a launch of a few dependent
// reads: `share` wavefronts take the parts of a cell in turn, as many as the workgroup has to
// spare, four parts' reads under way at once (eight: 9.6 us in place of 8.0 for a decoding step of
// 64 sequences), and add up through LDS in a fixed order.
constexpr int kJoinBlock = 1024;
constexpr int kJoinAhead = 4;

template <typename T, int DB, int RB>
__global__ __launch_bounds__(kJoinBlock) void latent_paged_join_kernel(PagedPlan p) {
  constexpr int ROWS = 32 * RB;
  constexpr int CELLS = DB * 8 * ROWS;
  constexpr int WAVES = kJoinBlock / 64;
  __shared__ float4 add[WAVES][64];
  __shared__ float2 add_stat[WAVES][64];
  const int32_t member = int32_t(blockIdx.y);
  const int32_t g = int32_t(blockIdx.x) >> 1;
  const int32_t *rec = p.joins + int32_t(blockIdx.x) * kJoinWords;
  const int32_t n = rec[0], g0 = rec[1], first = rec[2];
  if (n <= 1) return;
  const int32_t live = rec[4] - member * ROWS;  // rows of the item from this member's on
  const int lane = int(threadIdx.x) & 63, wave = int(threadIdx.x) >> 6;
  const int c0 = int(int64_t(CELLS) * (g - g0) / n), c1 = int(int64_t(CELLS) * (g - g0 + 1) / n);
  const int groups = (c1 - c0 + 63) / 64;  // of 64 cells
  int share = 1;
  while (share < WAVES && 2 * share * groups <= WAVES) share *= 2;
  const int side = WAVES / share;  // groups at a time
  for (int at = 0; at < groups; at += side) {
    const int cell = c0 + (at + wave / share) * 64 + lane;
    const int m = cell % ROWS;
    const bool mine = cell < c1 && m < live;
    float top = kNegInf, l = 0.0f;
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // what is held so far and `N` parts more, all at the highest maximum among them
    auto take = [&](auto count, const float2 *stat, const float4 *o) {
      constexpr int N = decltype(count)::value;
      float next = top;
#pragma unroll
      for (int u = 0; u < N; ++u) next = fmaxf(next, stat[u].x);
      const float ref = next == kNegInf ? 0.0f : next;
      const float f = __builtin_amdgcn_exp2f(top - ref);
      top = next;
      l *= f;
      t = make_float4(t.x * f, t.y * f, t.z * f, t.w * f);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const float w = __builtin_amdgcn_exp2f(stat[u].x - ref);
        l += stat[u].y * w;
        t.x += o[u].x * w;
        t.y += o[u].y * w;
        t.z += o[u].z * w;
        t.w += o[u].w * w;
      }
    };
    if (mine) {
      for (int32_t k0 = wave % share; k0 < n; k0 += kJoinAhead * share) {
        float2 stat[kJoinAhead];
        float4 o[kJoinAhead];
#pragma unroll
        for (int u = 0; u < kJoinAhead; ++u) {
          const int32_t k = k0 + u * share;
          stat[u] = make_float2(kNegInf, 0.0f);
          o[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (k < n) {
            const int64_t slot = (int64_t(g0 + k) * p.cluster + member) * 2 + (k == 0 ? first : 0);
            stat[u] = *reinterpret_cast<const float2 *>(p.stats + (slot * ROWS + m) * 2);
            o[u] = *reinterpret_cast<const float4 *>(p.parts + slot * ROWS * p.latent +
                                                     int64_t(cell) * 4);
          }
        }
        take(std::integral_constant<int, kJoinAhead>(), stat, o);
      }
    }
    if (share > 1) {
      add[wave][lane] = t;
      add_stat[wave][lane] = make_float2(top, l);
      __syncthreads();
      if (wave % share == 0)
        for (int k = 1; k < share; ++k)
          take(std::integral_constant<int, 1>(), &add_stat[wave + k][lane], &add[wave + k][lane]);
      __syncthreads();
    }
    if (mine && wave % share == 0) {
      const bool some = l > 0.0f || l != l;
      const float inv = some ? 1.0f / l : 0.0f;
      const int64_t row = int64_t(rec[3]) + member * ROWS + m;
      *reinterpret_cast<uint2 *>(static_cast<char *>(p.out) +
                                 row * p.latent * int64_t(sizeof(T)) + (cell / ROWS) * 8) =
          make_uint2(Mfma<T>::pack(t.x * inv, t.y * inv), Mfma<T>::pack(t.z * inv, t.w * inv));
      if (cell < ROWS && p.lse != nullptr)
        p.lse[row] = some ? natural<T>(top, l) : kNegInf;
    }
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
  return launch_kernel(join, dim3(uint32_t(p.clusters) * 2, uint32_t(p.cluster)), kJoinBlock, 0,
                       stream, &p);
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
