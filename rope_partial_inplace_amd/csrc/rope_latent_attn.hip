// rope_latent_attn.hip -- latent attention, expanded form, forward and gradients (gfx950).
//
// Head h of query token i attends to its sequence's tokens j, whose keys are an expanded part of
// its own and a rotated part shared by all heads:
//   s_ij = scale (<qn_ih, k_jh> + <qr_ih, r_j>),  p = softmax_j(s),  o_ih = sum_j p_ij v_jh
// causal: the last query sees every key and each earlier one a key less.  With g the gradient of
// o and D_ih = sum_j p_ij <g_ih, v_jh>:
//   dv_jh = sum_i p_ij g_ih,   ds_ij = p_ij (<g_ih, v_jh> - D_ih)
//   dq_ih = scale sum_j ds_ij [k_jh | r_j],  dk_jh = scale sum_i ds_ij qn_ih,
//   dr_j  = scale sum_h sum_i ds_ij qr_ih
//
// All of it is matrix products (2 (2 dim + 64) operations a visible pair forward, 2.5 times that
// backward with the probabilities computed again), bound by MFMA, by the LDS reads that feed it
// and by the exponentials between the products.  The shared key part is read as it is, never
// repeated for each head in memory.
//
// Forward, and dq: a workgroup is four wavefronts of 32 query rows of one head; 64 keys and
// values at a time pass through LDS in two buffers.  dk and dv: four pairs of wavefronts for 32
// keys each, over 64 query rows at a time.  dq and dk/dv are two kernels that both compute p again,
// the first of them twice (D needs all of a row before its first ds): nine products where atomics on
// dq would need seven, for sums in a fixed order.
//
// Probabilities and ds are rounded to the storage type between the products, as P is in the absorbed
// form: a relative error of at most half a step on each.  float16 ends at 65504 and has 14 exponents
// below 1, while ds is as small as the incoming gradient over the row's length and may be larger
// than any result: both are lifted or lowered by powers of two: constant ones for p, forward too, and for ds taken
// for each row of dq and each key of dk from what is summed there.
//
// Measured, bfloat16, causal, 32 heads of 128: 7 prompts of 300 to 6000 tokens forward 880 - 1080
// us, 0.74 - 0.91 PF/s (a large library product on this card: 1.2 - 1.35), with heads of 64 610 - 750
// us; 4 x 2048 tokens, forward 206 - 256 us, D and dq 453 - 570, dk and dv 462 - 597, dr 12.5, on
// average 0.79 PF/s of all eleven products (not causal, forward alone, 359 - 429 us).
// The range is the clock's, which falls to 1.7 - 2.1 GHz under such kernels.  What the products
// wait for: LDS reads, and the exponentials of a tile, which only the SIMD's other wavefront covers.
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

constexpr int kBlockThreads = kExpandedThreads;
constexpr int kRows = int(kExpandedRows);
constexpr int kTile = 64;  // keys (or query rows) in LDS at a time
constexpr float kLog2eF = 1.44269504f;

struct Span {
  int32_t first, count;
};

// Tokens of sequence b; offsets are device data, so values out of range are clamped.
__device__ inline Span span(const int64_t *off, int64_t stride, int64_t total, int64_t each,
                            int32_t b) {
  if (off == nullptr) return {int32_t(b * each), int32_t(each)};
  const int64_t o0 = min(max(off[b * stride], int64_t(0)), total);
  const int64_t o1 = min(max(off[(b + 1) * stride], o0), total);
  return {int32_t(o0), int32_t(o1 - o0)};
}

// A tile of a sequence's query (or key) tokens; sequence -1: there are fewer tiles.
struct TileAt {
  int32_t seq, tile;
};

__device__ inline int32_t wave_sum(int32_t x) {
  return __builtin_amdgcn_readlane(wave_scan(x), 63);
}

// The t-th tile of all sequences, longest first: a causal query tile j sees about j tiles of keys,
// a key tile as many tiles of queries as its sequence has behind it.  A head's tiles begin
// together on the compute units of one XCD, and one that began late would hold up the end.  (In the
// order of the sequences, each one's longest first, compute units idled 21% of a training step of
// 4 x 2048 tokens, and it took 1100 us in place of 1035; 7 prompts of 300 to 6000 tokens took 1004
// in place of 1013.)
//
// Up to 64 sequences, one a lane: with n_b tiles in sequence b, sum_b max(0, n_b - j) of them have
// an index (counted from the short end) of at least j, so a bisection over j finds the t-th.
//
// With more they come in their own order, and nothing is added up over them: a call has
// total / 128 + B tile numbers, and from off_b / 128 + b on there are enough for sequence b's tiles
// (some stay empty).  A search finds b, each of its steps a read of 64 offsets.  Adding up would cost
// each of more than B workgroups a time that grows with B: forward and gradients of 4096 sequences
// of 16 tokens and 16 heads 4.75 ms in place of 3.05, of 65536 of one token and 2 heads 90 in place
// of 5.2; 65 of 640 and 100 of 500 tokens 1.03 and 1.38 in place of 1.06 and 1.25.  Every 64 numbers
// are taken in bit-reversed order, or the empty ones, often every second, would leave every second
// compute unit idle (65 sequences of 128 tokens: 226 us in place of 175).
template <bool QUERY>
__device__ inline TileAt find_tile(const ExpandedPlan &p, int32_t t) {
  const int64_t *off = QUERY ? p.q_off : p.k_off;
  const int64_t each = QUERY ? p.q_each : p.k_each;
  const int32_t bound = int32_t(QUERY ? p.q_tiles : p.k_tiles);
  if (off == nullptr) {
    const int32_t per = int32_t((each + kRows - 1) / kRows), count = int32_t(p.B);
    if (t >= per * count) return {-1, 0};
    return {t % count, QUERY ? per - 1 - t / count : t / count};
  }
  const int64_t stride = QUERY ? p.q_off_stride : p.k_off_stride, total = QUERY ? p.Tq : p.Tk;
  const int lane = int(threadIdx.x) & 63;
  if (p.B <= 64) {
    const int32_t n = lane < p.B ? (span(off, stride, total, 0, lane).count + kRows - 1) / kRows : 0;
    if (t >= wave_sum(n)) return {-1, 0};
    int32_t j = 0, above = bound;  // more than t tiles from j on, and none from `above` on
    while (above - j > 1) {
      const int32_t mid = (j + above) / 2;
      if (wave_sum(max(0, n - mid)) > t)
        j = mid;
      else
        above = mid;
    }
    const int32_t rank = t - wave_sum(max(0, n - j - 1));
    const uint64_t with = __ballot(n > j);
    const int32_t place = __builtin_amdgcn_mbcnt_hi(uint32_t(with >> 32),
                                                    __builtin_amdgcn_mbcnt_lo(uint32_t(with), 0));
    const int32_t seq = __builtin_ctzll(__ballot(n > j && place == rank));
    return {seq, QUERY ? j : __builtin_amdgcn_readlane(n, seq) - 1 - j};
  }
  if (QUERY) t = bound - 1 - t;  // the last tiles first, at least
  if ((t | 63) < bound) t = (t & ~63) | int32_t(__brev(uint32_t(t)) >> 26);
  // the last sequence that begins at t or before is among the `left` from seq on
  for (int32_t seq = 0, left = int32_t(p.B);;) {  // ends: at most a 64th is left, rounded up
    const int32_t step = (left + 63) / 64, at = lane * step;
    const int64_t o = min(max(off[min(seq + at, int32_t(p.B)) * stride], int64_t(0)), total);
    const int32_t begin = int32_t(o / kRows) + seq + at;
    const uint64_t behind = __ballot(at >= left || begin > t);
    const int32_t n = behind == 0 ? 64 : __builtin_ctzll(behind);
    if (n == 0) return {-1, 0};
    if (step == 1) {
      seq += n - 1;
      const int32_t tile = t - __builtin_amdgcn_readlane(begin, n - 1);
      const Span s = span(off, stride, total, 0, seq);
      return {tile * int64_t(kRows) < s.count ? seq : -1, tile};
    }
    seq += (n - 1) * step;
    left = min(step, left - (n - 1) * step);
  }
}

// Workgroup number -> (head, tile number): the workgroups of a head, which share its keys and
// values, follow each other on one XCD.
__device__ inline bool head_and_tile(const ExpandedPlan &p, int64_t tiles, int32_t &head,
                                     int32_t &tile) {
  const int64_t total = int64_t(p.heads) * tiles;
  const int64_t per = (total + kXcds - 1) / kXcds;
  const int64_t at = int64_t(blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
  if (blockIdx.x / kXcds >= per || at >= total) return false;
  head = int32_t(at / tiles);
  tile = int32_t(at % tiles);
  return true;
}

// Rows [row0, row0 + 64) of a strided matrix into LDS panels 0 .. PANELS - 1 (8 KB each), this
// wavefront's share (of WAVES); rows past `last` repeat it.  stride in bytes, below 2^25 (plan): the
// rows of a tile lie within 2^31 bytes.
template <int PANELS, int WAVES = 4>
__device__ __forceinline__ void fetch_rows(const char *base, int64_t stride, int32_t row0,
                                           int32_t last, int wave, int lane,
                                           char *__restrict__ lds) {
  const auto buffer = buffer_at(base + int64_t(row0) * stride);
#pragma unroll
  for (int i = 0; i < 8 / WAVES; ++i) {
    const int rb = wave * (8 / WAVES) + i;
    const uint32_t row = uint32_t(min(8 * rb + (lane >> 3), last - row0));
    const uint32_t at = row * uint32_t(stride) +
                        ((uint32_t(lane & 7) ^ chunk_key(uint32_t(8 * rb + (lane >> 3)))) << 4);
#pragma unroll
    for (int n = 0; n < PANELS; ++n) load_lds16(buffer, at, n * 128, lds + n * 8192 + rb * 1024);
  }
}

// The compiler would read every operand just before its product; the barriers keep the reads of
// the next operands ahead of the products of these.
__device__ __forceinline__ void hold_order() { __builtin_amdgcn_sched_barrier(0); }

// Row operands of panel n: 32 rows from row0, k values 16 c .. + 15.
__device__ __forceinline__ void load_panel(const char *lds, int row0, int n, int lane,
                                           s16x8 (&f)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    f[c] = as_operand(*reinterpret_cast<const uint4 *>(
        lds + n * 8192 + panel_chunk(uint32_t(row0 + (lane & 31)), 2u * c + (uint32_t(lane) >> 5))));
}

// Transposed operand of 32 columns d of the 16 rows from row0.
__device__ __forceinline__ s16x8 load_column(const char *lds, int row0, int d, int lane) {
  return transposed_operand(lds + (d / 2) * 8192 + row0 * 128, uint32_t(lane), uint32_t(d & 1));
}

// acc[d] += (column blocks d of 32 LDS rows from row0) times the 32 x 32 operand whose two steps
// of 16 are b0, b1.
template <typename T, int BLOCKS>
__device__ __forceinline__ void column_product(const char *lds, int row0, int lane, s16x8 b0,
                                               s16x8 b1, f32x16 *acc) {
  s16x8 f[2][2];
  f[0][0] = load_column(lds, row0, 0, lane);
  f[0][1] = load_column(lds, row0 + 16, 0, lane);
#pragma unroll
  for (int d = 0; d < BLOCKS; ++d) {
    if (d + 1 < BLOCKS) {
      f[(d + 1) % 2][0] = load_column(lds, row0, d + 1, lane);
      f[(d + 1) % 2][1] = load_column(lds, row0 + 16, d + 1, lane);
    }
    hold_order();
    acc[d] = Mfma<T>::mul(f[d % 2][0], b0, acc[d]);
    acc[d] = Mfma<T>::mul(f[d % 2][1], b1, acc[d]);
    hold_order();
  }
}

// C += 32 rows of LDS panels (from row0) times register operands, AHEAD of them read ahead.
template <typename T, int PANELS, int AHEAD = 4>
__device__ __forceinline__ f32x16 row_product(const char *lds, int row0, int lane, const s16x8 *b,
                                              f32x16 c) {
  constexpr int STEPS = PANELS * 4 / AHEAD;
  s16x8 f[2][AHEAD];
  auto load = [](const char *lds, int row0, int lane, int n, s16x8 *to) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      to[k] = as_operand(*reinterpret_cast<const uint4 *>(
          lds + (n * AHEAD + k) / 4 * 8192 +
          panel_chunk(uint32_t(row0 + (lane & 31)),
                      2u * ((n * AHEAD + k) % 4) + (uint32_t(lane) >> 5))));
  };
  load(lds, row0, lane, 0, f[0]);
#pragma unroll
  for (int n = 0; n < STEPS; ++n) {
    if (n + 1 < STEPS) load(lds, row0, lane, n + 1, f[(n + 1) % 2]);
    hold_order();
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) c = Mfma<T>::mul(f[n % 2][k], b[n * AHEAD + k], c);
    hold_order();
  }
  return c;
}

// x[i] += 32 LDS rows of panels 0 .. PANELS - 1 (from row 32 i) times register operands, for both
// halves of a tile at once, a panel's operands read ahead.
template <typename T, int PANELS>
__device__ __forceinline__ void panel_products(const char *lds, int lane, const s16x8 *b,
                                               f32x16 (&x)[2]) {
  s16x8 f[2][2][4];
  load_panel(lds, 0, 0, lane, f[0][0]);
  load_panel(lds, 32, 0, lane, f[0][1]);
#pragma unroll
  for (int n = 0; n < PANELS; ++n) {
    if (n + 1 < PANELS) {
      load_panel(lds, 0, n + 1, lane, f[(n + 1) % 2][0]);
      load_panel(lds, 32, n + 1, lane, f[(n + 1) % 2][1]);
    }
    hold_order();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) x[i] = Mfma<T>::mul(f[n % 2][i][k], b[n * 4 + k], x[i]);
    hold_order();
  }
}

// 16-byte pieces of a row as register operands: 8 (lane / 32) elements into every 16.
template <int STEPS>
__device__ __forceinline__ void load_operands(const char *row, bool live, int lane, s16x8 *f) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
    f[k] = live ? as_operand(*reinterpret_cast<const uint4 *>(row + k * 32 + 16 * (lane >> 5)))
                : s16x8{};
}

// Row of this lane's column, four consecutive elements at a time: scaled, rounded, stored.
template <typename T, int BLOCKS>
__device__ __forceinline__ void store_columns(char *row, const f32x16 *acc, float f, int lane) {
#pragma unroll
  for (int d = 0; d < BLOCKS; ++d)
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint2 *>(row + (d * 8 + c * 2 + (lane >> 5)) * 8) =
          make_uint2(Mfma<T>::pack(acc[d][4 * c] * f, acc[d][4 * c + 1] * f),
                     Mfma<T>::pack(acc[d][4 * c + 2] * f, acc[d][4 * c + 3] * f));
}

// ---- forward ------------------------------------------------------------------------------

template <typename T, int DIM>
__global__ __launch_bounds__(kBlockThreads, 2) void latent_forward_kernel(ExpandedPlan p) {
  constexpr int NP = DIM / 64;             // panels of a key's own part, and of a value
  constexpr int TILE = (2 * NP + 1) * 8192;  // keys, shared key part, values
  __shared__ __attribute__((aligned(16))) char tiles[2 * TILE];
  int32_t head, tile;
  if (!head_and_tile(p, p.q_tiles, head, tile)) return;
  const TileAt at = find_tile<true>(p, tile);
  if (at.seq < 0) return;
  const Span q = span(p.q_off, p.q_off_stride, p.Tq, p.q_each, at.seq);
  const Span k = span(p.k_off, p.k_off_stride, p.Tk, p.k_each, at.seq);

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t row = at.tile * kRows + wave * 32 + (lane & 31);
  const bool live = row < q.count;
  s16x8 qf[NP * 4 + 4];
  load_operands<NP * 4 + 4>(static_cast<const char *>(p.q) +
                                (int64_t(q.first + row) * p.q_tok + head * p.q_head) *
                                    int64_t(sizeof(T)),
                            live, lane, qf);
  if (p.negative) {  // a negative scale becomes the queries' sign, so that maxima stay maxima
#pragma unroll
    for (int i = 0; i < NP * 4 + 4; ++i) qf[i] ^= short(0x8000);
  }
  // keys a row sees, the fewest and the most of the workgroup's rows
  const int32_t shift = k.count - q.count + 1;
  const int32_t limit = !live ? 0 : p.causal ? row + shift : k.count;
  const int32_t least = p.causal ? at.tile * kRows + shift : k.count;
  const int32_t most =
      p.causal ? min(min(at.tile * kRows + kRows, q.count) - 1 + shift, k.count) : k.count;

  const int64_t es = sizeof(T);
  const char *kb = static_cast<const char *>(p.k) + (int64_t(k.first) * p.k_tok + head * p.k_head) * es;
  const char *rb = static_cast<const char *>(p.kr) + int64_t(k.first) * p.kr_tok * es;
  const char *vb = static_cast<const char *>(p.v) + (int64_t(k.first) * p.v_tok + head * p.v_head) * es;
  auto fetch = [&](int32_t j0, char *__restrict__ to) {
    fetch_rows<NP>(kb, p.k_tok * es, j0, k.count - 1, wave, lane, to);
    fetch_rows<1>(rb, p.kr_tok * es, j0, k.count - 1, wave, lane, to + NP * 8192);
    fetch_rows<NP>(vb, p.v_tok * es, j0, k.count - 1, wave, lane, to + (NP + 1) * 8192);
  };

  float top = kNegInf, sum = 0.0f;
  f32x16 acc[NP * 2];
#pragma unroll
  for (int d = 0; d < NP * 2; ++d) acc[d] = f32x16{};

  auto step = [&](const char *__restrict__ cur, char *__restrict__ other, int32_t j0) {
    if (j0 + kTile < most) fetch(j0 + kTile, other);
    // S^T of the tile's two halves
    f32x16 s[2] = {};
    panel_products<T, NP + 1>(cur, lane, qf, s);
    if (j0 + kTile > min(least, k.count)) {  // some row does not see all of it
      asm volatile("");  // a branch: most tiles need no masks
#pragma unroll
      for (int r = 0; r < 32; ++r)
        if (j0 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4 >= limit) s[r / 16][r % 16] = kNegInf;
    }
    float best = kNegInf;
#pragma unroll
    for (int r = 0; r < 32; ++r) best = fmaxf(best, s[r / 16][r % 16]);
    best = max_halves(best) * p.scale_log2;  // the scale is not negative: see the operands
    // rescale only when the maximum rises by more than kSlack: until then larger weights are carried
    if (__any(best > top + Mfma<T>::kSlack)) {
      float f = 1.0f;
      if (best > top + Mfma<T>::kSlack) {
        f = __builtin_amdgcn_exp2f(top - best);
        top = best;
      }
      sum *= f;
#pragma unroll
      for (int d = 0; d < NP * 2; ++d) acc[d] *= f;
    }
    const float ref = top == kNegInf ? 0.0f : top - Mfma<T>::kLift;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float e[16], part = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][r], p.scale_log2, -ref));
        part += e[r];
      }
      sum += part;
      column_product<T, NP * 2>(cur + (NP + 1) * 8192, i * 32, lane, round8<T>(e),
                                round8<T>(e + 8), acc);
    }
  };

  if (most > 0) fetch(0, tiles);
  for (int32_t n = 0; n * kTile < most; ++n) {
    wait_loads_all();
    lds_barrier();
    step(tiles + (n & 1) * TILE, tiles + (~n & 1) * TILE, n * kTile);
  }
  sum = sum_halves(sum);
  if (!live) return;
  const bool some = sum > 0.0f || sum != sum;  // a row that sees nothing gets zeros
  const int64_t out_row = int64_t(q.first + row) * p.heads + head;
  store_columns<T, NP * 2>(static_cast<char *>(p.out) + out_row * DIM * es, acc,
                           some ? 1.0f / sum : 0.0f, lane);
  if (lane < 32) p.lse[out_row] = some ? natural<T>(top, sum) : kNegInf;
}

// ---- backward: D and dq -------------------------------------------------------------------

// D = sum_j p_j dP_j takes a pass of its own over the keys.  <g, o> would be the same sum, but for
// the rounding of o: its error dD goes into dq as scale dD sum_j p_j [k_j | r_j], which keys with a
// common offset do not average out (2048 keys, keys and values with offsets of one deviation in
// every channel, bfloat16: dq off by 5.2% of its norm in place of 0.29%; of three, 45% and 0.58%).
// Its two products run at 1.0 PF/s: 4 x 2048 tokens of 32 heads take this
// kernel 465 - 515 us in place of 310 - 337, five texts of 17 to 333 tokens 21 in place of 16.
template <typename T, int DIM>
__global__ __launch_bounds__(kBlockThreads, 2) void latent_dquery_kernel(ExpandedPlan p) {
  constexpr int NP = DIM / 64;
  constexpr int TILE = (2 * NP + 1) * 8192;
  __shared__ __attribute__((aligned(16))) char tiles[2 * TILE];
  int32_t head, tile;
  if (!head_and_tile(p, p.q_tiles, head, tile)) return;
  const TileAt at = find_tile<true>(p, tile);
  if (at.seq < 0) return;
  const Span q = span(p.q_off, p.q_off_stride, p.Tq, p.q_each, at.seq);
  const Span k = span(p.k_off, p.k_off_stride, p.Tk, p.k_each, at.seq);

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t es = sizeof(T);
  const int32_t row = at.tile * kRows + wave * 32 + (lane & 31);
  const bool live = row < q.count;
  const int64_t tok = q.first + row, out_row = tok * p.heads + head;
  s16x8 qf[NP * 4 + 4], gf[NP * 4];
  load_operands<NP * 4 + 4>(
      static_cast<const char *>(p.q) + (tok * p.q_tok + head * p.q_head) * es, live, lane, qf);
  load_operands<NP * 4>(
      static_cast<const char *>(p.grad) + (tok * p.g_tok + head * p.g_head) * es, live, lane, gf);
  float lse2 = __builtin_huge_valf();  // rows that see nothing, or do not exist: p = 0
  if (live) {
    const float l = p.lse[out_row];
    if (l != kNegInf) lse2 = l * kLog2eF;
  }
  const int32_t shift = k.count - q.count + 1;
  const int32_t limit = !live ? 0 : p.causal ? row + shift : k.count;
  const int32_t least = p.causal ? at.tile * kRows + shift : k.count;
  const int32_t most =
      p.causal ? min(min(at.tile * kRows + kRows, q.count) - 1 + shift, k.count) : k.count;

  const char *kb = static_cast<const char *>(p.k) + (int64_t(k.first) * p.k_tok + head * p.k_head) * es;
  const char *rb = static_cast<const char *>(p.kr) + int64_t(k.first) * p.kr_tok * es;
  const char *vb = static_cast<const char *>(p.v) + (int64_t(k.first) * p.v_tok + head * p.v_head) * es;
  auto fetch = [&](int32_t j0, char *__restrict__ to) {
    fetch_rows<NP>(kb, p.k_tok * es, j0, k.count - 1, wave, lane, to);
    fetch_rows<1>(rb, p.kr_tok * es, j0, k.count - 1, wave, lane, to + NP * 8192);
    fetch_rows<NP>(vb, p.v_tok * es, j0, k.count - 1, wave, lane, to + (NP + 1) * 8192);
  };
  const float scale2 = p.negative ? -p.scale_log2 : p.scale_log2;
  // p_j of score s of key j; whole: every row sees all of the tile
  auto weight = [&](float s, bool whole, int32_t j) {
    const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s, scale2, -lse2));
    return whole || j < limit ? w : 0.0f;
  };

  const int32_t count = most > 0 ? (most + kTile - 1) / kTile : 0;  // tiles
  const bool few = count <= 2;  // they stay in LDS for the second pass
  float delta = 0.0f, most_w = 0.0f, most_x = 0.0f;
  auto sum_step = [&](const char *__restrict__ cur, char *__restrict__ other, int32_t j0) {
    if (j0 + kTile < most)
      fetch(j0 + kTile, other);
    else if (!few)
      fetch(0, other);
    f32x16 s[2] = {}, dp[2] = {};
    panel_products<T, NP + 1>(cur, lane, qf, s);
    panel_products<T, NP>(cur + (NP + 1) * 8192, lane, gf, dp);
    const bool whole = j0 + kTile <= min(least, k.count);
    float part = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const float w = weight(s[r / 16][r % 16], whole, j0 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4);
      const float x = w * dp[r / 16][r % 16];
      part += x;
      if constexpr (Mfma<T>::kNarrow) {
        most_w = fmaxf(most_w, w);
        most_x = fmaxf(most_x, __builtin_fabsf(x));
      }
    }
    delta += part;
  };
  f32x16 acc[NP * 2 + 2];
  auto step = [&](const char *__restrict__ cur, char *__restrict__ other, int32_t j0) {
    if (!few && j0 + kTile < most) fetch(j0 + kTile, other);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x16 s = row_product<T, NP + 1, 2>(cur, i * 32, lane, qf, f32x16{});
      const f32x16 dp =
          row_product<T, NP, 2>(cur + (NP + 1) * 8192, i * 32, lane, gf, f32x16{});
      const bool whole = j0 + kTile <= min(least, k.count);
      float e[16];
#pragma unroll
      for (int r = 0; r < 16; ++r)
        e[r] = weight(s[r], whole, j0 + i * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4) *
               (dp[r] - delta);
      column_product<T, NP * 2 + 2>(cur, i * 32, lane, round8<T>(e), round8<T>(e + 8), acc);
    }
  };
  if (count > 0) fetch(0, tiles);
  for (int32_t n = 0; n < count; ++n) {
    wait_loads_all();
    lds_barrier();
    sum_step(tiles + (n & 1) * TILE, tiles + (~n & 1) * TILE, n * kTile);
  }
  delta = sum_halves(delta);
  if (live && lane < 32) p.delta[out_row] = delta;
  float store = p.scale;
  if constexpr (Mfma<T>::kNarrow) {
    // |ds_j| <= max p |dP| + max p |D|: the row's ds are lifted so that this comes to 2^14 .. 2^15
    // (the maxima's cost: below 4% of the kernel)
    const float bound = max_halves(most_x) + max_halves(most_w) * __builtin_fabsf(delta);
    const int up = min(15 - __builtin_amdgcn_frexp_expf(bound), 60);
    lse2 -= float(up);
    store = __builtin_ldexpf(store, -up);
  }
#pragma unroll
  for (int d = 0; d < NP * 2 + 2; ++d) acc[d] = f32x16{};
  const int32_t first = few ? 0 : count & 1;  // the buffer that holds tile 0
  for (int32_t n = 0; n < count; ++n) {
    wait_loads_all();
    lds_barrier();
    step(tiles + ((n + first) & 1) * TILE, tiles + (~(n + first) & 1) * TILE, n * kTile);
  }
  if (live)
    store_columns<T, NP * 2 + 2>(static_cast<char *>(p.dq) + out_row * (DIM + 64) * es, acc,
                                 store, lane);
}

// ---- backward: dk, dv and each head's share of the shared key part's gradient ---------------

// Two wavefronts for 32 keys, on one SIMD: the first computes S, p and dv, the second dP, ds and
// dk, five products of 32 rows by 64 each (dim 128), and p goes from the first to the second through
// LDS, in float32, where lane and register are the same on both sides.  One wavefront for both
// would need more registers than a half of a SIMD's (alone on its SIMD it took 4% longer than two
// of 16 keys), and 16 keys a wavefront, which do fit, read every tile twice as often: 569 us in
// place of 546 for 4 x 2048 tokens of 32 heads.
template <typename T, int DIM>
__global__ __launch_bounds__(kKeyThreads, 2) void latent_dkey_kernel(ExpandedPlan p) {
  constexpr int NP = DIM / 64;
  constexpr int TILE = (2 * NP + 1) * 8192;  // queries (own part, shared part), gradients
  constexpr int WAVES = kKeyThreads / 64;
  // (one LDS variable: with several the compiler would wait for the loads into the other buffer
  // before it reads this one)
  struct Lds {
    char tiles[2 * TILE];
    char weights[kRows / 32 * 8192];  // p: 32 keys and 64 query rows of each pair
    float stats[2][2][kTile];         // lse * log2(e), D
  };
  __shared__ __attribute__((aligned(16))) Lds lds;
  char *tiles = lds.tiles;
  auto &stats = lds.stats;
  int32_t head, tile;
  if (!head_and_tile(p, p.k_tiles, head, tile)) return;
  const TileAt at = find_tile<false>(p, tile);
  if (at.seq < 0) return;
  const Span q = span(p.q_off, p.q_off_stride, p.Tq, p.q_each, at.seq);
  const Span k = span(p.k_off, p.k_off_stride, p.Tk, p.k_each, at.seq);

  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t es = sizeof(T);
  const int pair = wave % (WAVES / 2);
  const bool second = wave >= WAVES / 2;
  const int32_t key = at.tile * kRows + pair * 32 + (lane & 31);
  const bool live = key < k.count;
  const int64_t tok = k.first + key;
  // query i sees key j if j < i + shift; n0: the first 64-row tile with a row that sees one
  const int32_t shift = k.count - q.count + 1;
  const int32_t first_i = p.causal ? max(0, at.tile * kRows - shift + 1) : 0;
  const int32_t n0 = first_i / kTile;
  const int32_t last_key = min(at.tile * kRows + kRows, k.count) - 1;

  const char *qb = static_cast<const char *>(p.q) + (int64_t(q.first) * p.q_tok + head * p.q_head) * es;
  const char *gb = static_cast<const char *>(p.grad) + (int64_t(q.first) * p.g_tok + head * p.g_head) * es;
  const float *lse = p.lse + int64_t(q.first) * p.heads + head;
  const float *del = p.delta + int64_t(q.first) * p.heads + head;
  // The statistics of a tile's rows, one row a lane, read a tile ahead by every wavefront (under a
  // condition the compiler would wait for them at its end) and put into LDS by the first.
  float next_lse = 0.0f, next_delta = 0.0f;
  // p, at most 1 (and a rounding of lse), goes to narrow types times 2^kUp
  constexpr float kUp = Mfma<T>::kNarrow ? 14.0f : 0.0f;
  constexpr float kDown = Mfma<T>::kNarrow ? 0x1p-14f : 1.0f;
  auto fetch = [&](int32_t i0, char *__restrict__ to) {
    fetch_rows<NP + 1, WAVES>(qb, p.q_tok * es, i0, q.count - 1, wave, lane, to);
    fetch_rows<NP, WAVES>(gb, p.g_tok * es, i0, q.count - 1, wave, lane, to + (NP + 1) * 8192);
  };
  auto fetch_stats = [&](int32_t i0) {
    const int64_t i = int64_t(min(i0 + lane, q.count - 1)) * p.heads;
    next_lse = lse[i];
    next_delta = del[i];
  };
  auto put_stats = [&](int slot, int32_t i0) {
    if (wave == 0) {  // rows that see nothing, or do not exist: p = exp2(s - infinity) = 0
      const bool real = i0 + lane < q.count;
      stats[slot][0][lane] =
          real && next_lse != kNegInf ? next_lse * kLog2eF - kUp : __builtin_huge_valf();
      stats[slot][1][lane] = real ? next_delta : 0.0f;
    }
  };
  const float scale2 = p.negative ? -p.scale_log2 : p.scale_log2;

  // The two wavefronts' ways are apart from here on, so that each has registers for its own
  // operands and accumulators only; they meet at the same barriers.
  auto run = [&](auto role) {
    constexpr bool SECOND = decltype(role)::value;
    constexpr int OPERANDS = SECOND ? NP * 4 : NP * 4 + 4, BLOCKS = SECOND ? NP * 2 + 2 : NP * 2;
    s16x8 f[OPERANDS];  // values; of the first wavefront, keys
    const char *row = SECOND ? static_cast<const char *>(p.v) + (tok * p.v_tok + head * p.v_head) * es
                             : static_cast<const char *>(p.k) + (tok * p.k_tok + head * p.k_head) * es;
    load_operands<NP * 4>(row, live, lane, f);
    if constexpr (!SECOND)
      load_operands<4>(static_cast<const char *>(p.kr) + tok * p.kr_tok * es, live, lane,
                       f + NP * 4);
    f32x16 acc[BLOCKS];  // dk and the shared part's gradient; dv
#pragma unroll
    for (int d = 0; d < BLOCKS; ++d) acc[d] = f32x16{};
    f32x16 x[2];  // dP of the tile's two halves, then ds; p
    // Narrow types: ds times `lift`, and so acc.  The rows that see a key are as different as their
    // gradients, so the key's factor is lowered, and what was summed with it, when one passes it.
    // (540 - 590 us in place of 515 - 565 for 4 x 2048 tokens of 32 heads in float16.)
    float lift = 0x1p26f;

    auto first_half = [&](const char *__restrict__ cur, char *__restrict__ other,
                          char *__restrict__ to, const float *__restrict__ st, int32_t i0) {
      if (i0 + kTile < q.count) fetch(i0 + kTile, other);
      const bool whole = !p.causal || last_key < i0 + shift;
      x[0] = x[1] = f32x16{};
      panel_products<T, SECOND ? NP : NP + 1>(cur + (SECOND ? (NP + 1) * 8192 : 0), lane, f, x);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (!SECOND) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int at_row = i * 32 + 8 * c + 4 * (lane >> 5);
            const f32x4 l = *reinterpret_cast<const f32x4 *>(st + at_row);
            f32x4 w;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              w[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i][4 * c + r], scale2, -l[r]));
              if (!whole) w[r] = key < i0 + at_row + r + shift ? w[r] : 0.0f;
              x[i][4 * c + r] = w[r];
            }
            *reinterpret_cast<f32x4 *>(to + i * 4096 + c * 1024 + lane * 16) = w;
          }
        }
      }
    };
    auto second_half = [&](const char *__restrict__ cur, const char *__restrict__ from,
                           const float *__restrict__ st) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float e[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          f32x4 w = {1.0f, 1.0f, 1.0f, 1.0f}, d = {};
          if constexpr (SECOND) {
            w = *reinterpret_cast<const f32x4 *>(from + i * 4096 + c * 1024 + lane * 16);
            d = *reinterpret_cast<const f32x4 *>(st + kTile + i * 32 + 8 * c + 4 * (lane >> 5));
          }
#pragma unroll
          for (int r = 0; r < 4; ++r)
            e[4 * c + r] = SECOND ? w[r] * (x[i][4 * c + r] - d[r]) : x[i][4 * c + r];
        }
        if constexpr (SECOND && Mfma<T>::kNarrow) {
          float high = 0.0f;
#pragma unroll
          for (int r = 0; r < 16; ++r) high = fmaxf(high, __builtin_fabsf(e[r]));
          high = max_halves(high);
          if (__any(high * lift > 65000.0f)) {
            float f = 1.0f;
            if (high * lift > 65000.0f) {  // 2^11 .. 2^12 from here on
              const float now = __builtin_ldexpf(1.0f, 12 - __builtin_amdgcn_frexp_expf(high));
              f = now / lift;
              lift = now;
            }
#pragma unroll
            for (int d = 0; d < BLOCKS; ++d) acc[d] *= f;
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) e[r] *= lift;
        }
        column_product<T, BLOCKS>(cur + (SECOND ? 0 : (NP + 1) * 8192), i * 32, lane,
                                  round8<T>(e), round8<T>(e + 8), acc);
      }
    };
    char *weights = lds.weights + pair * 8192;
    for (int32_t n = n0; n * kTile < q.count; ++n) {
      const int slot = (n - n0) & 1;
      wait_loads_all();
      put_stats(slot, n * kTile);
      lds_barrier();
      fetch_stats((n + 1) * kTile);
      const char *cur = tiles + slot * TILE;
      const float *st = &stats[slot][0][0];
      first_half(cur, tiles + (slot ^ 1) * TILE, weights, st, n * kTile);
      lds_barrier();
      second_half(cur, weights, st);
    }
    if (!live) return;
    const int64_t out_row = tok * p.heads + head;
    if constexpr (!SECOND) {
      store_columns<T, BLOCKS>(static_cast<char *>(p.dv) + out_row * DIM * es, acc, kDown, lane);
    } else {
      const float f = Mfma<T>::kNarrow ? p.scale * (kDown / lift) : p.scale;
      store_columns<T, NP * 2>(static_cast<char *>(p.dk) + out_row * DIM * es, acc, f, lane);
      float *part = p.dkr_part + (int64_t(head) * p.Tk + tok) * 64;
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const f32x16 &a = acc[NP * 2 + d];
          *reinterpret_cast<float4 *>(part + d * 32 + c * 8 + 4 * (lane >> 5)) =
              make_float4(a[4 * c] * f, a[4 * c + 1] * f, a[4 * c + 2] * f, a[4 * c + 3] * f);
        }
    }
  };
  if (n0 * kTile < q.count) {
    fetch_stats(n0 * kTile);
    fetch(n0 * kTile, tiles);
  }
  if (second)
    run(std::true_type());
  else
    run(std::false_type());
}

// The shared key part's gradient: the heads' shares added in order.  One thread for four
// elements of a token.  Tokens outside all sequences get zero gradients, here and (rows of
// dq, dk, dv) by the threads beyond.
template <typename T>
__global__ __launch_bounds__(kBlockThreads) void latent_dshared_kernel(ExpandedPlan p) {
  const int64_t i = int64_t(blockIdx.x) * kBlockThreads + threadIdx.x;
  const int64_t es = sizeof(T);
  const int64_t row = i / 16;
  const bool key = row < p.Tk;
  const int64_t tok = key ? row : row - p.Tk;
  if (!key && tok >= p.Tq) return;
  const int64_t *off = key ? p.k_off : p.q_off;
  bool inside = true;
  if (off != nullptr) {
    const int64_t stride = key ? p.k_off_stride : p.q_off_stride;
    inside = tok >= off[0] && tok < off[p.B * stride];
  }
  if (!key) {
    if (inside) return;
    const int64_t n = int64_t(p.heads) * (p.dim + 64) * es / 16;
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<char *>(p.dq) + tok * n * 16);
    for (int64_t j = i % 16; j < n; j += 16) to[j] = make_uint4(0, 0, 0, 0);
    return;
  }
  float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (inside) {
    const float *part = p.dkr_part + tok * 64 + (i % 16) * 4;
#pragma unroll 4
    for (int32_t h = 0; h < p.heads; ++h) {
      const float4 x = *reinterpret_cast<const float4 *>(part + int64_t(h) * p.Tk * 64);
      t.x += x.x;
      t.y += x.y;
      t.z += x.z;
      t.w += x.w;
    }
  } else {
    const int64_t n = int64_t(p.heads) * p.dim * es / 16;
    for (void *out : {p.dk, p.dv}) {
      uint4 *to = reinterpret_cast<uint4 *>(static_cast<char *>(out) + tok * n * 16);
      for (int64_t j = i % 16; j < n; j += 16) to[j] = make_uint4(0, 0, 0, 0);
    }
  }
  *reinterpret_cast<uint2 *>(static_cast<char *>(p.dkr) + (tok * 64 + (i % 16) * 4) * es) =
      make_uint2(Mfma<T>::pack(t.x, t.y), Mfma<T>::pack(t.z, t.w));
}

// ---- launches -------------------------------------------------------------------------------

uint32_t head_grid(int64_t heads, int64_t tiles) {
  return uint32_t((heads * tiles + kXcds - 1) / kXcds * kXcds);
}

template <typename T, int DIM>
int run_forward(ExpandedPlan &p, void *stream) {
  return launch_kernel(reinterpret_cast<const void *>(&latent_forward_kernel<T, DIM>),
                       dim3(head_grid(p.heads, p.q_tiles)), kBlockThreads, 0, stream, &p);
}

template <typename T, int DIM>
int run_backward(ExpandedPlan &p, void *stream) {
  int st = ROPE_OK;
  const bool any = p.heads > 0 && p.B > 0;
  if (any && p.q_tiles > 0)
    st = launch_kernel(reinterpret_cast<const void *>(&latent_dquery_kernel<T, DIM>),
                       dim3(head_grid(p.heads, p.q_tiles)), kBlockThreads, 0, stream, &p);
  if (st == ROPE_OK && any && p.k_tiles > 0)
    st = launch_kernel(reinterpret_cast<const void *>(&latent_dkey_kernel<T, DIM>),
                       dim3(head_grid(p.heads, p.k_tiles)), kKeyThreads, 0, stream, &p);
  if (st != ROPE_OK) return st;
  const int64_t threads = (p.Tk + (p.q_off != nullptr ? p.Tq : 0)) * 16;
  if (threads == 0) return ROPE_OK;
  return launch_kernel(reinterpret_cast<const void *>(&latent_dshared_kernel<T>),
                       dim3(uint32_t((threads + kBlockThreads - 1) / kBlockThreads)), kBlockThreads,
                       0, stream, &p);
}

}  // namespace
}  // namespace ropeamd

using namespace ropeamd;

ROPE_API int rope_latent_attention(const rope_tensor *query, const rope_tensor *key,
                                   const rope_tensor *key_rope, const rope_tensor *value,
                                   const rope_tensor *query_offsets,
                                   const rope_tensor *key_offsets, int64_t num_sequences,
                                   double scale, int causal, const rope_tensor *out,
                                   const rope_tensor *lse, void *stream) {
  ExpandedPlan plan;
  std::string err;
  const int st = plan_expanded(query, key, key_rope, value, query_offsets, key_offsets,
                               num_sequences, scale, causal, out, lse, &plan, &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
  if (plan.noop) return ROPE_OK;
  if (plan.dt == ROPE_F16)
    return plan.dim == 128 ? run_forward<_Float16, 128>(plan, stream)
                           : run_forward<_Float16, 64>(plan, stream);
  return plan.dim == 128 ? run_forward<__bf16, 128>(plan, stream)
                         : run_forward<__bf16, 64>(plan, stream);
}

ROPE_API int64_t rope_latent_attention_backward_workspace(int64_t query_tokens, int64_t key_tokens,
                                                          int64_t num_heads) {
  return expanded_workspace(query_tokens, key_tokens, num_heads);
}

ROPE_API int rope_latent_attention_backward(
    const rope_tensor *grad, const rope_tensor *query, const rope_tensor *key,
    const rope_tensor *key_rope, const rope_tensor *value, const rope_tensor *out,
    const rope_tensor *lse, const rope_tensor *query_offsets, const rope_tensor *key_offsets,
    int64_t num_sequences, double scale, int causal, const rope_tensor *dquery,
    const rope_tensor *dkey, const rope_tensor *dkey_rope, const rope_tensor *dvalue,
    void *workspace, int64_t workspace_bytes, void *stream) {
  ExpandedPlan plan;
  std::string err;
  const int st = plan_expanded_backward(grad, query, key, key_rope, value, out, lse, query_offsets,
                                        key_offsets, num_sequences, scale, causal, dquery, dkey,
                                        dkey_rope, dvalue, workspace, workspace_bytes, &plan, &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
  if (plan.noop) return ROPE_OK;
  if (plan.dt == ROPE_F16)
    return plan.dim == 128 ? run_backward<_Float16, 128>(plan, stream)
                           : run_backward<_Float16, 64>(plan, stream);
  return plan.dim == 128 ? run_backward<__bf16, 128>(plan, stream)
                         : run_backward<__bf16, 64>(plan, stream);
}
