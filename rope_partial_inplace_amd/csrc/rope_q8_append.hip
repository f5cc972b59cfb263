// rope_q8_append.hip -- rotating a batch's new keys by position and appending keys and values to a
// paged cache of 8-bit codes with a scale for each block of tokens and head, the queries rotated by
// the same launch (gfx950).
//
// Of a block's new elements x (keys after their rotation, in float32) the largest size `top` gives
// the scale the block needs -- int8: top / 127; e4m3: the smallest power of two >= top / 448 -- and
//   scale = max(need, present scale if the block holds earlier tokens),  code = round(x (1 / scale));
// where that raises the scale, the earlier tokens' codes c become round(c (old / scale)).
// A floating point code has the same relative precision under any scale that fits, so e4m3 gives up
// nothing with powers of two, and its codes are rounded once, however often the scale grows.
//
// A few operations for every 3 bytes moved: bound by HBM, and for a decoding step by its launch and
// its dependent reads.  One group of lanes (as many as a block's items of one head need, up to a
// wavefront) owns all tokens of a block and head, so that the maximum is a few lane exchanges, and
// nothing is shared between wavefronts: no atomics, no LDS, no order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "rope.h"
#include "rope_io.h"
#include "rope_launch.h"
#include "rope_q8.h"
#include "rope_q8_plan.h"

namespace ropeamd {
namespace {

// V elements of a row from `e` on, and (pairs) V more a partner's distance on, in float32.
template <int V, bool PAIR>
struct Elements {
  float a[V], b[PAIR ? V : 1];
  int32_t e;
  bool two;  // b holds elements
};

template <typename T, int V>
__device__ inline void load_floats(const T *p, float *f) {
  if constexpr (V == 1)
    f[0] = Io<T>::from_raw(*reinterpret_cast<const typename Io<T>::raw *>(p));
  else
    Io<T>::unpack(*reinterpret_cast<const uint4 *>(p), f);
}

// The V / 2 cos (or sin) values of a GPT-J vector: 8 bytes.
template <typename T>
__device__ inline void load_half_floats(const T *p, float *f) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  Io<T>::word_to_floats(w.x, f);
  Io<T>::word_to_floats(w.y, f + Io<T>::kPerWord);
}

// Item `unit` of a row, rotated where it lies in the slice (cs: the token's cosines and sines).
template <typename T, int V, bool NEOX>
__device__ inline Elements<V, NEOX || V == 1> item_of(const T *in, const T *cs, uint32_t unit,
                                                      uint32_t rot_items, int32_t rot_start,
                                                      int32_t half) {
  constexpr bool PAIR = NEOX || V == 1;
  Elements<V, PAIR> x;
  x.two = false;
  if (unit >= rot_items) {  // outside the slice
    x.e = int32_t(unit - rot_items) * V;
    if (x.e >= rot_start && rot_items != 0) x.e += 2 * half;
    load_floats<T, V>(in + x.e, x.a);
    return x;
  }
  x.e = rot_start + int32_t(unit) * (V == 1 && !NEOX ? 2 : V);
  float p[V], c[V], s[V];
  load_floats<T, V>(in + x.e, p);
  if constexpr (PAIR) {
    float q[V];
    load_floats<T, V>(in + x.e + (NEOX ? half : 1), q);
    load_floats<T, V>(cs + int32_t(unit) * V, c);
    load_floats<T, V>(cs + half + int32_t(unit) * V, s);
#pragma unroll
    for (int m = 0; m < V; ++m) {
      x.a[m] = p[m] * c[m] - q[m] * s[m];
      x.b[m] = q[m] * c[m] + p[m] * s[m];
    }
    x.two = true;
  } else {
    load_half_floats<T>(cs + int32_t(unit) * (V / 2), c);
    load_half_floats<T>(cs + half + int32_t(unit) * (V / 2), s);
#pragma unroll
    for (int m = 0; m < V / 2; ++m) {
      x.a[2 * m] = p[2 * m] * c[m] - p[2 * m + 1] * s[m];
      x.a[2 * m + 1] = p[2 * m + 1] * c[m] + p[2 * m] * s[m];
    }
  }
  return x;
}

template <typename T>
__device__ inline const T *angles(const AppendQ8Plan &p, int64_t token) {
  const int64_t pos = p.positions[token * p.pos_stride];
  return static_cast<const T *>(p.table) + min(max(pos, int64_t(0)), p.max_seq - 1) * p.table_stride;
}

// ---- queries: an item a lane, as in the append to a cache without codes -------------------------
template <typename T, int V, bool NEOX>
__device__ inline void rotate_queries(const AppendQ8Plan &p, int64_t block) {
  const AppendRows &r = p.query;
  const int64_t it = block * kQ8Block + threadIdx.x;
  if (it >= r.all) return;
  int64_t t;
  uint32_t i;  // item of the token
  if (p.idx32) {
    const uint32_t q = div_by(r.div_total, uint32_t(it));
    t = q;
    i = uint32_t(it) - q * r.total;
  } else {
    t = it / r.total;
    i = uint32_t(it - t * r.total);
  }
  const uint32_t h = div_by(r.div_items, i), unit = i - h * r.items;
  const T *in = static_cast<const T *>(r.in) + t * r.in_tok + int64_t(h) * r.in_head;
  T *out = static_cast<T *>(r.out) + t * r.out_tok + int64_t(h) * r.out_head;
  if (unit >= r.rot_items) {  // copied bit for bit
    int64_t e = int64_t(unit - r.rot_items) * V;
    if (e >= r.rot_start) e += 2 * p.half;
    if constexpr (V == 1)
      *reinterpret_cast<typename Io<T>::raw *>(out + e) =
          *reinterpret_cast<const typename Io<T>::raw *>(in + e);
    else
      *reinterpret_cast<uint4 *>(out + e) = *reinterpret_cast<const uint4 *>(in + e);
    return;
  }
  const auto x = item_of<T, V, NEOX>(in, angles<T>(p, t), unit, r.rot_items, r.rot_start, p.half);
  auto store = [&](T *to, const float *f) {
    if constexpr (V == 1)
      Io<T>::store1(to, 0, f[0]);
    else
      *reinterpret_cast<uint4 *>(to) = Io<T>::pack(f);
  };
  store(out + x.e, x.a);
  if constexpr (NEOX || V == 1)
    if (x.two) store(out + x.e + (NEOX ? p.half : 1), x.b);
}

// ---- keys and values -----------------------------------------------------------------------------
// What a wavefront has of a sequence: `count` new tokens, `first` and on of the batch, for one block,
// whose `before` earlier tokens precede them.
struct Place {
  int64_t first = 0, page = -1;
  int32_t count = 0, before = 0;
  int32_t row0 = 0, block = 0;  // the block's first row in its page, and its number there
};

// Place `u` of the plan's numbering, the same for all lanes; false: it has no tokens.
__device__ inline bool find_place(const AppendQ8Plan &p, int64_t u, Place *out) {
  const Sequences &s = p.seq;
  auto first_place = [&](int64_t offset, int64_t i) {
    return p.by_token ? offset : int64_t(div_by(p.div_block, uint32_t(offset))) + 2 * i;
  };
  auto offset = [&](int64_t i) {
    return min(max(s.offsets[i * s.off_stride], int64_t(0)), s.T);
  };
  int64_t b = 0, o0, o1;
  if (s.offsets == nullptr) {
    int64_t n = s.B;  // the last b with first_place(b) <= u, in [b, b + n)
    while (n > 1) {   // ends: halved every time
      const int64_t mid = n / 2;
      if (first_place((b + mid) * s.each, b + mid) <= u) {
        b += mid;
        n -= mid;
      } else {
        n = mid;
      }
    }
    o0 = b * s.each;
    o1 = o0 + s.each;
  } else {
    // the same, 64 offsets at a time: ascending, they make the lanes below a run from lane 0 on
    const int lane = int(threadIdx.x) & 63;
    int64_t n = s.B;
    while (n > 1) {  // ends: n becomes n / 64 rounded up, or less
      const int64_t step = (n + 63) >> 6, i = lane * step;
      const bool below = i < n && first_place(offset(b + i), b + i) <= u;
      const int64_t run = (63 - __builtin_clzll(__ballot(below) | 1ull)) * step;
      b += run;
      n = min(step, n - run);
    }
    o0 = offset(b);
    o1 = offset(b + 1);
  }
  const int64_t n = o1 - o0;
  const int64_t len = min(max(s.lens[b * s.len_stride], int64_t(0)), s.max_pages * s.page_size);
  const int64_t start = len - n;  // place of the sequence's first new token (below 0: cut off)
  const int64_t first = max(start, int64_t(0));
  const int64_t k0 = u - first_place(o0, b);
  if (n <= 0 || len <= first || k0 < 0) return false;
  // blocks divide pages, and pages start at place 0: place / block numbers a sequence's blocks
  int64_t lo;  // the first new token of this block
  if (p.by_token) {
    lo = start + k0;
    const bool begins = lo == first || (lo > first && lo == int64_t(p.block) *
                                            div_by(p.div_block, uint32_t(lo)));
    if (k0 >= n || !begins) return false;
  } else {
    lo = max(first, (div_by(p.div_block, uint32_t(first)) + k0) * p.block);
    if (lo >= len) return false;
  }
  const int64_t begin = int64_t(div_by(p.div_block, uint32_t(lo))) * p.block;
  const int64_t page = div_by(s.div_page, uint32_t(begin));
  out->page = s.table[b * s.table_seq + page * s.table_page];
  if (out->page < 0 || out->page >= s.num_pages) return false;
  out->first = o0 + (lo - start);
  out->count = int32_t(min(len, begin + p.block) - lo);
  out->before = int32_t(lo - begin);
  out->row0 = int32_t(begin - page * s.page_size);
  out->block = int32_t(div_by(p.div_block, uint32_t(out->row0)));
  return true;
}

template <typename T, int V, bool NEOX, bool E4M3>
__device__ inline void append_block(const AppendQ8Plan &p, const Place &at, int32_t head2) {
  const int lane = int(threadIdx.x) & 63;
  const bool mine = head2 < 2 * p.heads;
  const int64_t h = (mine ? head2 : 0) >> 1;
  const Q8Rows &r = p.kv[head2 & 1];
  const uint32_t lanes = uint32_t(p.lanes), l = uint32_t(lane) & (lanes - 1);
  const uint32_t n = mine ? uint32_t(at.count) * r.items : 0;
  auto read = [&](uint32_t i, uint32_t *row) {
    const uint32_t t = div_by(r.div_items, i);
    *row = t;
    const T *in = static_cast<const T *>(r.in) + (at.first + t) * r.in_tok + h * r.in_head;
    const T *cs = r.rot_items != 0 ? angles<T>(p, at.first + t) : nullptr;
    return item_of<T, V, NEOX>(in, cs, i - t * r.items, r.rot_items, r.rot_start, p.half);
  };
  float *scale_at = r.scales + at.page * r.s_page + at.block * r.s_block + h * r.s_head;
  const float old = mine && at.before > 0 ? *scale_at : 0.0f;

  float top = 0.0f;
  bool bad = false;
  for (uint32_t i = l; i < n; i += lanes) {
    uint32_t row;
    const auto x = read(i, &row);
#pragma unroll
    for (int m = 0; m < V; ++m) top = larger(top, x.a[m], &bad);
    if constexpr (NEOX || V == 1)
      if (x.two) {
#pragma unroll
        for (int m = 0; m < V; ++m) top = larger(top, x.b[m], &bad);
      }
  }
  for (uint32_t d = 1; d < lanes; d *= 2) top = fmaxf(top, __shfl_xor(top, int(d)));
  float now = needed_scale<E4M3>(top);
  if (!E4M3) {  // int8 has no NaN: the scale says it
    const uint64_t group = (lanes == 64 ? ~0ull : (1ull << lanes) - 1) << (uint32_t(lane) - l);
    if ((__ballot(bad) & group) != 0) now = __builtin_nanf("");
  }
  if (at.before > 0 && now == now && !(old <= now)) now = old;  // the larger; a NaN stays

  uint8_t *rows = r.codes + at.page * r.page + int64_t(at.row0) * r.row + h * r.head;
  if (mine && at.before > 0 && now != old) {  // the earlier tokens' codes under the new scale
    const float ratio = old / now;
    const int32_t width = r.wide_rows ? 16 : 1, pieces = r.dim / width;
    for (int32_t i = int32_t(l); i < at.before * pieces; i += int32_t(lanes)) {
      const int32_t t = i / pieces;
      uint8_t *c = rows + int64_t(t) * r.row + (i - t * pieces) * width;
      if (r.wide_rows) {
        const uint4 v = *reinterpret_cast<const uint4 *>(c);
        *reinterpret_cast<uint4 *>(c) = make_uint4(recode<E4M3>(v.x, ratio), recode<E4M3>(v.y, ratio),
                                                   recode<E4M3>(v.z, ratio), recode<E4M3>(v.w, ratio));
      } else {
        *c = uint8_t(recode<E4M3>(*c, ratio));
      }
    }
  }
  const float inv = 1.0f / now;
  for (uint32_t i = l; i < n; i += lanes) {
    uint32_t row;
    const auto x = read(i, &row);
    uint8_t *to = rows + int64_t(at.before + int32_t(row)) * r.row + x.e;
    store_codes<E4M3, V>(to, x.a, inv);
    if constexpr (NEOX || V == 1)
      if (x.two) store_codes<E4M3, V>(to + (NEOX ? p.half : 1), x.b, inv);
  }
  if (mine && l == 0 && (at.before == 0 || now != old)) *scale_at = now;
}

template <typename T, int V, bool NEOX, bool E4M3>
__global__ __launch_bounds__(kQ8Block) void append_q8_kernel(AppendQ8Plan p) {
  const int64_t all = p.kv_blocks + p.query_blocks;
  for (int64_t block = blockIdx.x; block < all; block += gridDim.x) {
    if (block >= p.kv_blocks) {
      rotate_queries<T, V, NEOX>(p, block - p.kv_blocks);
      continue;
    }
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int64_t w = block * (kQ8Block / 64) + wave;
    const int64_t u = p.idx32 ? int64_t(div_by(p.div_groups, uint32_t(w))) : w / p.head_groups;
    Place at;
    if (u >= p.places || !find_place(p, u, &at)) continue;
    const int32_t head2 = int32_t(w - u * p.head_groups) * (64 >> p.lanes_log2) +
                          ((int32_t(threadIdx.x) & 63) >> p.lanes_log2);
    append_block<T, V, NEOX, E4M3>(p, at, head2);
  }
}

template <typename T, bool E4M3>
const void *pick_append_q8(const AppendQ8Plan &p) {
  constexpr int V = Io<T>::kPer16;
#define ROPE_KA(VV, NX) reinterpret_cast<const void *>(&append_q8_kernel<T, VV, NX, E4M3>)
  if (p.vector_io) return p.neox ? ROPE_KA(V, true) : ROPE_KA(V, false);
  return p.neox ? ROPE_KA(1, true) : ROPE_KA(1, false);
#undef ROPE_KA
}

template <typename T>
const void *pick_append_q8_codes(const AppendQ8Plan &p) {
  return p.e4m3 ? pick_append_q8<T, true>(p) : pick_append_q8<T, false>(p);
}

}  // namespace
}  // namespace ropeamd

using namespace ropeamd;

ROPE_API int rope_append_paged_cache_q8(
    const rope_tensor *positions, const rope_tensor *query, const rope_tensor *key,
    const rope_tensor *value, const rope_tensor *cos_sin_cache, const rope_tensor *page_table,
    const rope_tensor *seq_lens, const rope_tensor *token_offsets, int64_t query_rot_start,
    int64_t key_rot_start, int is_neox_style, const rope_tensor *query_out,
    const rope_tensor *key_cache, const rope_tensor *value_cache, const rope_tensor *key_scales,
    const rope_tensor *value_scales, void *stream) {
  AppendQ8Plan plan;
  std::string err;
  const int st = plan_append_q8(positions, query, key, value, cos_sin_cache, page_table, seq_lens,
                                token_offsets, query_rot_start, key_rot_start, is_neox_style,
                                query_out, key_cache, value_cache, key_scales, value_scales, &plan,
                                &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
  if (plan.noop) return ROPE_OK;
  const void *fn = plan.dt == ROPE_F32   ? pick_append_q8_codes<float>(plan)
                   : plan.dt == ROPE_F16 ? pick_append_q8_codes<_Float16>(plan)
                                         : pick_append_q8_codes<__bf16>(plan);
  // a launch has fewer than 2^32 threads: more blocks than that are taken in turns
  const int64_t blocks = std::min(plan.kv_blocks + plan.query_blocks, int64_t(1) << 23);
  return launch_kernel(fn, dim3(uint32_t(blocks)), kQ8Block, 0, stream, &plan);
}
