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
// its dependent reads.  One group of lanes (as many as hold a block's elements of one head, 32 each) owns all
// its tokens, so that the maximum is a few lane exchanges; only those of long blocks are two or four
// wavefronts, which meet in LDS.  (11167 tokens of blocks of 32: 53.6 us with two for a head, 58.4 with
// four, which hold half as much each.)  No atomics, no order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <type_traits>

#include "rope.h"
#include "rope_io.h"
#include "rope_launch.h"
#include "rope_q8.h"
#include "rope_q8_plan.h"

namespace ropeamd {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes that are used once.
__device__ inline uint4 load_once(const void *p) {
  const u32x4 v = __builtin_nontemporal_load(static_cast<const u32x4 *>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ inline void store_once(void *p, const uint4 &v) {
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, static_cast<u32x4 *>(p));
}

// V elements as they lie in memory, and in float32.  ONCE: no other item reads them.
template <typename T, int V>
using Words = std::conditional_t<V == 1, typename Io<T>::raw, uint4>;

template <typename T, int V, bool ONCE>
__device__ inline Words<T, V> load_words(const T *p) {
  if constexpr (V == 1)
    return *reinterpret_cast<const typename Io<T>::raw *>(p);
  else
    return ONCE ? load_once(p) : *reinterpret_cast<const uint4 *>(p);
}

template <typename T, int V>
__device__ inline void to_floats(const Words<T, V> &w, float *f) {
  if constexpr (V == 1)
    f[0] = Io<T>::from_raw(w);
  else
    Io<T>::unpack(w, f);
}

template <typename T, int V, bool ONCE>
__device__ inline void load_floats(const T *p, float *f) {
  to_floats<T, V>(load_words<T, V, ONCE>(p), f);
}

// The V / 2 cos (or sin) values of a GPT-J vector: 8 bytes.
template <typename T>
__device__ inline void load_half_floats(const T *p, float *f) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  Io<T>::word_to_floats(w.x, f);
  Io<T>::word_to_floats(w.y, f + Io<T>::kPerWord);
}

// Where an item of a row lies: V elements from `e` on, and if it is rotated and made of pairs V more
// from e + partner on.
struct Spot {
  int32_t e;
  bool turned;
};

template <int V, bool NEOX>
__device__ inline Spot spot_of(uint32_t unit, uint32_t rot_items, int32_t rot_start, int32_t half) {
  Spot s;
  s.turned = unit < rot_items;
  int32_t e = int32_t(unit - rot_items) * V;  // outside the slice
  if (e >= rot_start && rot_items != 0) e += 2 * half;
  s.e = s.turned ? rot_start + int32_t(unit) * (V == 1 && !NEOX ? 2 : V) : e;
  return s;
}

template <bool NEOX>
__device__ inline int32_t partner(int32_t half) {
  return NEOX ? half : 1;
}

// The cosines and sines of an item (cs: its token's).  An item outside the slice takes some others: there
// are no branches, so that several items' loads are under way at once.
template <typename T, int V, bool NEOX>
struct Turn {
  static constexpr int N = NEOX || V == 1 ? V : V / 2;
  float c[N], s[N];
  __device__ void load(const T *cs, const Spot &at, uint32_t unit, int32_t half) {
    const int32_t u = at.turned ? int32_t(unit) : 0;
    if constexpr (NEOX || V == 1) {
      load_floats<T, V, false>(cs + u * V, c);
      load_floats<T, V, false>(cs + half + u * V, s);
    } else {
      load_half_floats<T>(cs + u * (V / 2), c);
      load_half_floats<T>(cs + half + u * (V / 2), s);
    }
  }
};

// An item as it lies in memory (`q`: the other halves of its pairs; of one outside the slice the same
// elements), and in float32, rotated where it lies in the slice.
template <typename T, int V, bool NEOX>
struct Item {
  static constexpr bool PAIR = NEOX || V == 1;
  Words<T, V> p, q;
  __device__ void load(const T *in, const Spot &at, int32_t half) {
    p = load_words<T, V, true>(in + at.e);
    if constexpr (PAIR) q = load_words<T, V, true>(in + at.e + (at.turned ? partner<NEOX>(half) : 0));
  }
  __device__ void rotate(const Turn<T, V, NEOX> &r, const Spot &at, float *a, float *b) const {
    float x[V];
    to_floats<T, V>(p, x);
    if constexpr (PAIR) {
      float y[V];
      to_floats<T, V>(q, y);
#pragma unroll
      for (int m = 0; m < V; ++m) {
        const float z = x[m] * r.c[m] - y[m] * r.s[m];
        b[m] = y[m] * r.c[m] + x[m] * r.s[m];
        a[m] = at.turned ? z : x[m];
      }
    } else {
#pragma unroll
      for (int m = 0; m < V / 2; ++m) {
        const float y = x[2 * m] * r.c[m] - x[2 * m + 1] * r.s[m];
        const float z = x[2 * m + 1] * r.c[m] + x[2 * m] * r.s[m];
        a[2 * m] = at.turned ? y : x[2 * m];
        a[2 * m + 1] = at.turned ? z : x[2 * m + 1];
      }
    }
  }
};

__device__ inline int64_t position(const AppendQ8Plan &p, int64_t token) {
  return p.positions[token * p.pos_stride];
}
template <typename T>
__device__ inline const T *angles(const AppendQ8Plan &p, int64_t pos) {
  return static_cast<const T *>(p.table) + min(max(pos, int64_t(0)), p.max_seq - 1) * p.table_stride;
}

// ---- queries ------------------------------------------------------------------------------------
// A thread takes one item of HEADS neighbouring heads, which share its cosines and sines.  All are loaded
// before the first is stored: the output may be the input itself, so behind a store the compiler would wait with
// the next load (11167 tokens of 32 heads of 128 and 8 + 8 in blocks of 32: 50.4 us so, 53.6 one by one).
template <typename T, int V, bool NEOX>
__device__ inline void rotate_queries(const AppendQ8Plan &p, int64_t block) {
  constexpr int HEADS = query_heads_of(NEOX);
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
  const uint32_t hg = div_by(r.div_items, i), unit = i - hg * r.items;
  const int64_t h = int64_t(hg) * HEADS;
  const T *in = static_cast<const T *>(r.in) + t * r.in_tok + h * r.in_head;
  T *out = static_cast<T *>(r.out) + t * r.out_tok + h * r.out_head;
  const Spot at = spot_of<V, NEOX>(unit, r.rot_items, r.rot_start, p.half);
  const int heads = int(min(p.query_heads - h, int64_t(HEADS)));
  const int64_t pos = position(p, t);
  Item<T, V, NEOX> x[HEADS];
#pragma unroll
  for (int k = 0; k < HEADS; ++k) x[k].load(in + min(k, heads - 1) * r.in_head, at, p.half);
  Turn<T, V, NEOX> turn;
  turn.load(angles<T>(p, pos), at, unit, p.half);
#pragma unroll
  for (int k = 0; k < HEADS; ++k) {
    if (k >= heads) break;
    T *y = out + k * r.out_head;
    float a[V], b[V];
    x[k].rotate(turn, at, a, b);
    // what lies outside the slice is copied bit for bit (raised to float32 and rounded again, all but a
    // NaN's payload would be)
    if constexpr (V == 1) {
      T v, w;
      Io<T>::store1(&v, 0, a[0]);
      Io<T>::store1(&w, 0, b[0]);
      *reinterpret_cast<typename Io<T>::raw *>(y + at.e) =
          at.turned ? __builtin_bit_cast(typename Io<T>::raw, v) : x[k].p;
      if (at.turned) *(y + at.e + partner<NEOX>(p.half)) = w;
    } else {
      const uint4 w = x[k].p, z = Io<T>::pack(a);
      store_once(y + at.e, make_uint4(at.turned ? z.x : w.x, at.turned ? z.y : w.y,
                                      at.turned ? z.z : w.z, at.turned ? z.w : w.w));
      if constexpr (NEOX)
        if (at.turned) store_once(y + at.e + p.half, Io<T>::pack(b));
    }
  }
}

// ---- keys and values -----------------------------------------------------------------------------
// What a wavefront has of a sequence: `count` new tokens, `first` and on of the batch, for one block,
// whose `before` earlier tokens precede them.
struct Place {
  int64_t first = 0, page = -1;
  int32_t count = 0, before = 0;
  int32_t row0 = 0, block = 0;  // the block's first row in its page, and its number there
};

// Place `u` of the plan's numbering, the same for all lanes; false: it has no tokens.  The page's number
// is read last and not looked at here, so that the tokens' elements can be on their way first.
__device__ inline bool find_place(const AppendQ8Plan &p, int64_t u, Place *out) {
  const Sequences &s = p.seq;
  auto first_place = [&](int64_t offset, int64_t i) {
    return p.by_token ? offset : int64_t(div_by(p.div_block, uint32_t(offset))) + 2 * i;
  };
  const int lane = int(threadIdx.x) & 63;
  const int64_t limit = s.max_pages * s.page_size;
  int64_t b = 0, o0, o1, len;
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
    len = s.lens[b * s.len_stride];
  } else {
    // the same, 64 offsets at a time: ascending, they make the lanes below a run from lane 0 on; the
    // last time with the lengths
    int64_t n = s.B;
    while (true) {  // ends: n becomes n / 64 rounded up, or less
      const int64_t step = (n + 63) >> 6, i = lane * step;
      int64_t o = 0, l = 0;
      if (i <= n && b + i <= s.B) o = min(max(s.offsets[(b + i) * s.off_stride], int64_t(0)), s.T);
      if (step == 1 && i < n) l = s.lens[(b + i) * s.len_stride];
      const bool below = i < n && first_place(o, b + i) <= u;
      const int run = 63 - __builtin_clzll(__ballot(below) | 1ull);
      b += run * step;
      if (step == 1) {
        o0 = __shfl(o, run);
        o1 = __shfl(o, (run + 1) & 63);
        len = __shfl(l, run);
        if (run == 63) o1 = min(max(s.offsets[(b + 1) * s.off_stride], int64_t(0)), s.T);
        break;
      }
      n = min(step, n - run * step);
    }
  }
  len = min(max(len, int64_t(0)), limit);
  const int64_t n = o1 - o0;
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
  out->first = o0 + (lo - start);
  out->count = int32_t(min(len, begin + p.block) - lo);
  out->before = int32_t(lo - begin);
  out->row0 = int32_t(begin - page * s.page_size);
  out->block = int32_t(div_by(p.div_block, uint32_t(out->row0)));
  return true;
}

// New tokens of one block and head by `lanes` neighbouring threads (head below 0: threads without one).
// ROT: rows with rotated items.  Blocks of up to kQ8Held elements a thread stay in registers between
// the maximum and the codes; longer ones are read again (the second time from the caches beside the
// compute unit).

template <typename T, int V, bool NEOX, bool E4M3, bool ROT>
__device__ inline void append_block(const AppendQ8Plan &p, const Q8Rows &r, const Place &at,
                                    int32_t head) {
  constexpr bool PAIR = ROT && (NEOX || V == 1);
  constexpr int ITEM = PAIR ? 2 * V : V, HELD = V == 1 ? 1 : kQ8Held / ITEM;
  const uint32_t lane = threadIdx.x & 63, lanes = uint32_t(p.lanes), l = threadIdx.x & (lanes - 1);
  const bool mine = head >= 0;
  const int64_t h = mine ? head : 0;
  const uint32_t n = mine ? uint32_t(at.count) * r.items : 0;
  const T *in = static_cast<const T *>(r.in) + at.first * r.in_tok + h * r.in_head;
  // Rows of at most `lanes` items lie side by side, 2^row_log2 threads each: a thread has item `unit` of
  // every rows-th row.  Item i of the block: V or (rotated pairs) 2 V floats.
  const uint32_t unit = l & ((1u << r.row_log2) - 1), row0 = l >> r.row_log2;
  const uint32_t rows_at_once = lanes >> r.row_log2, count = uint32_t(at.count);
  const Spot spot = spot_of<V, NEOX>(unit, r.rot_items, r.rot_start, p.half);
  auto read = [&](uint32_t row, const Spot &s, uint32_t item, float *f) {
    const T *from = in + int64_t(row) * r.in_tok;
    if constexpr (ROT) {
      Turn<T, V, NEOX> turn;
      Item<T, V, NEOX> x;
      const int64_t pos = position(p, at.first + row);
      x.load(from, s, p.half);
      turn.load(angles<T>(p, pos), s, item, p.half);
      x.rotate(turn, s, f, f + V);
    } else {
      load_floats<T, V, true>(from + s.e, f);
    }
  };
  const bool held = r.side_by_side && count <= rows_at_once * HELD;
  const bool mine_too = mine && unit < r.items;
  float x[HELD][ITEM];
  if (held) {
    // All rows' loads are under way before the first is needed; rows past the last one repeat it (loads behind
    // branches wait for each other: 50.3 us, not 48.3).
    const Spot s = unit < r.items ? spot : spot_of<V, NEOX>(0, r.rot_items, r.rot_start, p.half);
    const uint32_t item = unit < r.items ? unit : 0, last = max(count, 1u) - 1;
    if constexpr (ROT) {
      Item<T, V, NEOX> raw[HELD];
      int64_t pos[HELD];
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        const int64_t row = min(row0 + k * rows_at_once, last);
        pos[k] = position(p, at.first + row);
        raw[k].load(in + row * r.in_tok, s, p.half);
      }
#pragma unroll
      for (int k = 0; k < HELD; ++k) {
        Turn<T, V, NEOX> turn;
        turn.load(angles<T>(p, pos[k]), s, item, p.half);
        raw[k].rotate(turn, s, x[k], x[k] + V);
      }
    } else {
      Words<T, V> raw[HELD];
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        raw[k] = load_words<T, V, true>(in + int64_t(min(row0 + k * rows_at_once, last)) * r.in_tok + s.e);
#pragma unroll
      for (int k = 0; k < HELD; ++k) to_floats<T, V>(raw[k], x[k]);
    }
  }
  // the elements are on their way: now the page
  const bool kept = at.page >= 0 && at.page < p.seq.num_pages;  // else padding; the same for all lanes
  const int64_t page = kept ? at.page : 0;
  uint8_t *rows = r.codes + page * r.page + int64_t(at.row0) * r.row + h * r.head;
  float *scale_at = r.scales + page * r.s_page + at.block * r.s_block + h * r.s_head;
  const float old = kept && mine && at.before > 0 ? *scale_at : 0.0f;
  // the largest size, over all elements or the finite ones; any_high: of the wavefronts that meet
  uint32_t any_high = 0;
  auto largest = [&](auto only_finite) {
    constexpr bool FINITE = decltype(only_finite)::value;
    uint32_t high = 0;
    auto measure = [&](bool turned, const float *f) {
      auto take = [&](float y) {
        const uint32_t u = size_bits(y);
        high = max(high, FINITE && u >= kNonFinite ? 0u : u);
      };
#pragma unroll
      for (int m = 0; m < V; ++m) take(f[m]);
      if constexpr (PAIR)
        if (turned) {
#pragma unroll
          for (int m = 0; m < V; ++m) take(f[V + m]);
        }
    };
    if (held) {  // a row or an item read twice changes no maximum
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        if (k * rows_at_once < count) measure(spot.turned, x[k]);
      if (!mine) high = 0;
    } else {
      for (uint32_t i = l; i < n; i += lanes) {
        const uint32_t row = div_by(r.div_items, i), item = i - row * r.items;
        const Spot s = spot_of<V, NEOX>(item, r.rot_items, r.rot_start, p.half);
        read(row, s, item, x[0]);
        measure(s.turned, x[0]);
      }
    }
    for (uint32_t d = 1; d < lanes && d < 64; d *= 2)
      high = max(high, uint32_t(__shfl_xor(int(high), int(d))));
    any_high = high;
    if (lanes > 64) {  // with the block's other wavefronts
      __shared__ uint32_t highs[kQ8Block / 64];
      __syncthreads();
      if (lane == 0) highs[threadIdx.x >> 6] = high;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kQ8Block / 64; ++k) {
        any_high = max(any_high, highs[k]);
        if (lanes == kQ8Block || (k ^ int(threadIdx.x >> 6)) < 2) high = max(high, highs[k]);
      }
    }
    return high;
  };
  uint32_t high = largest(std::false_type());
  const bool bad = high >= kNonFinite;
  const bool check = __any(any_high >= kNonFinite);  // of several wavefronts the same for the workgroup
  if (check && E4M3) high = largest(std::true_type());
  if (!kept) return;
  float now = needed_scale<E4M3>(__uint_as_float(high));
  if (!E4M3 && bad) now = __builtin_nanf("");  // int8 has no NaN: the scale says it
  if (at.before > 0 && now == now && !(old <= now)) now = old;  // the larger; a NaN stays

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
  auto encode = [&](auto checked) {
    constexpr bool CHECK = decltype(checked)::value;
    auto write = [&](uint32_t row, const Spot &s, const float *f) {
      uint8_t *to = rows + int64_t(at.before + int32_t(row)) * r.row + s.e;
      store_codes<E4M3, CHECK, V>(to, f, inv);
      if constexpr (PAIR)
        if (s.turned) store_codes<E4M3, CHECK, V>(to + partner<NEOX>(p.half), f + V, inv);
    };
    if (held) {
#pragma unroll
      for (int k = 0; k < HELD; ++k)
        if (mine_too && row0 + k * rows_at_once < count) write(row0 + k * rows_at_once, spot, x[k]);
    } else {
      for (uint32_t i = l; i < n; i += lanes) {
        const uint32_t row = div_by(r.div_items, i), item = i - row * r.items;
        const Spot s = spot_of<V, NEOX>(item, r.rot_items, r.rot_start, p.half);
        read(row, s, item, x[0]);
        write(row, s, x[0]);
      }
    }
  };
  if (E4M3 && check)
    encode(std::true_type());
  else
    encode(std::false_type());
  if (mine && l == 0 && (at.before == 0 || now != old)) *scale_at = now;
}

// Five wavefronts a SIMD: with six the NeoX forms of e4m3 spill 24 registers (blocks of 16, bf16: 51 us, not 55.5).
template <typename T, int V, bool NEOX, bool E4M3>
__global__ __launch_bounds__(kQ8Block) __attribute__((amdgpu_waves_per_eu(5))) void
append_q8_kernel(AppendQ8Plan p) {
  const int64_t block = p.first_block + blockIdx.x;
  if (block >= p.kv_blocks) {
    rotate_queries<T, V, NEOX>(p, block - p.kv_blocks);
    return;
  }
  // a wavefront's part of a place, or that of two or four
  const int each = max(6, p.lanes_log2);
  const int64_t w = block * (kQ8Block >> each) + __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> each);
  const int64_t u = p.idx32 ? int64_t(div_by(p.div_groups, uint32_t(w))) : w / p.head_groups;
  Place at;
  // Wavefronts that meet in LDS are of one place, and all of its keys or all of its values (the plan sees to it), so
  // they return together.  Those of two a head go on without tokens instead: with nothing but a return here the
  // compiler waits for the page's number before it asks for the tokens (blocks of 16, NeoX: 52.9 us, not 49.1).
  const bool some = u < p.places && find_place(p, u, &at);
  if (!some && p.lanes != 128) return;
  if (!some) at = Place();
  // the first half of a place's wavefronts takes keys, the second values
  int32_t group = int32_t(w - u * p.head_groups);
  const bool keys = group < p.head_groups / 2;
  if (!keys) group -= p.head_groups / 2;
  int32_t head = group;
  if (p.lanes < 64)
    head = group * (64 >> p.lanes_log2) + ((int32_t(threadIdx.x) & 63) >> p.lanes_log2);
  if (head >= p.heads || !some) head = -1;
  if (keys)
    append_block<T, V, NEOX, E4M3, true>(p, p.kv[0], at, head);
  else
    append_block<T, V, NEOX, E4M3, false>(p, p.kv[1], at, head);
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
  // a launch has fewer than 2^32 threads
  const int64_t blocks = plan.kv_blocks + plan.query_blocks, most = int64_t(1) << 23;
  for (; plan.first_block < blocks; plan.first_block += most) {
    const int64_t n = std::min(blocks - plan.first_block, most);
    const int rc = launch_kernel(fn, dim3(uint32_t(n)), kQ8Block, 0, stream, &plan);
    if (rc != ROPE_OK) return rc;
  }
  return ROPE_OK;
}
