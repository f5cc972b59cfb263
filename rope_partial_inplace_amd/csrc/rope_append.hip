// rope_append.hip -- rotating a batch's new keys by position and appending keys and values to a
// paged cache, the queries rotated by the same launch (gfx950).
//
// For token t with table row [c | s] = cos_sin_cache[positions[t]], every query and key head has
// its slice [start, start + rd) rotated, pair by pair:  o1 = x1 c - x2 s,  o2 = x2 c + x1 s
// (NeoX pairs lie rd/2 apart, GPT-J pairs side by side); the rest of a head and the values are
// copied bit for bit.  Keys and values go to slot slots[t] of the cache: page slot / pageSize,
// row slot % pageSize.
//
// A few flops for every 4 bytes moved: bound by HBM.  An item is one 16-byte vector (two for a
// NeoX pair), so nothing is staged and a wavefront's accesses are runs of whole lines; all
// of a token's groups go into one launch because a decoding step's batch is bound by launch
// latency (64 tokens of 32 + 8 + 8 heads: one launch in place of two or three).
//
// Measured, from HBM (seven sets of inputs in turn): 8192 tokens of 32 + 8 + 8 heads of 128, float16,
// half of each head rotated (203 MB): 46 us, 4.4 TB/s; the same in float32 (405 MB): 82 us, 4.9 TB/s;
// 32768 latent rows of 576 with 16 query tails of 64 (211 MB): 50 us, 4.2 TB/s; a dense copy of 1 GiB
// reaches 6.8 TB/s, so a third of the time is still the kernel's.  64 tokens: 4.0 us, its launch and
// three dependent reads (position, table row, slot).
//
// Rows that are not made of whole 16-byte vectors go an element (or GPT-J pair) at a time: 180 us in
// place of 46 (heads of 126), 170 in place of 50 (rows of 578).
//
// Below, times of alternatives are of calls back to back on the same inputs, which the Infinity Cache
// of 256 MB holds in part (34 us for the first of the above, 39 for the third).  A slot's page and
// row come from a 64-bit division: a 32-bit one by a multiplication, or a test for caches without
// gaps, was no faster (34.2 us each).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "rope.h"
#include "rope_append_plan.h"
#include "rope_io.h"
#include "rope_launch.h"

// The formulas are two products and one sum, each rounded to float32.
#pragma clang fp contract(off)

namespace ropeamd {
namespace {

__device__ inline uint32_t div_by(const FastDiv &f, uint32_t n) {
  const uint32_t t = __umulhi(f.m, n);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// V elements of a row, as they lie in memory: one 16-byte access, or one element.
template <typename T, int V>
struct Item {
  uint4 raw;
  __device__ void load(const T *p) { raw = *reinterpret_cast<const uint4 *>(p); }
  // streamed: what is written here is read by later launches (32768 latent rows 45.6 -> 39.0 us;
  // streamed loads were slower, 34 -> 44 us at 8192 tokens of 48 heads)
  __device__ void store(T *p) const {
    const u32x4 v = {raw.x, raw.y, raw.z, raw.w};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
  }
  __device__ void floats(float *f) const { Io<T>::unpack(raw, f); }
  __device__ void set(const float *f) { raw = Io<T>::pack(f); }
  // the V/2 cos (or sin) values of a GPT-J vector: 8 bytes
  __device__ void load_half(const T *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    raw.x = w.x;
    raw.y = w.y;
  }
  __device__ void half_floats(float *f) const {
    Io<T>::word_to_floats(raw.x, f);
    Io<T>::word_to_floats(raw.y, f + Io<T>::kPerWord);
  }
};

template <typename T>
struct Item<T, 1> {
  typename Io<T>::raw raw;
  __device__ void load(const T *p) { raw = *reinterpret_cast<const typename Io<T>::raw *>(p); }
  __device__ void store(T *p) const { *reinterpret_cast<typename Io<T>::raw *>(p) = raw; }
  __device__ void floats(float *f) const { f[0] = Io<T>::from_raw(raw); }
  __device__ void set(const float *f) {
    T v;
    Io<T>::store1(&v, 0, f[0]);
    raw = __builtin_bit_cast(typename Io<T>::raw, v);
  }
};

// Workgroups are dealt to the three groups of rows one after the other (plan), so that a group's
// pointers and strides are scalars, and a lane carries one item (two: no faster at 8192 tokens of
// 48 heads, 8% slower at 32768 latent rows).
template <typename T, int V, bool NEOX>
__global__ __launch_bounds__(kAppendBlock) void append_paged_kernel(AppendPlan p) {
  const int64_t blocks0 = p.rows[0].blocks, blocks01 = blocks0 + p.rows[1].blocks;
  const int64_t all = blocks01 + p.rows[2].blocks;
  for (int64_t block = blockIdx.x; block < all; block += gridDim.x) {
    const int group = block < blocks0 ? 0 : block < blocks01 ? 1 : 2;
    const AppendRows &r = p.rows[group];
    const int64_t it = (block - (group == 0 ? 0 : group == 1 ? blocks0 : blocks01)) * kAppendBlock +
                       threadIdx.x;
    if (it >= r.all) continue;
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
    // the loads that depend on nothing first: position, slot, the row's elements
    const int64_t pos = r.rot_items != 0 ? p.positions[t * p.pos_stride] : 0;
    const int64_t slot = group != 0 ? p.slots[t * p.slot_stride] : 0;
    // an item's elements: from e on, and (pairs) from e + partner on
    const bool turn = unit < r.rot_items;
    int64_t e;
    if (turn) {
      e = r.rot_start + int64_t(unit) * (V == 1 && !NEOX ? 2 : V);
    } else {  // outside the slice
      e = int64_t(unit - r.rot_items) * V;
      if (e >= r.rot_start && r.rot_items != 0) e += 2 * p.half;
    }
    constexpr bool PAIR = NEOX || V == 1;
    const int64_t partner = NEOX ? int64_t(p.half) : int64_t(1);
    Item<T, V> x, y, c, s;
    x.load(in + e);
    if (PAIR && turn) y.load(in + e + partner);

    T *out = static_cast<T *>(r.out) + int64_t(h) * r.out_head;
    if (group == 0) {
      out += t * r.out_tok;
    } else {
      const int64_t page = slot / p.page_size;
      out += page * r.out_page + (slot - page * p.page_size) * r.out_tok;
    }
    // a slot outside the cache (negative: a padding token) takes nothing
    const bool keep = group == 0 || (slot >= 0 && slot < p.num_slots);
    if (!turn) {  // copied bit for bit
      if (keep) x.store(out + e);
      continue;
    }
    const int64_t at = min(max(pos, int64_t(0)), p.max_seq - 1);
    const T *row = static_cast<const T *>(p.table) + at * p.table_stride;
    float a[V], cv[V], sv[V], u[V];
    if constexpr (PAIR) {
      float b[V], w[V];
      c.load(row + int64_t(unit) * V);
      s.load(row + p.half + int64_t(unit) * V);
      x.floats(a);
      y.floats(b);
      c.floats(cv);
      s.floats(sv);
#pragma unroll
      for (int m = 0; m < V; ++m) {
        u[m] = a[m] * cv[m] - b[m] * sv[m];
        w[m] = b[m] * cv[m] + a[m] * sv[m];
      }
      y.set(w);
      if (keep) y.store(out + e + partner);
    } else {
      c.load_half(row + int64_t(unit) * (V / 2));
      s.load_half(row + p.half + int64_t(unit) * (V / 2));
      x.floats(a);
      c.half_floats(cv);
      s.half_floats(sv);
#pragma unroll
      for (int m = 0; m < V / 2; ++m) {
        u[2 * m] = a[2 * m] * cv[m] - a[2 * m + 1] * sv[m];
        u[2 * m + 1] = a[2 * m + 1] * cv[m] + a[2 * m] * sv[m];
      }
    }
    x.set(u);
    if (keep) x.store(out + e);
  }
}

template <typename T>
const void *pick_append(const AppendPlan &p) {
  constexpr int V = Io<T>::kPer16;
#define ROPE_KA(VV, NX) reinterpret_cast<const void *>(&append_paged_kernel<T, VV, NX>)
  if (p.vector_io) return p.neox ? ROPE_KA(V, true) : ROPE_KA(V, false);
  return p.neox ? ROPE_KA(1, true) : ROPE_KA(1, false);
#undef ROPE_KA
}

}  // namespace
}  // namespace ropeamd

using namespace ropeamd;

ROPE_API int rope_append_paged_cache(const rope_tensor *positions, const rope_tensor *slots,
                                     const rope_tensor *query, const rope_tensor *key,
                                     const rope_tensor *value, const rope_tensor *cos_sin_cache,
                                     int64_t query_rot_start, int64_t key_rot_start,
                                     int is_neox_style, const rope_tensor *query_out,
                                     const rope_tensor *key_cache, const rope_tensor *value_cache,
                                     void *stream) {
  AppendPlan plan;
  std::string err;
  const int st = plan_append(positions, slots, query, key, value, cos_sin_cache, query_rot_start,
                             key_rot_start, is_neox_style, query_out, key_cache, value_cache,
                             &plan, &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
  if (plan.noop) return ROPE_OK;
  const void *fn = plan.dt == ROPE_F32   ? pick_append<float>(plan)
                   : plan.dt == ROPE_F16 ? pick_append<_Float16>(plan)
                                         : pick_append<__bf16>(plan);
  int64_t blocks = plan.rows[0].blocks + plan.rows[1].blocks + plan.rows[2].blocks;
  if (blocks > kMaxGrid) blocks = kMaxGrid;
  return launch_kernel(fn, dim3(uint32_t(blocks)), kAppendBlock, 0, stream, &plan);
}
