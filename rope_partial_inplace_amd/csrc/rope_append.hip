// rope_append.hip -- rotating a batch's new keys by position and appending keys and values to a
// paged cache, the queries rotated by the same launch (gfx950).
//
// For token t with table row [c | s] = cos_sin_cache[positions[t]], every query and key head has
// its slice [start, start + rd) rotated, pair by pair:  o1 = x1 c - x2 s,  o2 = x2 c + x1 s
// (NeoX pairs lie rd/2 apart, GPT-J pairs side by side); the rest of a head and the values are
// copied bit for bit.  Keys and values go to slot slots[t] of the cache: page slot / pageSize,
// row slot % pageSize.
//
// A few flops for every 4 bytes moved: bound by HBM.  One lane carries one 16-byte vector (two
// for a NeoX pair), so nothing is staged and a wavefront's accesses are runs of whole lines; all
// of a token's groups go into one launch because a decoding step's batch is bound by launch
// latency (64 tokens of 32 + 8 + 8 heads: one launch in place of two or three).
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

constexpr int kAppendBlock = 256;

__device__ inline uint32_t div_by(const FastDiv &f, uint32_t n) {
  const uint32_t t = __umulhi(f.m, n);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}

// V elements of a row as floats, and back (one 16-byte access, or one element).
template <typename T, int V>
__device__ inline void load_row(const T *p, float *f) {
  if constexpr (V == 1) {
    f[0] = Io<T>::load1(p, 0);
  } else {
    Io<T>::unpack(*reinterpret_cast<const uint4 *>(p), f);
  }
}

template <typename T, int V>
__device__ inline void store_row(T *p, const float *f) {
  if constexpr (V == 1) {
    Io<T>::store1(p, 0, f[0]);
  } else {
    *reinterpret_cast<uint4 *>(p) = Io<T>::pack(f);
  }
}

// The V/2 cos (or sin) values of a GPT-J vector: 8 bytes.
template <typename T, int V>
__device__ inline void load_half(const T *p, float *f) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  Io<T>::word_to_floats(w.x, f);
  Io<T>::word_to_floats(w.y, f + Io<T>::kPerWord);
}

template <typename T, int V, bool NEOX>
__global__ __launch_bounds__(kAppendBlock) void append_paged_kernel(AppendPlan p) {
  const int64_t stride = int64_t(gridDim.x) * kAppendBlock;
  for (int64_t it = int64_t(blockIdx.x) * kAppendBlock + threadIdx.x; it < p.items; it += stride) {
    int64_t t;
    uint32_t i;  // item of the token
    if (p.idx32) {
      const uint32_t q = div_by(p.div_token, uint32_t(it));
      t = q;
      i = uint32_t(it) - q * p.items_per_token;
    } else {
      t = it / p.items_per_token;
      i = uint32_t(it - t * p.items_per_token);
    }
    const int64_t pos_raw = p.positions[t * p.pos_stride];
    // the row group the item belongs to (fields picked apart: the plan is read with scalar loads)
    const uint32_t n0 = p.rows[0].total, n01 = n0 + p.rows[1].total;
    const bool is_q = i < n0, is_k = !is_q && i < n01;
    const AppendRows &r = is_q ? p.rows[0] : is_k ? p.rows[1] : p.rows[2];
    const uint32_t j = i - (is_q ? 0u : is_k ? n0 : n01);
    const uint32_t h = div_by(r.div_items, j), u = j - h * r.items;
    const T *in = static_cast<const T *>(r.in) + t * r.in_tok + int64_t(h) * r.in_head;
    T *out = static_cast<T *>(r.out) + int64_t(h) * r.out_head;
    bool keep = true;
    if (is_q) {
      out += t * r.out_tok;
    } else {
      // a slot outside the cache (negative: a padding token) takes nothing
      const int64_t s = p.slots[t * p.slot_stride];
      keep = s >= 0 && s < p.num_slots;
      if (p.linear) {
        out += s * r.out_tok;
      } else {
        const int64_t page = p.page32 ? int64_t(div_by(p.div_page, uint32_t(s))) : s / p.page_size;
        out += page * r.out_page + (s - page * p.page_size) * r.out_tok;
      }
    }
    if (!keep) continue;
    if (u >= r.rot_items) {  // outside the slice: copied bit for bit
      int64_t e = int64_t(u - r.rot_items) * V;
      if (e >= r.rot_start && r.rot_items != 0) e += 2 * p.half;
      if constexpr (V == 1) {
        reinterpret_cast<typename Io<T>::raw *>(out)[e] =
            reinterpret_cast<const typename Io<T>::raw *>(in)[e];
      } else {
        *reinterpret_cast<uint4 *>(out + e) = *reinterpret_cast<const uint4 *>(in + e);
      }
      continue;
    }
    const int64_t pos = min(max(pos_raw, int64_t(0)), p.max_seq - 1);
    const T *row = static_cast<const T *>(p.table) + pos * p.table_stride;
    if constexpr (NEOX) {
      const int64_t e = r.rot_start + int64_t(u) * V;
      float a[V], b[V], c[V], s[V], x[V], y[V];
      load_row<T, V>(in + e, a);
      load_row<T, V>(in + e + p.half, b);
      load_row<T, V>(row + int64_t(u) * V, c);
      load_row<T, V>(row + p.half + int64_t(u) * V, s);
#pragma unroll
      for (int m = 0; m < V; ++m) {
        x[m] = a[m] * c[m] - b[m] * s[m];
        y[m] = b[m] * c[m] + a[m] * s[m];
      }
      store_row<T, V>(out + e, x);
      store_row<T, V>(out + e + p.half, y);
    } else if constexpr (V == 1) {
      const int64_t e = r.rot_start + 2 * int64_t(u);
      const float a = Io<T>::load1(in, e), b = Io<T>::load1(in, e + 1);
      const float c = Io<T>::load1(row, u), s = Io<T>::load1(row, p.half + int64_t(u));
      Io<T>::store1(out, e, a * c - b * s);
      Io<T>::store1(out, e + 1, b * c + a * s);
    } else {
      const int64_t e = r.rot_start + int64_t(u) * V;
      float a[V], c[V / 2], s[V / 2], x[V];
      load_row<T, V>(in + e, a);
      load_half<T, V>(row + int64_t(u) * (V / 2), c);
      load_half<T, V>(row + p.half + int64_t(u) * (V / 2), s);
#pragma unroll
      for (int m = 0; m < V / 2; ++m) {
        x[2 * m] = a[2 * m] * c[m] - a[2 * m + 1] * s[m];
        x[2 * m + 1] = a[2 * m + 1] * c[m] + a[2 * m] * s[m];
      }
      store_row<T, V>(out + e, x);
    }
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
  int64_t blocks = (plan.items + kAppendBlock - 1) / kAppendBlock;
  if (blocks > kMaxGrid) blocks = kMaxGrid;
  return launch_kernel(fn, dim3(uint32_t(blocks)), kAppendBlock, 0, stream, &plan);
}
