// rope_check.h -- checks of tensor descriptions shared by the planning sources of librope_amd.so
// (host only; library-internal).
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "rope.h"

namespace ropeamd {

inline int bytes_of(rope_dtype dt) {
  switch (dt) {
    case ROPE_F32: return 4;
    case ROPE_F16: return 2;
    case ROPE_BF16: return 2;
    case ROPE_I64: return 8;
    case ROPE_I8: return 1;
    case ROPE_E4M3: return 1;
  }
  return 0;
}

inline bool is_float(rope_dtype dt) { return dt == ROPE_F32 || dt == ROPE_F16 || dt == ROPE_BF16; }

inline bool valid_rank(const rope_tensor *t) {
  if (t->ndim < 1 || t->ndim > 4) return false;
  for (int d = 0; d < t->ndim; ++d)
    if (t->shape[d] < 0) return false;
  return true;
}

// Elements of t (saturating at INT64_MAX instead of overflowing).
inline int64_t count(const rope_tensor *t) {
  int64_t n = 1;
  for (int d = 0; d < t->ndim; ++d)
    if (__builtin_mul_overflow(n, t->shape[d], &n)) return INT64_MAX;
  return n;
}

// The element count and the offset of the furthest element are at most 2^53 (byte offsets of
// elements of up to 8 bytes stay below 2^56, far beyond any device memory), computed without
// overflow.  A descriptor outside that cannot describe real memory, and the planning
// arithmetic on it would overflow.
inline bool addressable(const rope_tensor *t) {
  constexpr int64_t kLimit = int64_t(1) << 53;
  int64_t n = 1, far = 0;
  for (int d = 0; d < t->ndim; ++d) {
    int64_t off;
    if (__builtin_mul_overflow(n, t->shape[d], &n) || n > kLimit) return false;
    if (t->shape[d] == 0) continue;
    if (__builtin_mul_overflow(t->shape[d] - 1, t->stride[d], &off) || off < -kLimit ||
        off > kLimit)
      return false;
    far += off < 0 ? -off : off;  // at most 4 * 2^53: no overflow
    if (far >= kLimit) return false;
  }
  return true;
}

// Row-major contiguity; a dimension of size 1 may have any stride, and a view with no
// elements has no layout to check (reading R12: an empty x is a successful no-op).
inline bool row_major(const rope_tensor *t) {
  if (count(t) == 0) return true;
  int64_t want = 1;
  for (int d = t->ndim - 1; d >= 0; --d) {
    if (t->shape[d] > 1 && t->stride[d] != want) return false;
    want *= t->shape[d];
  }
  return true;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int reject(std::string *err, int code, const char *why) {
  if (err) *err = why;
  return code;
}

// Bytes [first, last) an N-d view reaches (non-negative strides).
inline void extent(const rope_tensor *t, uintptr_t *first, uintptr_t *last) {
  int64_t far = 0;
  for (int d = 0; d < t->ndim; ++d) far += (t->shape[d] - 1) * t->stride[d];
  *first = reinterpret_cast<uintptr_t>(t->data);
  *last = *first + uintptr_t((far + 1) * bytes_of(t->dtype));
}

inline bool overlap(const rope_tensor *a, const rope_tensor *b) {
  uintptr_t a0, a1, b0, b1;
  extent(a, &a0, &a1);
  extent(b, &b0, &b1);
  return a0 < b1 && b0 < a1;
}

inline bool identical_view(const rope_tensor *a, const rope_tensor *b) {
  if (a->data != b->data || a->ndim != b->ndim || a->dtype != b->dtype) return false;
  for (int d = 0; d < a->ndim; ++d) {
    if (a->shape[d] != b->shape[d]) return false;
    if (a->shape[d] > 1 && a->stride[d] != b->stride[d]) return false;
  }
  return true;
}

// Whether a and b (non-negative strides, non-empty) provably share no element: their extents
// are apart, or they interleave -- modulo some stride M that divides every longer stride of
// both, each view stays inside a window of its own (query, key and value columns of one
// projection's rows; the key and value halves of one cache allocation).
inline bool disjoint(const rope_tensor *a, const rope_tensor *b) {
  if (!overlap(a, b)) return true;
  for (const rope_tensor *s : {a, b})
    for (int d = 0; d < s->ndim; ++d) {
      if (s->shape[d] <= 1 || s->stride[d] <= 0) continue;
      const int64_t M = s->stride[d] * bytes_of(s->dtype);
      int64_t window[2];
      bool fits = true;
      for (int v = 0; v < 2; ++v) {
        const rope_tensor *t = v == 0 ? a : b;
        const int64_t es = bytes_of(t->dtype);
        window[v] = es;
        for (int e = 0; e < t->ndim; ++e) {
          if (t->shape[e] <= 1) continue;
          const int64_t st = t->stride[e] * es;
          if (st % M != 0) window[v] += (t->shape[e] - 1) * st;
        }
        fits &= window[v] <= M;
      }
      if (!fits) continue;
      const uintptr_t pa = reinterpret_cast<uintptr_t>(a->data) % uintptr_t(M);
      const uintptr_t pb = reinterpret_cast<uintptr_t>(b->data) % uintptr_t(M);
      const int64_t gap = int64_t((pb + uintptr_t(M) - pa) % uintptr_t(M));
      if (window[0] <= gap && gap + window[1] <= M) return true;
    }
  return false;
}

// Whether distinct indices of t provably reach distinct elements: taken from the shortest
// stride up, each stride passes everything the shorter ones reach.
inline bool injective(const rope_tensor *t) {
  int order[4], n = 0;
  for (int d = 0; d < t->ndim; ++d)
    if (t->shape[d] > 1) order[n++] = d;
  std::sort(order, order + n, [t](int x, int y) { return t->stride[x] < t->stride[y]; });
  int64_t reach = 0;
  for (int i = 0; i < n; ++i) {
    if (t->stride[order[i]] <= reach) return false;
    reach += (t->shape[order[i]] - 1) * t->stride[order[i]];
  }
  return true;
}

inline bool non_negative_strides(const rope_tensor *t) {
  for (int d = 0; d < t->ndim; ++d)
    if (t->shape[d] > 1 && t->stride[d] < 0) return false;
  return true;
}

// Unit stride along the last dimension.
inline bool unit_inner(const rope_tensor *t) {
  return t->shape[t->ndim - 1] <= 1 || t->stride[t->ndim - 1] == 1;
}

// Every row start on a 16-byte boundary: the base and each outer stride.
inline bool rows_aligned16(const rope_tensor *t) {
  if (!aligned16(t->data)) return false;
  for (int d = 0; d + 1 < t->ndim; ++d)
    if (t->shape[d] > 1 && (t->stride[d] * bytes_of(t->dtype)) % 16 != 0) return false;
  return true;
}

// Checks that the operators on caches make of all their tensors (NULL entries are absent ones).
inline int common_checks(std::initializer_list<const rope_tensor *> all, std::string *err) {
  for (const rope_tensor *t : all)
    if (t != nullptr && valid_rank(t) && count(t) > 0 && t->data == nullptr)
      return reject(err, ROPE_ERR_PARAM_NULLPTR, "a non-empty tensor has NULL data");
  for (const rope_tensor *t : all)
    if (t != nullptr && (!valid_rank(t) || !addressable(t)))
      return reject(err, ROPE_ERR_PARAM_INVALID, "bad shape or extent");
  for (const rope_tensor *t : all)
    if (t != nullptr && !non_negative_strides(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "negative strides are not supported");
  return ROPE_OK;
}

inline bool is_i64_vector(const rope_tensor *t) { return t->dtype == ROPE_I64 && t->ndim == 1; }

// Outputs share no element with each other or with an input.
inline bool outputs_apart(std::initializer_list<const rope_tensor *> outs,
                          std::initializer_list<const rope_tensor *> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if (*o == nullptr || count(*o) == 0) continue;
    for (auto q = o + 1; q != outs.end(); ++q)
      if (*q != nullptr && count(*q) > 0 && !disjoint(*o, *q)) return false;
    for (const rope_tensor *i : ins)
      if (i != nullptr && count(i) > 0 && !disjoint(*o, i)) return false;
  }
  return true;
}

// Whether [p, p + bytes) shares memory with t's extent.
inline bool touches(const void *p, int64_t bytes, const rope_tensor *t) {
  if (t == nullptr || count(t) == 0 || bytes <= 0) return false;
  uintptr_t a, b;
  extent(t, &a, &b);
  const uintptr_t w = reinterpret_cast<uintptr_t>(p);
  return a < w + uintptr_t(bytes) && w < b;
}

}  // namespace ropeamd
