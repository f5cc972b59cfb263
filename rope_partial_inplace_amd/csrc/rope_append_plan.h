// rope_append_plan.h -- launch plan of the paged-cache append (library-internal).
#pragma once

#include <cstdint>
#include <string>

#include "rope.h"
#include "rope_plan.h"

namespace ropeamd {

// One of the three groups of rows a token has: its query heads, its key heads, its value heads.
// A row of `heads` heads is cut into work items.  Rotated items come first: NeoX, a vector of
// the slice's first half with its partner rd/2 further on; GPT-J, a run of whole pairs.  Then
// the vectors outside the slice, copied bit for bit.
struct AppendRows {
  const void *in = nullptr;
  void *out = nullptr;  // query_out, or the cache's first slot
  int64_t in_tok = 0, in_head = 0;    // input strides (elements)
  int64_t out_head = 0;               // output head stride
  int64_t out_tok = 0, out_page = 0;  // query: token stride; caches: strides inside / of a page
  int32_t rot_start = 0;
  uint32_t rot_items = 0;  // rotated items of a head
  uint32_t items = 0;      // items of a head
  uint32_t total = 0;      // items of the group for one token: heads * items
  int64_t all = 0;         // items of the group for all tokens
  int64_t blocks = 0;      // workgroups
  FastDiv div_items, div_total;
};

struct AppendPlan {
  rope_dtype dt = ROPE_F32;
  bool neox = true;
  bool vector_io = false;  // 16-byte items (else one element, or one pair, at a time)
  bool noop = false;
  // item numbers of a group, and of its last lanes, fit 32 bits: decoded by multiplications
  // (64-bit divisions: 34.7 in place of 34.3 us at 8192 tokens of 48 heads, back to back)
  bool idx32 = true;
  const int64_t *positions = nullptr, *slots = nullptr;
  int64_t pos_stride = 0, slot_stride = 0;
  const void *table = nullptr;
  int64_t table_stride = 0, max_seq = 0;
  int32_t half = 0;  // rotaryDim / 2
  int64_t T = 0;
  int64_t num_slots = 0, page_size = 1;
  AppendRows rows[3];  // query, key, value (total 0: absent)
};

constexpr int kAppendBlock = 256;

int plan_append(const rope_tensor *positions, const rope_tensor *slots, const rope_tensor *query,
                const rope_tensor *key, const rope_tensor *value,
                const rope_tensor *cos_sin_cache, int64_t query_rot_start, int64_t key_rot_start,
                int is_neox_style, const rope_tensor *query_out, const rope_tensor *key_cache,
                const rope_tensor *value_cache, AppendPlan *plan, std::string *err);

}  // namespace ropeamd
