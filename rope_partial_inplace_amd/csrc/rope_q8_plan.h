// rope_q8_plan.h -- launch plans of the append to and the attention over a paged cache in 8 bits
// (library-internal).
#pragma once

#include <cstdint>
#include <string>

#include "rope.h"
#include "rope_append_plan.h"
#include "rope_plan.h"

namespace ropeamd {

// Where sequences lie: lengths, pages and the rows of a packed batch (offsets NULL: `each` rows).
struct Sequences {
  const int64_t *table = nullptr, *lens = nullptr, *offsets = nullptr;
  int64_t table_seq = 0, table_page = 0, len_stride = 0, off_stride = 0;
  int64_t num_pages = 0, max_pages = 0, page_size = 1;
  int64_t T = 0, B = 0, each = 0;
  FastDiv div_page;
};

// ---- append -----------------------------------------------------------------------------------
// Keys or values: where their rows, codes and scales lie.
struct Q8Rows {
  const void *in = nullptr;
  int64_t in_tok = 0, in_head = 0;  // elements
  uint8_t *codes = nullptr;
  int64_t page = 0, row = 0, head = 0;  // strides of the codes (bytes)
  float *scales = nullptr;
  int64_t s_page = 0, s_block = 0, s_head = 0;
  int32_t dim = 0;
  int32_t rot_start = 0;
  uint32_t rot_items = 0;  // rotated items of a row, in the order of AppendRows
  uint32_t items = 0;
  bool wide_rows = false;  // code rows split into aligned 16-byte pieces
  // A row's items fit the threads of a block, 2^row_log2 of them.  Such rows are loaded with no look at their
  // items, so it is false where there are none.
  bool side_by_side = false;
  int32_t row_log2 = 0;
  FastDiv div_items;
};

struct AppendQ8Plan {
  rope_dtype dt = ROPE_F32;
  bool neox = true, vector_io = false, noop = false, e4m3 = false;
  bool idx32 = true;  // query items and wavefronts are numbered in 32 bits
  // A wavefront (for long blocks two or four) takes one place of tokens (one block of a sequence) and several
  // of its heads.
  // Places are numbered so that their sequence can be found from the offsets alone: by token, where
  // all but a block's first new token have nothing to do, or, fewer for long appends, from
  // offsets[b] / block + 2 b on, which is enough for the blocks a sequence's tokens can touch.
  bool by_token = true;
  int32_t lanes = 64;      // threads of a head's block: a power of two from 4 to 256
  int32_t lanes_log2 = 0;
  int64_t places = 0, kv_blocks = 0, query_blocks = 0;
  int64_t first_block = 0;  // of a launch
  int64_t query_heads = 0;
  int32_t head_groups = 2;  // wavefronts of a place: half of them for keys, half for values
  int32_t heads = 0;
  int32_t block = 1;  // tokens of a scale
  int32_t half = 0;   // rotaryDim / 2
  const int64_t *positions = nullptr;
  int64_t pos_stride = 0;
  const void *table = nullptr;  // cos and sin
  int64_t table_stride = 0, max_seq = 0;
  Sequences seq;
  FastDiv div_groups, div_block;
  Q8Rows kv[2];
  AppendRows query;
};

constexpr int kQ8Block = 256;
// Query heads of a thread, whose items are all under way at once: with the pairs' two parts apart (NeoX) two
// heads are as many loads as four with them together.
constexpr int query_heads_of(bool neox) { return neox ? 2 : 4; }
constexpr int kQ8Held = 32;  // elements that a thread holds

int plan_append_q8(const rope_tensor *positions, const rope_tensor *query, const rope_tensor *key,
                   const rope_tensor *value, const rope_tensor *cos_sin_cache,
                   const rope_tensor *page_table, const rope_tensor *seq_lens,
                   const rope_tensor *token_offsets, int64_t query_rot_start,
                   int64_t key_rot_start, int is_neox_style, const rope_tensor *query_out,
                   const rope_tensor *key_cache, const rope_tensor *value_cache,
                   const rope_tensor *key_scales, const rope_tensor *value_scales,
                   AppendQ8Plan *plan, std::string *err);

// ---- attention --------------------------------------------------------------------------------
// Wavefronts of a SIMD for heads of `width` and `tiles` 16-row tiles; a call has as many workgroups as the card
// then holds, 256 compute units at a time.  Two, where the registers allow three (heads of 128, one tile): what is
// under way is enough, and fewer streams at a time reach more of HBM's rate (64 decoding sequences 70.5 -> 67
// us, six of 60-131k tokens 289 -> 281).
constexpr int q8_waves(int width, int tiles) {
  return width == 64 ? 3 : width == 128 || tiles == 1 ? 2 : 1;
}
constexpr int64_t kQ8ManyRows = 128;  // rows of a workgroup where there are many
constexpr int kQ8JoinWords = 8;
// Cached tokens that a workgroup takes at a time: 32 of each of the wavefronts of a head, of which there are
// 4 >> heads_log2; 64, or 32, where there are many rows.
constexpr int q8_step_log2(int64_t rows, int64_t width, int heads_log2) {
  return rows == kQ8ManyRows ? (width == 256 ? 5 : 6) : 7 - heads_log2;
}

// Keys or values of the cache.
struct Q8Cache {
  const uint8_t *codes = nullptr;
  int64_t page = 0, head = 0;  // bytes
  int32_t row = 0;
  const float *scales = nullptr;
  int64_t s_page = 0, s_block = 0, s_head = 0;
};

struct AttnQ8Plan {
  rope_dtype dt = ROPE_BF16;
  bool e4m3 = false, noop = false;
  int32_t mode = 0;  // 2: pages of whole runs of 16 tokens and scales of whole runs of 4; 1: such pages
  const void *q = nullptr;
  int64_t q_tok = 0, q_head = 0;
  Q8Cache k, v;
  Sequences seq;
  int32_t heads = 0, kv_heads = 0, group = 1, head_size = 0, block = 1;
  FastDiv div_group, div_block;
  float scale_log2 = 0;
  int32_t rows = 16;   // query rows of a workgroup
  int32_t groups = 0;  // workgroups
  // Wavefronts of a workgroup take different key heads of the same tokens (sets of 2 or 4) where those lie
  // side by side: 128 bytes of every token, 1 KB apart, are no good way through HBM, and with a scale for
  // each token the lines of scales are shared, too (six sequences of 60-131k tokens of 8 heads of 128: 331 us
  // with sets of 1, 300 with 2, 281 with 4; 64 of 9000, heads of 64: 202 -> 134).  Caches that keep a head's tokens
  // together have sets of 1 (64 of 9000, heads of 128: 212 us, with 4: 218).
  int32_t abreast = 1, abreast_log2 = 0, head_sets = 0;
  int32_t step_log2 = 7;  // cached tokens of a workgroup at a time
  bool small = false;  // the items' cost (in tokens' steps) fits 31 bits, whatever the lengths
  void *out = nullptr;
  float *lse = nullptr;
  // workspace: for a workgroup's first and last part the record of the item it is part of, its
  // rows' maxima and sums, and its unnormalised outputs
  int64_t *joins = nullptr;  // [groups][2][kQ8JoinWords]
  float *stats = nullptr;    // [groups][2][abreast][rows][2]
  float *parts = nullptr;    // [groups][2][abreast][rows][head_size]
};

int64_t attention_q8_workspace(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_size,
                               int64_t sequences);

int plan_attention_q8(const rope_tensor *query, const rope_tensor *key_cache,
                      const rope_tensor *value_cache, const rope_tensor *key_scales,
                      const rope_tensor *value_scales, const rope_tensor *page_table,
                      const rope_tensor *seq_lens, const rope_tensor *query_offsets, double scale,
                      const rope_tensor *out, const rope_tensor *lse, void *workspace,
                      int64_t workspace_bytes, AttnQ8Plan *plan, std::string *err);

}  // namespace ropeamd
