// rope_latent_plan.h -- launch plans of the latent attention operators (library-internal).
#pragma once

#include <cstdint>
#include <string>

#include "rope.h"
#include "rope_plan.h"

namespace ropeamd {

constexpr int64_t kLatentRope = 64;  // rotated tail of a latent row and of an expanded query

// ---- absorbed form over a paged cache -----------------------------------------------------
// Rows of a sequence are its (query token, head) pairs, r = token * heads + head.  A workgroup
// holds 32 * row_blocks of them, a cluster of `cluster` workgroups that many times more: the
// rows of one item.  An item walks its sequence's cache in steps of 64 tokens.  All items' steps,
// one item after another, are shared out evenly between the clusters, so that a batch of very
// different lengths loads every compute unit alike; an item that several clusters had a part of
// is joined by a second kernel.
constexpr int64_t kPagedGroups = kComputeUnits;  // one workgroup per compute unit (LDS)
constexpr int64_t kPagedStep = 64;
constexpr int64_t kJoinWords = 8;
constexpr int64_t kXcds = 8;  // consecutive workgroups go to the eight XCDs in turn

struct PagedPlan {
  rope_dtype dt = ROPE_BF16;
  bool noop = false;
  const void *q = nullptr, *cache = nullptr;
  int64_t q_tok = 0, q_head = 0, c_page = 0, c_row = 0;  // strides in elements
  const int64_t *table = nullptr, *lens = nullptr, *offsets = nullptr;
  int64_t table_seq = 0, table_page = 0, len_stride = 0, off_stride = 0;
  int64_t num_pages = 0, max_pages = 0, page_size = 1;
  FastDiv div_page, div_heads;
  int64_t T = 0, B = 0, queries = 0;  // queries: tokens of every sequence without offsets
  int32_t heads = 0, latent = 0;
  float scale_log2 = 0;   // |scale| * log2(e), above 0: the softmax runs in powers of two
  bool negative = false;  // scale < 0: the kernel turns the queries' signs
  void *out = nullptr;
  float *lse = nullptr;
  int32_t row_blocks = 1;  // 32-row blocks of a workgroup (1 or 2)
  int32_t cluster = 1;     // workgroups of an item (1 or 2), on one XCD
  int32_t clusters = 0;
  // workspace
  // [clusters][2][kJoinWords], for a cluster's first and last part: clusters that share the item
  // (0: no part), the first of them, its part, the item's first row, rows from there
  int32_t *joins = nullptr;
  float *stats = nullptr;     // [2 * groups][rows][2]: running maximum and sum of a part
  float *parts = nullptr;     // [2 * groups][latent / 4][rows][4]: unnormalised output of a part
};

int plan_paged(const rope_tensor *query, const rope_tensor *cache, const rope_tensor *page_table,
               const rope_tensor *seq_lens, const rope_tensor *query_offsets, int64_t latent_dim,
               double scale, const rope_tensor *out, const rope_tensor *lse, void *workspace,
               int64_t workspace_bytes, PagedPlan *plan, std::string *err);

// Workspace of a call, for `tokens` query tokens of `heads` heads in `sequences` sequences.
int64_t paged_workspace(int64_t tokens, int64_t heads, int64_t latent, int64_t sequences);

// ---- expanded form --------------------------------------------------------------------------
constexpr int64_t kExpandedRows = 128;  // query rows (or keys) of a workgroup
constexpr int kExpandedThreads = 256;   // of a workgroup
constexpr int kKeyThreads = 512;        // of one of dk and dv
constexpr int64_t kLaunchThreads = int64_t(1) << 32;  // a launch has fewer

struct ExpandedPlan {
  rope_dtype dt = ROPE_BF16;
  bool noop = false, causal = true;
  const void *q = nullptr, *k = nullptr, *kr = nullptr, *v = nullptr;
  int64_t q_tok = 0, q_head = 0, k_tok = 0, k_head = 0, kr_tok = 0, v_tok = 0, v_head = 0;
  const int64_t *q_off = nullptr, *k_off = nullptr;
  int64_t q_off_stride = 0, k_off_stride = 0;
  int64_t Tq = 0, Tk = 0, B = 0, q_each = 0, k_each = 0;  // *_each: tokens without offsets
  int32_t heads = 0, dim = 0;
  float scale = 0;
  float scale_log2 = 0;   // |scale| * log2(e), above 0
  bool negative = false;  // scale < 0: the forward kernel turns the queries' signs
  void *out = nullptr;
  float *lse = nullptr;
  // backward
  const void *grad = nullptr;
  int64_t g_tok = 0, g_head = 0;
  void *dq = nullptr, *dk = nullptr, *dkr = nullptr, *dv = nullptr;
  float *delta = nullptr;   // workspace [Tq][heads]
  float *dkr_part = nullptr;  // workspace [heads][Tk][64]
  int64_t q_tiles = 0, k_tiles = 0;  // upper bounds over all sequences
};

int plan_expanded(const rope_tensor *query, const rope_tensor *key, const rope_tensor *key_rope,
                  const rope_tensor *value, const rope_tensor *query_offsets,
                  const rope_tensor *key_offsets, int64_t num_sequences, double scale, int causal,
                  const rope_tensor *out, const rope_tensor *lse, ExpandedPlan *plan,
                  std::string *err);

int plan_expanded_backward(const rope_tensor *grad, const rope_tensor *query,
                           const rope_tensor *key, const rope_tensor *key_rope,
                           const rope_tensor *value, const rope_tensor *out,
                           const rope_tensor *lse, const rope_tensor *query_offsets,
                           const rope_tensor *key_offsets, int64_t num_sequences, double scale,
                           int causal, const rope_tensor *dquery, const rope_tensor *dkey,
                           const rope_tensor *dkey_rope, const rope_tensor *dvalue,
                           void *workspace, int64_t workspace_bytes, ExpandedPlan *plan,
                           std::string *err);

int64_t expanded_workspace(int64_t query_tokens, int64_t key_tokens, int64_t heads);

}  // namespace ropeamd
