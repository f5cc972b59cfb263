// rope_latent_plan.cpp -- argument checks and launch plans of the latent attention operators
// (host only; every refusal happens before any HIP call).
#include "rope_latent_plan.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "rope_check.h"

namespace ropeamd {
namespace {

constexpr double kLog2e = 1.4426950408889634;
constexpr int64_t kIndexLimit = int64_t(1) << 30;  // token and row numbers stay well inside int32

bool half_precision(rope_dtype dt) { return dt == ROPE_F16 || dt == ROPE_BF16; }

// Checks that every operator here makes of its tensors (NULL entries are absent ones).
int common_checks(std::initializer_list<const rope_tensor *> all, std::string *err) {
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

bool is_i64_vector(const rope_tensor *t) { return t->dtype == ROPE_I64 && t->ndim == 1; }

// Outputs share no element with each other or with an input.
bool outputs_apart(std::initializer_list<const rope_tensor *> outs,
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
bool touches(const void *p, int64_t bytes, const rope_tensor *t) {
  if (t == nullptr || count(t) == 0 || bytes <= 0) return false;
  uintptr_t a, b;
  extent(t, &a, &b);
  const uintptr_t w = reinterpret_cast<uintptr_t>(p);
  return a < w + uintptr_t(bytes) && w < b;
}

// Rows of an item: as many as a sequence's (token, head) rows fill, 32, 64 or 128.
int64_t paged_rows(int64_t tokens, int64_t heads, int64_t sequences) {
  const int64_t rows = heads * ((tokens + sequences - 1) / std::max<int64_t>(sequences, 1));
  return rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

}  // namespace

int64_t paged_workspace(int64_t tokens, int64_t heads, int64_t latent, int64_t sequences) {
  if (tokens <= 0 || heads <= 0 || latent <= 0 || sequences <= 0) return 0;
  const int64_t rows = std::min<int64_t>(64, paged_rows(tokens, heads, sequences));
  return up(kPagedGroups * 16, 256) + up(2 * kPagedGroups * rows * 8, 256) +
         2 * kPagedGroups * rows * latent * 4;
}

int plan_paged(const rope_tensor *query, const rope_tensor *cache, const rope_tensor *page_table,
               const rope_tensor *seq_lens, const rope_tensor *query_offsets, int64_t latent_dim,
               double scale, const rope_tensor *out, const rope_tensor *lse, void *workspace,
               int64_t workspace_bytes, PagedPlan *plan, std::string *err) {
  *plan = PagedPlan();
  for (const rope_tensor *t : {query, cache, page_table, seq_lens, out})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  const int st = common_checks({query, cache, page_table, seq_lens, query_offsets, out, lse}, err);
  if (st != ROPE_OK) return st;

  const rope_dtype dt = query->dtype;
  if (!half_precision(dt))
    return reject(err, ROPE_ERR_PARAM_INVALID, "query must be float16 or bfloat16");
  if (cache->dtype != dt || out->dtype != dt)
    return reject(err, ROPE_ERR_PARAM_INVALID, "latent_cache and out must share query's dtype");
  if (lse != nullptr && lse->dtype != ROPE_F32)
    return reject(err, ROPE_ERR_PARAM_INVALID, "lse must be float32");
  if (!is_i64_vector(seq_lens) || page_table->dtype != ROPE_I64 || page_table->ndim != 2 ||
      (query_offsets != nullptr && !is_i64_vector(query_offsets)))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "seq_lens [B], page_table [B, maxPages], query_offsets [B + 1] must be int64");
  if (query->ndim != 3 || cache->ndim != 3 || out->ndim != 3 || (lse != nullptr && lse->ndim != 2))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "query and out must be 3-D, latent_cache 3-D, lse 2-D");
  if (latent_dim != 128 && latent_dim != 256 && latent_dim != 512)
    return reject(err, ROPE_ERR_PARAM_INVALID, "latent_dim must be 128, 256 or 512");
  const int64_t T = query->shape[0], H = query->shape[1], B = seq_lens->shape[0];
  if (query->shape[2] != latent_dim + kLatentRope || cache->shape[2] != latent_dim + kLatentRope)
    return reject(err, ROPE_ERR_PARAM_INVALID, "query and cache rows must be latent_dim + 64 wide");
  if (out->shape[0] != T || out->shape[1] != H || out->shape[2] != latent_dim ||
      (lse != nullptr && (lse->shape[0] != T || lse->shape[1] != H)))
    return reject(err, ROPE_ERR_PARAM_INVALID, "out must be [T, heads, latent_dim], lse [T, heads]");
  if (page_table->shape[0] != B)
    return reject(err, ROPE_ERR_PARAM_INVALID, "page_table and seq_lens differ in sequences");
  if (query_offsets != nullptr ? query_offsets->shape[0] != B + 1 : (B == 0 ? T != 0 : T % B != 0))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "query_offsets must be [B + 1]; without it every sequence has T / B queries");
  if (!std::isfinite(scale)) return reject(err, ROPE_ERR_PARAM_INVALID, "scale must be finite");
  if (T >= kIndexLimit || H >= kIndexLimit || T * H >= kIndexLimit || B >= kIndexLimit)
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many query rows");
  if (page_table->shape[1] >= kIndexLimit || cache->shape[1] >= kIndexLimit ||
      page_table->shape[1] * cache->shape[1] >= kIndexLimit || cache->shape[0] >= kIndexLimit)
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many pages or tokens per sequence");
  if (!unit_inner(query) || !unit_inner(cache) || !rows_aligned16(query) || !rows_aligned16(cache))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "query and cache rows need unit inner stride and 16-byte aligned starts");
  if (!row_major(out) || (lse != nullptr && !row_major(lse)))
    return reject(err, ROPE_ERR_PARAM_INVALID, "out and lse must be contiguous");
  if (!aligned16(out->data)) return reject(err, ROPE_ERR_PARAM_INVALID, "out must be 16-byte aligned");
  if (T == 0 || H == 0 || B == 0) {
    plan->noop = true;
    return ROPE_OK;
  }
  if (!outputs_apart({out, lse}, {query, cache, page_table, seq_lens, query_offsets}))
    return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
  const int64_t need = paged_workspace(T, H, latent_dim, B);
  if (workspace == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "workspace is NULL");
  if (workspace_bytes < need || !aligned16(workspace))
    return reject(err, ROPE_ERR_PARAM_INVALID, "workspace too small or not 16-byte aligned");
  for (const rope_tensor *t : {query, cache, page_table, seq_lens, query_offsets, out, lse})
    if (touches(workspace, need, t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "workspace overlaps a tensor");

  PagedPlan &p = *plan;
  p.dt = dt;
  p.q = query->data;
  p.q_tok = query->stride[0];
  p.q_head = query->stride[1];
  p.cache = cache->data;
  p.c_page = cache->stride[0];
  p.c_row = cache->stride[1];
  p.table = static_cast<const int64_t *>(page_table->data);
  p.table_seq = page_table->stride[0];
  p.table_page = page_table->stride[1];
  p.lens = static_cast<const int64_t *>(seq_lens->data);
  p.len_stride = seq_lens->stride[0];
  if (query_offsets != nullptr) {
    p.offsets = static_cast<const int64_t *>(query_offsets->data);
    p.off_stride = query_offsets->stride[0];
  }
  p.num_pages = cache->shape[0];
  // a cache without rows holds no token of any sequence
  p.page_size = std::max<int64_t>(cache->shape[1], 1);
  p.max_pages = p.num_pages == 0 || cache->shape[1] == 0 ? 0 : page_table->shape[1];
  p.div_page = make_fastdiv(uint32_t(p.page_size));
  p.div_heads = make_fastdiv(uint32_t(H));
  p.T = T;
  p.B = B;
  p.queries = query_offsets != nullptr ? 0 : T / B;
  p.heads = int32_t(H);
  p.latent = int32_t(latent_dim);
  p.scale_log2 = float(scale * kLog2e);
  p.out = out->data;
  p.lse = lse != nullptr ? static_cast<float *>(lse->data) : nullptr;
  const int64_t item_rows = paged_rows(T, H, B);
  const int64_t rows = std::min<int64_t>(64, item_rows);  // of a workgroup
  p.row_blocks = int32_t(rows / 32);
  p.cluster = int32_t(item_rows / rows);
  // no more clusters than steps there can be, and whole rounds of the XCDs
  const int64_t items = B + T * H / item_rows;
  const int64_t steps =
      std::max<int64_t>(1, up(p.max_pages * p.page_size, kPagedStep) / kPagedStep);
  const int64_t most = kPagedGroups / p.cluster;
  p.clusters = int32_t(
      steps >= most ? most : std::min<int64_t>(most, up(items * steps, kXcds)));
  // Parts of one item are few when there are many items, many when there is one: the fewer
  // items, the more workgroups share the joining of one.
  p.join_slices = int32_t(items <= 8 ? 32 : items <= 64 ? 16 : 8);
  char *w = static_cast<char *>(workspace);
  p.joins = reinterpret_cast<int32_t *>(w);
  w += up(kPagedGroups * 16, 256);
  p.stats = reinterpret_cast<float *>(w);
  w += up(2 * kPagedGroups * rows * 8, 256);
  p.parts = reinterpret_cast<float *>(w);
  return ROPE_OK;
}

}  // namespace ropeamd
