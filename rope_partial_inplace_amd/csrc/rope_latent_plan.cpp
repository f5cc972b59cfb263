// rope_latent_plan.cpp -- argument checks and launch plans of the latent attention operators
// (host only; every refusal happens before any HIP call).
#include "rope_latent_plan.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <limits>

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

// Rows of an item: as many as a sequence's (token, head) rows fill, 32, 64 or 128.  More rows read
// the cache fewer times and spread a tile's LDS reads over more products; fewer leave smaller parts
// to join.  Microseconds, bfloat16, latent_dim 512, for items of 32 | 64 | 128 rows:
//   6 sequences of 60000 to 131072 tokens, 128 heads   295 | 210 | 190
//   4 sequences of 16000 / 4000 tokens, 128 heads      59 / 29 | 47 / 31 | 45 / 30
//   8 sequences of 16000 / 4000 tokens, 64 heads       59 / 29 | 48 / 31 | -
//   64 sequences of 200 to 9000 tokens, 32 heads       52 | 54 | -
// Short contexts lose a little by it (24 sequences of 1200 tokens with 48 rows take 26.0 us with
// 32, 28.3 with 64; of 5000 tokens 53.1 and 45.9), but their lengths are not known here.
int64_t paged_rows(int64_t tokens, int64_t heads, int64_t sequences) {
  const int64_t n = std::max<int64_t>(sequences, 1);
  const int64_t rows = heads * (tokens / n + (tokens % n != 0));
  return rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

// |scale| * log2(e), and whether the scale is negative.  Not 0, which would turn a masked score of
// -infinity into a NaN: the smallest positive number makes no difference beside scores of any size.
// False where the product is beyond float32.
bool set_scale(double scale, float *scale_log2, bool *negative) {
  const double x = std::fabs(scale) * kLog2e;
  if (!(x <= std::numeric_limits<float>::max())) return false;  // infinite and NaN too
  *scale_log2 = std::max(float(x), std::numeric_limits<float>::denorm_min());
  *negative = scale < 0;
  return true;
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

}  // namespace

int64_t paged_workspace(int64_t tokens, int64_t heads, int64_t latent, int64_t sequences) {
  // sizes that the call has no work for, or refuses
  if (tokens <= 0 || heads <= 0 || latent <= 0 || sequences <= 0) return 0;
  if (tokens >= kIndexLimit || heads >= kIndexLimit || latent > 512) return 0;
  const int64_t rows = std::min<int64_t>(64, paged_rows(tokens, heads, sequences));
  return up(kPagedGroups * 2 * kJoinWords * 4, 256) + up(2 * kPagedGroups * rows * 8, 256) +
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
  if (!set_scale(scale, &plan->scale_log2, &plan->negative))
    return reject(err, ROPE_ERR_PARAM_INVALID, "scale must be finite, and below 2^127 in size");
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
  if (items > 0x7fffffff / (steps + 8))
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many query rows and pages for one call");
  const int64_t most = kPagedGroups / p.cluster;
  p.clusters = int32_t(
      steps >= most ? most : std::min<int64_t>(most, up(items * steps, kXcds)));
  char *w = static_cast<char *>(workspace);
  p.joins = reinterpret_cast<int32_t *>(w);
  w += up(kPagedGroups * 2 * kJoinWords * 4, 256);
  p.stats = reinterpret_cast<float *>(w);
  w += up(2 * kPagedGroups * rows * 8, 256);
  p.parts = reinterpret_cast<float *>(w);
  return ROPE_OK;
}

// ---- expanded form --------------------------------------------------------------------------

namespace {

// Whether a launch of whole rounds of the XCDs can have `groups` workgroups of `threads`.
bool launch_fits(int64_t groups, int64_t threads) {
  return up(groups, kXcds) * threads < kLaunchThreads;
}

// The rows of a tile of 64 tokens are addressed by 32-bit byte offsets from its first.
bool token_stride_fits(const rope_tensor *t) {
  return t->shape[0] <= 1 || t->stride[0] * bytes_of(t->dtype) < (int64_t(1) << 25);
}

int64_t tiles_bound(int64_t tokens, int64_t sequences, int64_t each, bool offsets) {
  return offsets ? tokens / kExpandedRows + sequences
                 : sequences * ((each + kExpandedRows - 1) / kExpandedRows);
}

}  // namespace

int64_t expanded_workspace(int64_t query_tokens, int64_t key_tokens, int64_t heads) {
  // sizes that the call has no sums for, or refuses
  if (query_tokens < 0 || key_tokens < 0 || heads <= 0) return 0;
  if (query_tokens >= kIndexLimit || key_tokens >= kIndexLimit || heads >= kIndexLimit ||
      std::max(query_tokens, key_tokens) * heads >= int64_t(1) << 40)
    return 0;
  return up(query_tokens * heads * 4, 256) + key_tokens * heads * kLatentRope * 4;
}

int plan_expanded(const rope_tensor *query, const rope_tensor *key, const rope_tensor *key_rope,
                  const rope_tensor *value, const rope_tensor *query_offsets,
                  const rope_tensor *key_offsets, int64_t num_sequences, double scale, int causal,
                  const rope_tensor *out, const rope_tensor *lse, ExpandedPlan *plan,
                  std::string *err) {
  *plan = ExpandedPlan();
  for (const rope_tensor *t : {query, key, key_rope, value, out, lse})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  if ((query_offsets == nullptr) != (key_offsets == nullptr))
    return reject(err, ROPE_ERR_PARAM_NULLPTR, "query_offsets and key_offsets come together");
  const int st =
      common_checks({query, key, key_rope, value, query_offsets, key_offsets, out, lse}, err);
  if (st != ROPE_OK) return st;
  const rope_dtype dt = query->dtype;
  if (!half_precision(dt))
    return reject(err, ROPE_ERR_PARAM_INVALID, "query must be float16 or bfloat16");
  for (const rope_tensor *t : {key, key_rope, value, out})
    if (t->dtype != dt)
      return reject(err, ROPE_ERR_PARAM_INVALID, "key, value and out must share query's dtype");
  if (lse->dtype != ROPE_F32) return reject(err, ROPE_ERR_PARAM_INVALID, "lse must be float32");
  for (const rope_tensor *t : {query_offsets, key_offsets})
    if (t != nullptr && !is_i64_vector(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "offsets must be int64 [B + 1]");
  if (query->ndim != 3 || key->ndim != 3 || key_rope->ndim != 2 || value->ndim != 3 ||
      out->ndim != 3 || lse->ndim != 2)
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "query, key, value and out must be 3-D, key_rope and lse 2-D");
  const int64_t Tq = query->shape[0], H = query->shape[1], Tk = key->shape[0];
  const int64_t dim = key->shape[2];
  if (dim != 64 && dim != 128)
    return reject(err, ROPE_ERR_PARAM_INVALID, "key heads must be 64 or 128 wide");
  if (query->shape[2] != dim + kLatentRope || key_rope->shape[1] != kLatentRope ||
      value->shape[2] != dim)
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "widths: query key + 64, key_rope 64, value that of key");
  if (key->shape[1] != H || value->shape[1] != H || key_rope->shape[0] != Tk ||
      value->shape[0] != Tk)
    return reject(err, ROPE_ERR_PARAM_INVALID, "heads or key tokens differ");
  if (out->shape[0] != Tq || out->shape[1] != H || out->shape[2] != dim || lse->shape[0] != Tq ||
      lse->shape[1] != H)
    return reject(err, ROPE_ERR_PARAM_INVALID, "out must be [Tq, heads, dim], lse [Tq, heads]");
  int64_t B = num_sequences;
  if (query_offsets != nullptr) {
    B = query_offsets->shape[0] - 1;
    if (B < 0 || key_offsets->shape[0] != B + 1 || (num_sequences != 0 && num_sequences != B))
      return reject(err, ROPE_ERR_PARAM_INVALID,
                    "offsets must be [B + 1] each, num_sequences B or 0 with them");
  } else if (B < 1 || Tq % B != 0 || Tk % B != 0) {
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "without offsets num_sequences must divide both token counts");
  }
  if (!set_scale(scale, &plan->scale_log2, &plan->negative))
    return reject(err, ROPE_ERR_PARAM_INVALID, "scale must be finite, and below 2^127 in size");
  if (Tq >= kIndexLimit || Tk >= kIndexLimit || H >= kIndexLimit || B >= kIndexLimit)
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many tokens, heads or sequences");
  for (const rope_tensor *t : {query, key, key_rope, value})
    if (!unit_inner(t) || !rows_aligned16(t))
      return reject(err, ROPE_ERR_PARAM_INVALID,
                    "rows need unit inner stride and 16-byte aligned starts");
  for (const rope_tensor *t : {query, key, key_rope, value})
    if (!token_stride_fits(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "a token's stride is 32 MiB or more");
  if (!row_major(out) || !row_major(lse) || !aligned16(out->data))
    return reject(err, ROPE_ERR_PARAM_INVALID, "out and lse must be contiguous, out 16-byte aligned");
  ExpandedPlan &p = *plan;
  p.q_tiles = tiles_bound(Tq, B, query_offsets != nullptr ? 0 : Tq / std::max<int64_t>(B, 1),
                          query_offsets != nullptr);
  p.k_tiles = tiles_bound(Tk, B, query_offsets != nullptr ? 0 : Tk / std::max<int64_t>(B, 1),
                          query_offsets != nullptr);
  if (H * std::max(p.q_tiles, p.k_tiles) > 0x7fffff00 ||
      !launch_fits(H * p.q_tiles, kExpandedThreads))
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many tokens and heads for one launch");
  if (!outputs_apart({out, lse}, {query, key, key_rope, value, query_offsets, key_offsets}))
    return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
  p.noop = Tq == 0 || H == 0 || B == 0;
  p.dt = dt;
  p.causal = causal != 0;
  p.q = query->data;
  p.q_tok = query->stride[0];
  p.q_head = query->stride[1];
  p.k = key->data;
  p.k_tok = key->stride[0];
  p.k_head = key->stride[1];
  p.kr = key_rope->data;
  p.kr_tok = key_rope->stride[0];
  p.v = value->data;
  p.v_tok = value->stride[0];
  p.v_head = value->stride[1];
  if (query_offsets != nullptr) {
    p.q_off = static_cast<const int64_t *>(query_offsets->data);
    p.k_off = static_cast<const int64_t *>(key_offsets->data);
    p.q_off_stride = query_offsets->stride[0];
    p.k_off_stride = key_offsets->stride[0];
  } else {
    p.q_each = Tq / B;
    p.k_each = Tk / B;
  }
  p.Tq = Tq;
  p.Tk = Tk;
  p.B = B;
  p.heads = int32_t(H);
  p.dim = int32_t(dim);
  p.scale = float(scale);
  p.out = out->data;
  p.lse = static_cast<float *>(lse->data);
  return ROPE_OK;
}

int plan_expanded_backward(const rope_tensor *grad, const rope_tensor *query,
                           const rope_tensor *key, const rope_tensor *key_rope,
                           const rope_tensor *value, const rope_tensor *out,
                           const rope_tensor *lse, const rope_tensor *query_offsets,
                           const rope_tensor *key_offsets, int64_t num_sequences, double scale,
                           int causal, const rope_tensor *dquery, const rope_tensor *dkey,
                           const rope_tensor *dkey_rope, const rope_tensor *dvalue,
                           void *workspace, int64_t workspace_bytes, ExpandedPlan *plan,
                           std::string *err) {
  for (const rope_tensor *t : {grad, dquery, dkey, dkey_rope, dvalue})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  int st = plan_expanded(query, key, key_rope, value, query_offsets, key_offsets, num_sequences,
                         scale, causal, out, lse, plan, err);
  if (st != ROPE_OK) return st;
  st = common_checks({grad, dquery, dkey, dkey_rope, dvalue}, err);
  if (st != ROPE_OK) return st;
  const rope_tensor *outs[4] = {dquery, dkey, dkey_rope, dvalue};
  const rope_tensor *like[4] = {query, key, key_rope, value};
  for (int i = 0; i < 4; ++i) {
    if (outs[i]->dtype != query->dtype || outs[i]->ndim != like[i]->ndim)
      return reject(err, ROPE_ERR_PARAM_INVALID, "gradients must have their input's dtype and rank");
    for (int d = 0; d < like[i]->ndim; ++d)
      if (outs[i]->shape[d] != like[i]->shape[d])
        return reject(err, ROPE_ERR_PARAM_INVALID, "gradients must have their input's shape");
    if (!row_major(outs[i]) || !aligned16(outs[i]->data))
      return reject(err, ROPE_ERR_PARAM_INVALID, "gradients must be contiguous, 16-byte aligned");
  }
  if (grad->dtype != query->dtype || grad->ndim != 3)
    return reject(err, ROPE_ERR_PARAM_INVALID, "grad must have out's dtype and shape");
  for (int d = 0; d < 3; ++d)
    if (grad->shape[d] != out->shape[d])
      return reject(err, ROPE_ERR_PARAM_INVALID, "grad must have out's dtype and shape");
  if (!unit_inner(grad) || !rows_aligned16(grad) || !token_stride_fits(grad))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "rows need unit inner stride, 16-byte aligned starts, token strides below 32 MiB");
  if (!outputs_apart({dquery, dkey, dkey_rope, dvalue},
                     {grad, query, key, key_rope, value, out, lse, query_offsets, key_offsets}))
    return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
  ExpandedPlan &p = *plan;
  // without heads or sequences there are still zero gradients to write
  p.noop = p.Tq == 0 && p.Tk == 0;
  if (p.noop) return ROPE_OK;
  // the kernels of dk and dv, and of dkey_rope: refused before the first of them is enqueued
  if (!launch_fits(p.heads * p.k_tiles, kKeyThreads) ||
      !launch_fits((p.Tk + p.Tq) * 16 / kExpandedThreads + 1, kExpandedThreads))
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many tokens and heads for one launch");
  const int64_t need = expanded_workspace(p.Tq, p.Tk, p.heads);
  if (need > 0 && workspace == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "workspace is NULL");
  if (workspace_bytes < need || !aligned16(workspace))
    return reject(err, ROPE_ERR_PARAM_INVALID, "workspace too small or not 16-byte aligned");
  for (const rope_tensor *t : {grad, query, key, key_rope, value, out, lse, query_offsets,
                               key_offsets, dquery, dkey, dkey_rope, dvalue})
    if (touches(workspace, need, t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "workspace overlaps a tensor");
  p.grad = grad->data;
  p.g_tok = grad->stride[0];
  p.g_head = grad->stride[1];
  p.dq = dquery->data;
  p.dk = dkey->data;
  p.dkr = dkey_rope->data;
  p.dv = dvalue->data;
  p.delta = static_cast<float *>(workspace);
  p.dkr_part = reinterpret_cast<float *>(static_cast<char *>(workspace) + up(p.Tq * p.heads * 4, 256));
  return ROPE_OK;
}

}  // namespace ropeamd
