// rope_append_plan.cpp -- argument checks and launch plan of the paged-cache append (host only;
// every refusal happens before any HIP call).
#include "rope_append_plan.h"

#include <algorithm>

#include "rope_check.h"

namespace ropeamd {
namespace {

// Items of one head of `dim` elements with the slice [start, start + rd) rotated (rd 0: none).
// vec > 1: 16-byte vectors; vec 1: an element, or a GPT-J pair, at a time.  `skip_copy` leaves
// out the unrotated part (an output that is its own input already holds it).
void head_items(AppendRows *r, int64_t dim, int64_t start, int64_t rd, int64_t vec, bool neox,
                bool skip_copy) {
  const int64_t pair_run = vec > 1 ? vec : 2;
  r->rot_start = int32_t(start);
  r->rot_items = uint32_t(neox ? rd / 2 / vec : rd / pair_run);
  r->items = r->rot_items + (skip_copy ? 0u : uint32_t((dim - rd) / vec));
}

}  // namespace

int plan_append(const rope_tensor *positions, const rope_tensor *slots, const rope_tensor *query,
                const rope_tensor *key, const rope_tensor *value, const rope_tensor *table,
                int64_t query_rot_start, int64_t key_rot_start, int is_neox_style,
                const rope_tensor *query_out, const rope_tensor *key_cache,
                const rope_tensor *value_cache, AppendPlan *plan, std::string *err) {
  *plan = AppendPlan();
  for (const rope_tensor *t : {positions, slots, key, table, key_cache})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  if ((query == nullptr) != (query_out == nullptr))
    return reject(err, ROPE_ERR_PARAM_NULLPTR, "query and query_out come together");
  if ((value == nullptr) != (value_cache == nullptr))
    return reject(err, ROPE_ERR_PARAM_NULLPTR, "value and value_cache come together");
  const rope_tensor *all[9] = {positions, slots,     key,   table,      key_cache,
                               query,     query_out, value, value_cache};
  for (const rope_tensor *t : all)
    if (t != nullptr && valid_rank(t) && count(t) > 0 && t->data == nullptr)
      return reject(err, ROPE_ERR_PARAM_NULLPTR, "a non-empty tensor has NULL data");

  if (positions->dtype != ROPE_I64 || slots->dtype != ROPE_I64)
    return reject(err, ROPE_ERR_PARAM_INVALID, "positions and slots must be int64");
  const rope_dtype dt = key->dtype;
  if (!is_float(dt)) return reject(err, ROPE_ERR_PARAM_INVALID, "key dtype unsupported");
  for (const rope_tensor *t : {table, key_cache, query, query_out, value, value_cache})
    if (t != nullptr && t->dtype != dt)
      return reject(err, ROPE_ERR_PARAM_INVALID, "all float tensors must share key's dtype");
  for (const rope_tensor *t : all)
    if (t != nullptr && (!valid_rank(t) || !addressable(t)))
      return reject(err, ROPE_ERR_PARAM_INVALID, "bad shape or extent");
  if (positions->ndim != 1 || slots->ndim != 1)
    return reject(err, ROPE_ERR_PARAM_INVALID, "positions and slots must be [numTokens]");
  if (table->ndim != 2 || key->ndim != 3 || key_cache->ndim != 4 ||
      (query != nullptr && (query->ndim != 3 || query_out->ndim != 3)) ||
      (value != nullptr && (value->ndim != 3 || value_cache->ndim != 4)))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "table must be 2-D, query, key and value 3-D, caches 4-D");
  const int64_t T = key->shape[0];
  if (positions->shape[0] != T || slots->shape[0] != T ||
      (query != nullptr && query->shape[0] != T) || (value != nullptr && value->shape[0] != T))
    return reject(err, ROPE_ERR_PARAM_INVALID, "token counts differ");
  for (int d = 1; d < 3; ++d)
    if (key_cache->shape[d + 1] != key->shape[d] ||
        (value != nullptr && value_cache->shape[d + 1] != value->shape[d]))
      return reject(err, ROPE_ERR_PARAM_INVALID, "cache heads or widths differ from key/value");
  if (value != nullptr &&
      (value_cache->shape[0] != key_cache->shape[0] || value_cache->shape[1] != key_cache->shape[1]))
    return reject(err, ROPE_ERR_PARAM_INVALID, "key and value cache differ in pages");
  if (query != nullptr)
    for (int d = 0; d < 3; ++d)
      if (query_out->shape[d] != query->shape[d])
        return reject(err, ROPE_ERR_PARAM_INVALID, "query_out shape differs from query");
  const int64_t rd = table->shape[1];
  if (table->shape[0] == 0 || rd == 0 || rd % 2 != 0)
    return reject(err, ROPE_ERR_PARAM_INVALID, "cos_sin_cache must be [maxSeqLen > 0, even > 0]");
  // widths bound: items of a token stay below 2^31 and element offsets in a head below 2^31
  constexpr int64_t kMaxWidth = int64_t(1) << 24;
  if (T > 0x7fffffff) return reject(err, ROPE_ERR_PARAM_INVALID, "too many tokens");
  for (const rope_tensor *t : {key, query, value})
    if (t != nullptr && (t->shape[2] > kMaxWidth || t->shape[1] > kMaxWidth ||
                         t->shape[1] * t->shape[2] > kMaxWidth))
      return reject(err, ROPE_ERR_PARAM_INVALID, "too many elements per token");
  if (key_rot_start < 0 || key_rot_start > key->shape[2] - rd)
    return reject(err, ROPE_ERR_PARAM_INVALID, "key_rot_start: the slice leaves the key head");
  if (query != nullptr && (query_rot_start < 0 || query_rot_start > query->shape[2] - rd))
    return reject(err, ROPE_ERR_PARAM_INVALID, "query_rot_start: the slice leaves the query head");
  for (const rope_tensor *t : all)
    if (t != nullptr && !non_negative_strides(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "negative strides are not supported");
  for (const rope_tensor *t : {key, table, key_cache, query, query_out, value, value_cache})
    if (t != nullptr && !unit_inner(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "rows need unit inner stride");
  const bool any_rows = key->shape[1] * key->shape[2] > 0 ||
                        (query != nullptr && query->shape[1] > 0) ||
                        (value != nullptr && value->shape[1] * value->shape[2] > 0);
  if (T == 0 || !any_rows) {
    plan->noop = true;
    return ROPE_OK;
  }
  for (const rope_tensor *t : {query_out, key_cache, value_cache}) {
    if (t == nullptr || count(t) == 0) continue;
    if (!injective(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "an output's strides reach an element twice");
    for (const rope_tensor *o : all) {
      if (o == nullptr || o == t || count(o) == 0) continue;
      if (t == query_out && o == query && identical_view(t, o)) continue;
      if (!disjoint(t, o))
        return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
    }
  }

  AppendPlan &p = *plan;
  const int64_t es = bytes_of(dt);
  p.dt = dt;
  p.neox = is_neox_style != 0;
  p.positions = static_cast<const int64_t *>(positions->data);
  p.slots = static_cast<const int64_t *>(slots->data);
  p.pos_stride = positions->stride[0];
  p.slot_stride = slots->stride[0];
  p.table = table->data;
  p.table_stride = table->stride[0];
  p.max_seq = table->shape[0];
  p.half = int32_t(rd / 2);
  p.T = T;
  p.page_size = std::max<int64_t>(key_cache->shape[1], 1);
  p.num_slots = key_cache->shape[0] * key_cache->shape[1];

  // 16-byte items where every head row, the slice and the table rows split into whole vectors.
  const int64_t v = 16 / es;
  bool vec = rd % (p.neox ? 2 * v : v) == 0 && rows_aligned16(table);
  const rope_tensor *ins[3] = {query, key, value};
  const rope_tensor *outs[3] = {query_out, key_cache, value_cache};
  const int64_t starts[3] = {query_rot_start, key_rot_start, 0};
  for (int g = 0; g < 3; ++g)
    if (ins[g] != nullptr && count(ins[g]) > 0)
      vec = vec && ins[g]->shape[2] % v == 0 && starts[g] % v == 0 && rows_aligned16(ins[g]) &&
            (count(outs[g]) == 0 || rows_aligned16(outs[g]));
  p.vector_io = vec;

  int64_t items = 0;
  for (int g = 0; g < 3; ++g) {
    AppendRows &r = p.rows[g];
    if (ins[g] == nullptr || count(ins[g]) == 0) continue;
    if (g > 0 && p.num_slots == 0) continue;  // a cache without slots takes nothing
    const rope_tensor *in = ins[g], *out = outs[g];
    r.in = in->data;
    r.out = out->data;
    r.in_tok = in->stride[0];
    r.in_head = in->stride[1];
    const int o = g == 0 ? 0 : 1;  // caches have a page dimension in front
    r.out_page = g == 0 ? 0 : out->stride[0];
    r.out_tok = out->stride[o];
    r.out_head = out->stride[o + 1];
    const bool in_place = g == 0 && query_out->data == query->data;
    head_items(&r, in->shape[2], starts[g], g == 2 ? 0 : rd, vec ? v : 1, p.neox, in_place);
    r.total = uint32_t(in->shape[1]) * r.items;
    r.all = T * int64_t(r.total);  // below 2^31 * 2^24
    r.div_items = make_fastdiv(std::max(1u, r.items));
    r.div_total = make_fastdiv(std::max(1u, r.total));
    items += r.all;
  }
  if (items == 0) {
    p.noop = true;
    return ROPE_OK;
  }
  for (AppendRows &r : p.rows) {
    r.blocks = (r.all + kAppendBlock - 1) / kAppendBlock;
    p.idx32 = p.idx32 && r.all + kAppendBlock < (int64_t(1) << 31);
  }
  return ROPE_OK;
}

}  // namespace ropeamd
