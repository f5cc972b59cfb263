// rope_q8_plan.cpp -- argument checks and launch plans of the append to and the attention over a
// paged cache in 8 bits (host only; every refusal happens before any HIP call).
#include "rope_q8_plan.h"

#include <algorithm>
#include <cmath>
#include <limits>

#include "rope_check.h"

namespace ropeamd {
namespace {

constexpr double kLog2e = 1.4426950408889634;
constexpr int64_t kIndexLimit = int64_t(1) << 30;  // token, row and page numbers stay inside int32
constexpr int64_t kMaxRow = int64_t(1) << 24;      // bytes from one cached token to the next

bool is_codes(rope_dtype dt) { return dt == ROPE_I8 || dt == ROPE_E4M3; }

// Checks of the codes and scales of the keys and values, and of the sequences' tables.
int check_cache(const rope_tensor *kc, const rope_tensor *vc, const rope_tensor *ks,
                const rope_tensor *vs, const rope_tensor *table, const rope_tensor *lens,
                const rope_tensor *offsets, int64_t T, std::string *err) {
  if (!is_codes(kc->dtype) || vc->dtype != kc->dtype)
    return reject(err, ROPE_ERR_PARAM_INVALID, "caches must be int8, or both float8 e4m3");
  if (ks->dtype != ROPE_F32 || vs->dtype != ROPE_F32)
    return reject(err, ROPE_ERR_PARAM_INVALID, "scales must be float32");
  if (kc->ndim != 4 || vc->ndim != 4 || ks->ndim != 3 || vs->ndim != 3)
    return reject(err, ROPE_ERR_PARAM_INVALID, "caches must be 4-D, scales 3-D");
  for (int d = 0; d < 3; ++d)
    if (kc->shape[d] != vc->shape[d] || ks->shape[d] != vs->shape[d])
      return reject(err, ROPE_ERR_PARAM_INVALID, "keys and values differ in pages, rows or heads");
  if (ks->shape[0] != kc->shape[0] || ks->shape[2] != kc->shape[2])
    return reject(err, ROPE_ERR_PARAM_INVALID, "scales must be [pages, blocks, key heads]");
  if (kc->shape[1] > 0 && (ks->shape[1] < 1 || kc->shape[1] % ks->shape[1] != 0))
    return reject(err, ROPE_ERR_PARAM_INVALID, "the blocks of a page must divide its rows");
  if (!is_i64_vector(lens) || table->dtype != ROPE_I64 || table->ndim != 2 ||
      (offsets != nullptr && !is_i64_vector(offsets)))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "seq_lens [B], page_table [B, maxPages], offsets [B + 1] must be int64");
  const int64_t B = lens->shape[0];
  if (table->shape[0] != B)
    return reject(err, ROPE_ERR_PARAM_INVALID, "page_table and seq_lens differ in sequences");
  if (offsets != nullptr ? offsets->shape[0] != B + 1 : (B == 0 ? T != 0 : T % B != 0))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "offsets must be [B + 1]; without them every sequence has T / B rows");
  if (table->shape[1] >= kIndexLimit || kc->shape[1] >= kIndexLimit ||
      table->shape[1] * kc->shape[1] >= kIndexLimit || kc->shape[0] >= kIndexLimit ||
      B >= kIndexLimit)
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many pages, sequences or tokens per sequence");
  if (!unit_inner(kc) || !unit_inner(vc))
    return reject(err, ROPE_ERR_PARAM_INVALID, "cache rows need unit inner stride");
  return ROPE_OK;
}

Sequences sequences_of(const rope_tensor *table, const rope_tensor *lens,
                       const rope_tensor *offsets, const rope_tensor *cache, int64_t T) {
  Sequences s;
  s.table = static_cast<const int64_t *>(table->data);
  s.table_seq = table->stride[0];
  s.table_page = table->stride[1];
  s.lens = static_cast<const int64_t *>(lens->data);
  s.len_stride = lens->stride[0];
  s.T = T;
  s.B = lens->shape[0];
  if (offsets != nullptr) {
    s.offsets = static_cast<const int64_t *>(offsets->data);
    s.off_stride = offsets->stride[0];
  } else {
    s.each = s.B > 0 ? T / s.B : 0;
  }
  s.num_pages = cache->shape[0];
  s.max_pages = table->shape[1];
  s.page_size = std::max<int64_t>(cache->shape[1], 1);
  s.div_page = make_fastdiv(uint32_t(s.page_size));
  return s;
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Whether every row start of t is a multiple of `bytes` (any power of two).
bool rows_aligned(const rope_tensor *t, int64_t bytes) {
  if (reinterpret_cast<uintptr_t>(t->data) % uintptr_t(bytes) != 0) return false;
  for (int d = 0; d + 1 < t->ndim; ++d)
    if (t->shape[d] > 1 && (t->stride[d] * bytes_of(t->dtype)) % bytes != 0) return false;
  return true;
}

}  // namespace

int plan_append_q8(const rope_tensor *positions, const rope_tensor *query, const rope_tensor *key,
                   const rope_tensor *value, const rope_tensor *table,
                   const rope_tensor *page_table, const rope_tensor *seq_lens,
                   const rope_tensor *offsets, int64_t query_rot_start, int64_t key_rot_start,
                   int is_neox_style, const rope_tensor *query_out, const rope_tensor *key_cache,
                   const rope_tensor *value_cache, const rope_tensor *key_scales,
                   const rope_tensor *value_scales, AppendQ8Plan *plan, std::string *err) {
  *plan = AppendQ8Plan();
  for (const rope_tensor *t : {positions, key, value, table, page_table, seq_lens, key_cache,
                               value_cache, key_scales, value_scales})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  if ((query == nullptr) != (query_out == nullptr))
    return reject(err, ROPE_ERR_PARAM_NULLPTR, "query and query_out come together");
  const int st = common_checks({positions, query, key, value, table, page_table, seq_lens, offsets,
                                query_out, key_cache, value_cache, key_scales, value_scales}, err);
  if (st != ROPE_OK) return st;

  const rope_dtype dt = key->dtype;
  if (!is_float(dt)) return reject(err, ROPE_ERR_PARAM_INVALID, "key dtype unsupported");
  for (const rope_tensor *t : {value, table, query, query_out})
    if (t != nullptr && t->dtype != dt)
      return reject(err, ROPE_ERR_PARAM_INVALID,
                    "query, value and cos_sin_cache must share key's dtype");
  if (!is_i64_vector(positions))
    return reject(err, ROPE_ERR_PARAM_INVALID, "positions must be int64 [numTokens]");
  if (table->ndim != 2 || key->ndim != 3 || value->ndim != 3 ||
      (query != nullptr && (query->ndim != 3 || query_out->ndim != 3)))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "cos_sin_cache must be 2-D, query, key and value 3-D");
  const int64_t T = key->shape[0];
  if (positions->shape[0] != T || value->shape[0] != T ||
      (query != nullptr && query->shape[0] != T))
    return reject(err, ROPE_ERR_PARAM_INVALID, "token counts differ");
  const int ck = check_cache(key_cache, value_cache, key_scales, value_scales, page_table,
                             seq_lens, offsets, T, err);
  if (ck != ROPE_OK) return ck;
  if (key_cache->shape[2] != key->shape[1] || value->shape[1] != key->shape[1] ||
      key_cache->shape[3] != key->shape[2] || value_cache->shape[3] != value->shape[2])
    return reject(err, ROPE_ERR_PARAM_INVALID, "cache heads or widths differ from key/value");
  if (query != nullptr)
    for (int d = 0; d < 3; ++d)
      if (query_out->shape[d] != query->shape[d])
        return reject(err, ROPE_ERR_PARAM_INVALID, "query_out shape differs from query");
  const int64_t rd = table->shape[1];
  if (table->shape[0] == 0 || rd == 0 || rd % 2 != 0)
    return reject(err, ROPE_ERR_PARAM_INVALID, "cos_sin_cache must be [maxSeqLen > 0, even > 0]");
  if (T >= kIndexLimit) return reject(err, ROPE_ERR_PARAM_INVALID, "too many tokens");
  constexpr int64_t kMaxWidth = int64_t(1) << 24;  // elements of a token, as of the other append
  for (const rope_tensor *t : {key, query, value})
    if (t != nullptr && (t->shape[2] > kMaxWidth || t->shape[1] > kMaxWidth ||
                         t->shape[1] * t->shape[2] > kMaxWidth))
      return reject(err, ROPE_ERR_PARAM_INVALID, "too many elements per token");
  // the kernel numbers a block's elements of a head in 32 bits
  if (key_cache->shape[1] > 0 && key_cache->shape[1] / key_scales->shape[1] *
                                         std::max(key->shape[2], value->shape[2]) >= kIndexLimit)
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many elements in a block of a head");
  if (key_rot_start < 0 || key_rot_start > key->shape[2] - rd)
    return reject(err, ROPE_ERR_PARAM_INVALID, "key_rot_start: the slice leaves the key head");
  if (query != nullptr && (query_rot_start < 0 || query_rot_start > query->shape[2] - rd))
    return reject(err, ROPE_ERR_PARAM_INVALID, "query_rot_start: the slice leaves the query head");
  for (const rope_tensor *t : {key, value, table, query, query_out})
    if (t != nullptr && !unit_inner(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "rows need unit inner stride");
  if (T == 0) {
    plan->noop = true;
    return ROPE_OK;
  }
  const rope_tensor *all[13] = {positions, query,     key,       value,       table,
                                page_table, seq_lens, offsets,   query_out,   key_cache,
                                value_cache, key_scales, value_scales};
  for (const rope_tensor *t : {query_out, key_cache, value_cache, key_scales, value_scales}) {
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

  AppendQ8Plan &p = *plan;
  const int64_t es = bytes_of(dt), v = 16 / es;
  p.dt = dt;
  p.neox = is_neox_style != 0;
  p.e4m3 = key_cache->dtype == ROPE_E4M3;
  p.positions = static_cast<const int64_t *>(positions->data);
  p.pos_stride = positions->stride[0];
  p.table = table->data;
  p.table_stride = table->stride[0];
  p.max_seq = table->shape[0];
  p.half = int32_t(rd / 2);
  p.heads = int32_t(key->shape[1]);
  p.seq = sequences_of(page_table, seq_lens, offsets, key_cache, T);

  // Whole 16-byte vectors of the inputs, and as many codes at a time, where everything is aligned.
  bool vec = rd % (p.neox ? 2 * v : v) == 0 && rows_aligned16(table);
  const rope_tensor *ins[3] = {query, key, value};
  const int64_t starts[3] = {query_rot_start, key_rot_start, 0};
  for (int g = 0; g < 3; ++g)
    if (ins[g] != nullptr && count(ins[g]) > 0)
      vec = vec && ins[g]->shape[2] % v == 0 && starts[g] % v == 0 && rows_aligned16(ins[g]);
  if (query != nullptr && count(query) > 0) vec = vec && rows_aligned16(query_out);
  for (const rope_tensor *t : {key_cache, value_cache})
    if (count(t) > 0) vec = vec && rows_aligned(t, v);
  p.vector_io = vec;
  const int64_t step = vec ? v : 1, run = vec ? v : 2;  // elements of an item, of a GPT-J one

  if (query != nullptr && count(query) > 0) {
    AppendRows &r = p.query;
    const bool in_place = query_out->data == query->data;
    r.in = query->data;
    r.out = query_out->data;
    r.in_tok = query->stride[0];
    r.in_head = query->stride[1];
    r.out_tok = query_out->stride[0];
    r.out_head = query_out->stride[1];
    r.rot_start = int32_t(query_rot_start);
    r.rot_items = uint32_t(p.neox ? rd / 2 / step : rd / run);
    r.items = r.rot_items + (in_place ? 0u : uint32_t((query->shape[2] - rd) / step));
    p.query_heads = query->shape[1];
    const int64_t each = query_heads_of(p.neox);
    r.total = uint32_t((query->shape[1] + each - 1) / each) * r.items;
    r.all = T * int64_t(r.total);  // below 2^30 * 2^24
    r.div_items = make_fastdiv(std::max(1u, r.items));
    r.div_total = make_fastdiv(std::max(1u, r.total));
    p.query_blocks = (r.all + kQ8Block - 1) / kQ8Block;
    p.idx32 = r.all + kQ8Block < (int64_t(1) << 31);  // else all numbers in 64
  }

  const bool any = p.heads > 0 && p.seq.B > 0 && p.seq.max_pages > 0 && key_cache->shape[0] > 0 &&
                   key_cache->shape[1] > 0;
  if (any) {
    p.block = int32_t(key_cache->shape[1] / key_scales->shape[1]);
    p.div_block = make_fastdiv(uint32_t(p.block));
    const rope_tensor *caches[2] = {key_cache, value_cache}, *scales[2] = {key_scales, value_scales};
    const int64_t spread = T / p.block + 2 * p.seq.B;
    p.by_token = T <= spread;
    p.places = p.by_token ? T : spread;
    const int64_t tokens = p.by_token ? 1 : p.block;  // of a place; numbered by token, mostly one
    int64_t lanes = 4;  // that hold them
    for (int g = 0; g < 2; ++g) {
      Q8Rows &r = p.kv[g];
      const rope_tensor *in = ins[g + 1], *c = caches[g], *s = scales[g];
      r.in = in->data;
      r.in_tok = in->stride[0];
      r.in_head = in->stride[1];
      r.codes = static_cast<uint8_t *>(c->data);
      r.page = c->stride[0];
      r.row = c->stride[1];
      r.head = c->stride[2];
      r.scales = static_cast<float *>(s->data);
      r.s_page = s->stride[0];
      r.s_block = s->stride[1];
      r.s_head = s->stride[2];
      r.dim = int32_t(in->shape[2]);
      r.wide_rows = in->shape[2] % 16 == 0 && rows_aligned16(c);
      const int64_t turned = g == 0 ? rd : 0;
      r.rot_start = int32_t(starts[g + 1]);
      r.rot_items = uint32_t(p.neox ? turned / 2 / step : turned / run);
      r.items = r.rot_items + uint32_t((in->shape[2] - turned) / step);
      r.div_items = make_fastdiv(std::max(1u, r.items));
      while ((uint32_t(1) << r.row_log2) < r.items) ++r.row_log2;
      const int64_t item = g == 0 && (p.neox || step == 1) ? 2 * step : step;  // elements held for one
      lanes = std::max({lanes, (tokens << r.row_log2) * item / kQ8Held,
                        std::min(int64_t(64), int64_t(1) << r.row_log2)});
    }
    p.lanes = 4;
    while (p.lanes < kQ8Block && p.lanes < lanes) p.lanes *= 2;
    while ((1 << p.lanes_log2) != p.lanes) ++p.lanes_log2;
    for (Q8Rows &r : p.kv) {  // a row's items of one wavefront; rows of width 0 have none, and no address
      r.side_by_side = r.items > 0 && (1 << r.row_log2) <= std::min(p.lanes, 64);
      if (!r.side_by_side) r.row_log2 = 0;
    }
    const int64_t heads_each = std::max(1, 64 / p.lanes), units = kQ8Block / std::max(64, p.lanes);
    // whole workgroups for keys, and for values: the wavefronts of one meet in LDS
    p.head_groups = 2 * int32_t(up((p.heads + heads_each - 1) / heads_each, p.lanes > 64 ? units : 1));
    p.div_groups = make_fastdiv(uint32_t(p.head_groups));
    p.kv_blocks = (p.places * p.head_groups + units - 1) / units;
    p.idx32 = p.idx32 && p.kv_blocks * units < (int64_t(1) << 31);
  }
  if (p.kv_blocks + p.query_blocks == 0) p.noop = true;
  return ROPE_OK;
}

// Rows of a workgroup: one or two tiles of 16, as many as a sequence's (token, head) rows of a key
// head fill, or those of the kernel for many.  64 sequences of 200-9000 tokens, 8 key heads of 128 (64), with 32 rows
// each 99 us (64); with 40, 48, 64 and 96 111, 115, 116 and 127 (80, 79, 82 and 87) by that kernel, in tiles of 32
// rows 135, 137, 143 and 220 (85, 85, 89 and 140).  One class serves a call, by the mean number of queries:
// sequences that are far from it are served worse than in a call of their own (256 that decode and a piece of 2048
// tokens 493 us, in two calls 243 + 79).
static int64_t q8_rows(int64_t tokens, int64_t group, int64_t sequences) {
  const int64_t n = std::max<int64_t>(sequences, 1);
  const int64_t rows = group * (tokens / n + (tokens % n != 0));
  return rows <= 16 ? 16 : rows <= 32 ? 32 : kQ8ManyRows;
}

// Workgroups: as many as the card holds at a time.
static int64_t q8_groups(int64_t rows, int64_t width) {
  return 256 * (rows == kQ8ManyRows ? (width == 256 ? 1 : 2) : q8_waves(int(width), int(rows / 16)));
}

// Key heads of a workgroup, at most.
static int64_t q8_abreast(int64_t rows, int64_t kv_heads) {
  return rows == kQ8ManyRows ? 1 : kv_heads % 4 == 0 ? 4 : kv_heads % 2 == 0 ? 2 : 1;
}

int64_t attention_q8_workspace(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_size,
                               int64_t sequences) {
  // sizes that the call has no work for, or refuses
  if (tokens <= 0 || heads <= 0 || kv_heads <= 0 || head_size <= 0 || sequences <= 0) return 0;
  if (tokens >= kIndexLimit || heads >= kIndexLimit || head_size > 256 || heads % kv_heads != 0)
    return 0;
  const int64_t rows = q8_rows(tokens, heads / kv_heads, sequences);
  const int64_t groups = q8_groups(rows, head_size);
  const int64_t lines = groups * 2 * q8_abreast(rows, kv_heads) * rows;
  return up(groups * 2 * kQ8JoinWords * 8, 256) + up(lines * 8, 256) + lines * head_size * 4;
}

int plan_attention_q8(const rope_tensor *query, const rope_tensor *key_cache,
                      const rope_tensor *value_cache, const rope_tensor *key_scales,
                      const rope_tensor *value_scales, const rope_tensor *page_table,
                      const rope_tensor *seq_lens, const rope_tensor *offsets, double scale,
                      const rope_tensor *out, const rope_tensor *lse, void *workspace,
                      int64_t workspace_bytes, AttnQ8Plan *plan, std::string *err) {
  *plan = AttnQ8Plan();
  for (const rope_tensor *t : {query, key_cache, value_cache, key_scales, value_scales, page_table,
                               seq_lens, out})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  const int st = common_checks({query, key_cache, value_cache, key_scales, value_scales,
                                page_table, seq_lens, offsets, out, lse}, err);
  if (st != ROPE_OK) return st;
  const rope_dtype dt = query->dtype;
  if (dt != ROPE_F16 && dt != ROPE_BF16)
    return reject(err, ROPE_ERR_PARAM_INVALID, "query must be float16 or bfloat16");
  if (out->dtype != dt)
    return reject(err, ROPE_ERR_PARAM_INVALID, "out must share query's dtype");
  if (lse != nullptr && lse->dtype != ROPE_F32)
    return reject(err, ROPE_ERR_PARAM_INVALID, "lse must be float32");
  if (query->ndim != 3 || out->ndim != 3 || (lse != nullptr && lse->ndim != 2))
    return reject(err, ROPE_ERR_PARAM_INVALID, "query and out must be 3-D, lse 2-D");
  const int64_t T = query->shape[0], H = query->shape[1], D = query->shape[2];
  const int ck = check_cache(key_cache, value_cache, key_scales, value_scales, page_table,
                             seq_lens, offsets, T, err);
  if (ck != ROPE_OK) return ck;
  const int64_t B = seq_lens->shape[0], N = key_cache->shape[2];
  if (D != 64 && D != 128 && D != 256)
    return reject(err, ROPE_ERR_PARAM_INVALID, "heads must be 64, 128 or 256 wide");
  if (key_cache->shape[3] != D || value_cache->shape[3] != D)
    return reject(err, ROPE_ERR_PARAM_INVALID, "cache rows must be as wide as the query's");
  if (N < 1 ? H != 0 : H % N != 0)
    return reject(err, ROPE_ERR_PARAM_INVALID, "query heads must be a multiple of the key heads");
  if (out->shape[0] != T || out->shape[1] != H || out->shape[2] != D ||
      (lse != nullptr && (lse->shape[0] != T || lse->shape[1] != H)))
    return reject(err, ROPE_ERR_PARAM_INVALID, "out must be [T, heads, D], lse [T, heads]");
  const double scaled = scale * kLog2e;
  if (!(std::fabs(scaled) <= std::numeric_limits<float>::max()))
    return reject(err, ROPE_ERR_PARAM_INVALID, "scale must be finite, and below 2^127 in size");
  if (T >= kIndexLimit || H >= kIndexLimit || T * H >= kIndexLimit)
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many query rows");
  if (!unit_inner(query) || !rows_aligned16(query) || !rows_aligned16(key_cache) ||
      !rows_aligned16(value_cache))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "query and cache rows need unit inner stride and 16-byte aligned starts");
  for (const rope_tensor *t : {key_cache, value_cache})
    if (t->shape[1] > 1 && t->stride[1] >= kMaxRow)
      return reject(err, ROPE_ERR_PARAM_INVALID, "cached tokens must lie less than 2^24 apart");
  if (!row_major(out) || (lse != nullptr && !row_major(lse)))
    return reject(err, ROPE_ERR_PARAM_INVALID, "out and lse must be contiguous");
  if (!aligned16(out->data)) return reject(err, ROPE_ERR_PARAM_INVALID, "out must be 16-byte aligned");
  if (T == 0 || H == 0 || B == 0) {
    plan->noop = true;
    return ROPE_OK;
  }
  if (!outputs_apart({out, lse}, {query, key_cache, value_cache, key_scales, value_scales,
                                  page_table, seq_lens, offsets}))
    return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
  const int64_t need = attention_q8_workspace(T, H, N, D, B);
  if (workspace == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "workspace is NULL");
  if (workspace_bytes < need || !aligned16(workspace))
    return reject(err, ROPE_ERR_PARAM_INVALID, "workspace too small or not 16-byte aligned");
  for (const rope_tensor *t : {query, key_cache, value_cache, key_scales, value_scales, page_table,
                               seq_lens, offsets, out, lse})
    if (touches(workspace, need, t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "workspace overlaps a tensor");

  AttnQ8Plan &p = *plan;
  p.dt = dt;
  p.e4m3 = key_cache->dtype == ROPE_E4M3;
  p.q = query->data;
  p.q_tok = query->stride[0];
  p.q_head = query->stride[1];
  const rope_tensor *caches[2] = {key_cache, value_cache}, *scales[2] = {key_scales, value_scales};
  for (int g = 0; g < 2; ++g) {
    Q8Cache &c = g == 0 ? p.k : p.v;
    c.codes = static_cast<const uint8_t *>(caches[g]->data);
    c.page = caches[g]->stride[0];
    c.row = caches[g]->shape[1] > 1 ? int32_t(caches[g]->stride[1]) : 0;
    c.head = caches[g]->stride[2];
    c.scales = static_cast<const float *>(scales[g]->data);
    c.s_page = scales[g]->stride[0];
    c.s_block = scales[g]->stride[1];
    c.s_head = scales[g]->stride[2];
  }
  p.seq = sequences_of(page_table, seq_lens, offsets, key_cache, T);
  // a cache without pages or rows holds no tokens: every length is clamped to 0
  if (key_cache->shape[0] == 0 || key_cache->shape[1] == 0) p.seq.max_pages = 0;
  p.block = key_cache->shape[1] > 0 ? int32_t(key_cache->shape[1] / key_scales->shape[1]) : 1;
  p.mode = p.seq.page_size % 16 != 0 ? 0 : p.block % 4 != 0 ? 1 : 2;
  p.heads = int32_t(H);
  p.kv_heads = int32_t(N);
  p.group = int32_t(H / N);
  p.head_size = int32_t(D);
  p.div_group = make_fastdiv(uint32_t(p.group));
  p.div_block = make_fastdiv(uint32_t(p.block));
  p.scale_log2 = float(scaled);
  p.rows = int32_t(q8_rows(T, p.group, B));
  p.groups = int32_t(q8_groups(p.rows, D));
  p.out = out->data;
  p.lse = lse != nullptr ? static_cast<float *>(lse->data) : nullptr;
  const int64_t rows = p.rows;
  const bool side_by_side = p.seq.page_size == 1 || p.k.head < p.k.row;
  p.abreast = side_by_side ? int32_t(q8_abreast(rows, N)) : 1;
  while ((1 << p.abreast_log2) < p.abreast) ++p.abreast_log2;
  p.head_sets = p.kv_heads / p.abreast;
  p.step_log2 = q8_step_log2(rows, D, p.abreast_log2);
  // tiles: as many as the rows fill, and one begun for every sequence; steps, and what beginning costs
  const double tiles = double(p.head_sets) * (double(T) * double(p.group) / double(rows) + double(B));
  const double steps = double(p.seq.max_pages) * double(p.seq.page_size) / double(1 << p.step_log2) + 16;
  p.small = tiles * steps < double(int64_t(1) << 30);
  char *w = static_cast<char *>(workspace);
  p.joins = reinterpret_cast<int64_t *>(w);
  w += up(p.groups * 2 * kQ8JoinWords * 8, 256);
  p.stats = reinterpret_cast<float *>(w);
  w += up(2 * p.groups * p.abreast * rows * 8, 256);
  p.parts = reinterpret_cast<float *>(w);
  return ROPE_OK;
}

}  // namespace ropeamd
