// rope_pages_plan.cpp -- argument checks and launch plans of the operators on a cache's pages (host
// only; every refusal happens before any HIP call).
#include "rope_pages_plan.h"

#include <algorithm>
#include <numeric>
#include <tuple>
#include <utility>

#include "rope_check.h"

namespace ropeamd {
namespace {

constexpr int64_t kIndexLimit = int64_t(1) << 30;  // pages, rows, sequences; entries of a table 2^40
constexpr int64_t kMaxCaches = int64_t(1) << 16;
constexpr int64_t kMaxPageWords = int64_t(1) << 31;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// What caches of one description have in common: a page as one dense block, `part` bytes of it for each of
// `parts` blocks of its tokens (0: copied whole only), and the bytes from a cache's first to its last.
struct CacheKind {
  const rope_tensor *like = nullptr;
  int64_t elements = 0, bytes = 0, page = 0, part = 0, reach = 0;
  uint32_t parts = 0;
};

bool alike(const rope_tensor *a, const rope_tensor *b) {
  if (a->ndim != b->ndim || a->dtype != b->dtype) return false;
  for (int d = 0; d < a->ndim; ++d)
    if (a->shape[d] != b->shape[d] || a->stride[d] != b->stride[d]) return false;
  return true;
}

// False where a page of t is no dense block.
bool describe(const rope_tensor *t, int64_t page_size, CacheKind *k) {
  int order[3], n = 0;
  for (int d = 1; d < t->ndim; ++d)
    if (t->shape[d] > 1) order[n++] = d;
  std::sort(order, order + n, [t](int x, int y) { return t->stride[x] < t->stride[y]; });
  int64_t dense = 1;
  for (int i = 0; i < n; ++i) {
    if (t->stride[order[i]] != dense) return false;
    dense *= t->shape[order[i]];
  }
  const int64_t es = bytes_of(t->dtype);
  k->bytes = dense * es;
  k->page = t->shape[0] > 1 ? t->stride[0] * es : 0;
  // The parts of a page that tokens lie in, where they are outermost.  By the form alone, [pages, pageSize, ..] or
  // scales as the 8-bit cache has them: a length that only fits may be heads, or keys and values, of which a part
  // would lack some.
  const int64_t n1 = t->ndim >= 3 ? t->shape[1] : 0;
  const bool tokens = n1 > 0 && n1 == page_size;
  const bool blocks = n1 > 0 && t->ndim == 3 && t->dtype == ROPE_F32 && page_size % n1 == 0;
  if (page_size > 0 && (tokens || blocks) && (n1 == 1 || order[n - 1] == 1)) {
    k->part = k->bytes / n1;
    k->parts = uint32_t(n1);
  }
  uintptr_t a, b;
  extent(t, &a, &b);
  k->reach = int64_t(b - a);
  return true;
}

// False where a page has too many words.
bool cache_of(const rope_tensor *t, const CacheKind &k, PageCache *c) {
  c->base = static_cast<char *>(t->data);
  c->page = k.page;
  const uint64_t all = reinterpret_cast<uintptr_t>(t->data) | uint64_t(k.page) | uint64_t(k.bytes) |
                       uint64_t(k.part);
  PageRun &r = c->run;
  while (r.width < 4 && (all >> r.width & 1) == 0) ++r.width;
  if (k.bytes >> r.width >= kMaxPageWords) return false;
  r.vecs = uint32_t(k.bytes >> r.width);
  r.parts = k.part > 0 ? k.parts : 0;
  r.part_words = uint32_t(k.part >> r.width);
  if (r.vecs < 64) {
    r.lanes_log2 = 0;
    while ((1u << r.lanes_log2) < r.vecs) ++r.lanes_log2;
  }
  return true;
}

auto order_of(const PageRun &r) { return std::tie(r.vecs, r.width, r.parts, r.part_words); }

// Where a cache lies: from its first byte to its last, pages of `bytes` bytes every `page` (0: one page).
struct Extent {
  uintptr_t first, end;
  int64_t bytes, page;
  const rope_tensor *t;
};

// Whether n caches whose extents meet provably share no byte because they lie side by side in every page of one
// allocation (all layers' keys, values and scales of a page together): modulo the greatest common divisor of
// their page strides, their pages are windows of their own.  n caches take n log n steps: the
// checks of 128 such caches 9 us, of 512 34 (compared in pairs 292 and 4900).
bool side_by_side(const Extent *c, size_t n) {
  int64_t m = 0;
  for (size_t i = 0; i < n; ++i) m = std::gcd(m, c[i].page);
  if (m == 0) return false;
  std::vector<std::pair<int64_t, int64_t>> windows(n);  // place, bytes
  for (size_t i = 0; i < n; ++i) windows[i] = {int64_t(c[i].first % uintptr_t(m)), c[i].bytes};
  std::sort(windows.begin(), windows.end());
  for (size_t i = 0; i < n; ++i) {
    const int64_t next = i + 1 < n ? windows[i + 1].first : windows[0].first + m;
    if (windows[i].first + windows[i].second > next) return false;
  }
  return true;
}

bool caches_apart(const std::vector<Extent> &c) {  // sorted by their first bytes
  for (size_t i = 0, end; i < c.size(); i = end) {
    uintptr_t last = c[i].end;
    for (end = i + 1; end < c.size() && c[end].first < last; ++end) last = std::max(last, c[end].end);
    if (end - i == 1 || side_by_side(&c[i], end - i)) continue;
    for (size_t k = i; k < end; ++k)
      for (size_t l = k + 1; l < end && c[l].first < c[k].end; ++l)
        if (!disjoint(c[k].t, c[l].t)) return false;
  }
  return true;
}

// The caches of a call: checked, and without those that hold nothing.  All layers' are described alike, so
// what follows from a description is worked out once for each of the last few (128 caches of a fork took 31 us
// of the host, with the comparisons below by extents 6).
int check_caches(const rope_tensor *caches, int64_t num_caches, int64_t *pages, int64_t page_size,
                 std::vector<PageCache> *list, std::vector<Extent> *extents, std::string *err) {
  list->clear();
  if (num_caches < 0 || num_caches > kMaxCaches)
    return reject(err, ROPE_ERR_PARAM_INVALID, "num_caches must be in [0, 65536]");
  if (num_caches > 0 && caches == nullptr)
    return reject(err, ROPE_ERR_PARAM_NULLPTR, "caches is NULL");
  extents->reserve(size_t(num_caches));
  list->reserve(size_t(num_caches));
  constexpr int kKinds = 8;
  CacheKind kinds[kKinds];
  int known = 0;
  for (int64_t i = 0; i < num_caches; ++i) {
    const rope_tensor *t = caches + i;
    const CacheKind *kind = nullptr;
    for (int k = 0; k < std::min(known, kKinds) && kind == nullptr; ++k)
      if (alike(kinds[k].like, t)) kind = &kinds[k];
    if (kind == nullptr || (kind->elements > 0 && t->data == nullptr)) {
      const int st = common_checks({t}, err);
      if (st != ROPE_OK) return st;
      if (bytes_of(t->dtype) == 0)
        return reject(err, ROPE_ERR_PARAM_INVALID, "a cache's dtype is unsupported");
      if (*pages < 0) *pages = t->shape[0];
      if (t->shape[0] != *pages)
        return reject(err, ROPE_ERR_PARAM_INVALID, "the caches differ in pages");
      CacheKind &k = kinds[known++ % kKinds];
      k = CacheKind();
      k.like = t;
      k.elements = count(t);
      if (k.elements > 0 && !describe(t, page_size, &k))
        return reject(err, ROPE_ERR_PARAM_INVALID,
                      "a page of a cache must be one dense block of less than 2^31 words");
      if (k.elements > 0 && !injective(t))
        return reject(err, ROPE_ERR_PARAM_INVALID, "the pages of a cache overlap");
      kind = &k;
    }
    if (kind->elements == 0) continue;
    PageCache c;
    if (!cache_of(t, *kind, &c))
      return reject(err, ROPE_ERR_PARAM_INVALID,
                    "a page of a cache must be one dense block of less than 2^31 words");
    const uintptr_t first = reinterpret_cast<uintptr_t>(t->data);
    extents->push_back({first, first + uintptr_t(kind->reach), kind->bytes, kind->page, t});
    list->push_back(c);
  }
  const auto before = [](const Extent &x, const Extent &y) { return x.first < y.first; };
  if (!std::is_sorted(extents->begin(), extents->end(), before))
    std::sort(extents->begin(), extents->end(), before);
  if (!caches_apart(*extents)) return reject(err, ROPE_ERR_PARAM_INVALID, "caches overlap");
  // pages that are alike side by side (the numbers are sorted, and the caches, of 64 bytes, put there once)
  std::vector<uint32_t> place(list->size());
  for (size_t i = 0; i < place.size(); ++i) place[i] = uint32_t(i);
  const std::vector<PageCache> &c = *list;
  std::stable_sort(place.begin(), place.end(),
                   [&c](uint32_t x, uint32_t y) { return order_of(c[x].run) < order_of(c[y].run); });
  std::vector<PageCache> sorted;
  sorted.reserve(place.size());
  for (const uint32_t i : place) sorted.push_back(c[i]);
  list->swap(sorted);
  return ROPE_OK;
}

// Whether t, if it holds anything, shares memory with one of the caches.
bool meets_caches(const rope_tensor *t, const std::vector<Extent> &caches) {
  if (t == nullptr || count(t) == 0) return false;
  uintptr_t first, end;
  extent(t, &first, &end);
  for (const Extent &e : caches)
    if (first < e.end && e.first < end && !disjoint(t, e.t)) return true;
  return false;
}

bool in_caches(const void *p, int64_t bytes, const std::vector<Extent> &caches) {
  const uintptr_t first = reinterpret_cast<uintptr_t>(p);
  for (const Extent &e : caches)
    if (bytes > 0 && first < e.end && e.first < first + uintptr_t(bytes)) return true;
  return false;
}

PageTable table_of(const rope_tensor *t) {
  return {static_cast<int64_t *>(t->data), t->shape[0], t->shape[1], t->stride[0], t->stride[1]};
}

const int64_t *i64(const rope_tensor *t) { return static_cast<const int64_t *>(t->data); }
int64_t *i64_out(const rope_tensor *t) { return static_cast<int64_t *>(t->data); }

}  // namespace

size_t take_caches(const std::vector<PageCache> &list, size_t at, int words, PageCaches *to) {
  to->runs = to->count = 0;
  for (; at < list.size() && to->count < kPageCaches; ++at) {
    const PageCache &c = list[at];
    if (to->runs == 0 || order_of(to->run[to->runs - 1]) != order_of(c.run)) {
      if (to->runs == kPageRuns) break;
      to->run[to->runs] = c.run;
      to->run[to->runs++].first = to->count;
    }
    ++to->run[to->runs - 1].count;
    to->base[to->count] = c.base;
    to->page[to->count++] = c.page;
  }
  for (int r = 0; r < to->runs; ++r) {
    PageRun &run = to->run[r];
    if (run.lanes_log2 == 6)
      run.pieces = (run.vecs + 64 * uint32_t(words) - 1) / (64 * uint32_t(words));
    run.div_pieces = make_fastdiv(run.pieces);
  }
  return at;
}

int plan_copy_pages(const rope_tensor *sources, const rope_tensor *targets,
                    const rope_tensor *caches, int64_t num_caches, CopyPagesPlan *plan,
                    std::vector<PageCache> *list, std::string *err) {
  *plan = CopyPagesPlan();
  for (const rope_tensor *t : {sources, targets})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  const int st = common_checks({sources, targets}, err);
  if (st != ROPE_OK) return st;
  if (!is_i64_vector(sources) || !is_i64_vector(targets) || sources->shape[0] != targets->shape[0])
    return reject(err, ROPE_ERR_PARAM_INVALID, "sources and targets must be int64 of one length");
  int64_t pages = -1;
  std::vector<Extent> extents;
  const int ck = check_caches(caches, num_caches, &pages, 0, list, &extents, err);
  if (ck != ROPE_OK) return ck;
  if (pages >= kIndexLimit || sources->shape[0] >= kIndexLimit)
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many pages");
  if (meets_caches(sources, extents) || meets_caches(targets, extents))
    return reject(err, ROPE_ERR_PARAM_INVALID, "a cache overlaps another tensor");
  plan->sources = i64(sources);
  plan->targets = i64(targets);
  plan->source_stride = sources->stride[0];
  plan->target_stride = targets->stride[0];
  plan->moves = sources->shape[0];
  plan->num_pages = pages;
  if (plan->moves == 0) list->clear();
  return ROPE_OK;
}

int64_t fork_workspace(int64_t sequences, int64_t rows, int64_t pages) {
  if (sequences < 0 || rows < 0 || pages < 0 || sequences >= kIndexLimit || rows >= kIndexLimit ||
      pages >= kIndexLimit)
    return 0;
  const int64_t chunks = (pages + kPageChunk - 1) / kPageChunk;
  return 256 + 3 * up(sequences * 4, 256) + up(rows * 8, 256) + up(rows * 24, 256) +
         up(chunks * 4, 256) + up(pages * 4, 256);
}

int plan_fork_pages(const rope_tensor *page_table, const rope_tensor *seq_lens,
                    const rope_tensor *parents, const rope_tensor *grow,
                    const rope_tensor *ref_counts, int64_t page_size, const rope_tensor *caches,
                    int64_t num_caches, const rope_tensor *page_table_out,
                    const rope_tensor *seq_lens_out, const rope_tensor *ref_counts_out,
                    const rope_tensor *shortage, void *workspace, int64_t workspace_bytes,
                    ForkPlan *plan, std::vector<PageCache> *list, std::string *err) {
  *plan = ForkPlan();
  for (const rope_tensor *t : {page_table, seq_lens, parents, ref_counts, page_table_out,
                               seq_lens_out, ref_counts_out, shortage})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  const int st = common_checks({page_table, seq_lens, parents, grow, ref_counts, page_table_out,
                                seq_lens_out, ref_counts_out, shortage}, err);
  if (st != ROPE_OK) return st;
  for (const rope_tensor *t : {page_table, page_table_out})
    if (t->dtype != ROPE_I64 || t->ndim != 2)
      return reject(err, ROPE_ERR_PARAM_INVALID, "page tables must be int64 and 2-D");
  for (const rope_tensor *t : {seq_lens, parents, grow, ref_counts, seq_lens_out, ref_counts_out,
                               shortage})
    if (t != nullptr && !is_i64_vector(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "lengths, rows and counts must be int64 and 1-D");
  const int64_t B = seq_lens->shape[0], R = parents->shape[0], pages = ref_counts->shape[0];
  if (page_table->shape[0] != B || page_table_out->shape[0] != R || seq_lens_out->shape[0] != R ||
      (grow != nullptr && grow->shape[0] != R))
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "page_table and seq_lens are [B, ..], parents, grow and the new ones [R, ..]");
  if (ref_counts_out->shape[0] != pages || shortage->shape[0] != 1)
    return reject(err, ROPE_ERR_PARAM_INVALID, "ref_counts_out must be [pages], shortage [1]");
  if (page_table_out->shape[1] < page_table->shape[1])
    return reject(err, ROPE_ERR_PARAM_INVALID, "page_table_out is narrower than page_table");
  if (page_size < 1 || page_size >= kIndexLimit)
    return reject(err, ROPE_ERR_PARAM_INVALID, "page_size must be in [1, 2^30)");
  if (B >= kIndexLimit || R >= kIndexLimit || pages >= kIndexLimit ||
      page_table_out->shape[1] >= kIndexLimit || page_table_out->shape[1] * page_size >= kIndexLimit ||
      B * page_table->shape[1] >= (int64_t(1) << 40) ||
      R * page_table_out->shape[1] >= (int64_t(1) << 40))
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many pages, rows or tokens");
  int64_t cache_pages = pages;
  std::vector<Extent> extents;
  const int ck = check_caches(caches, num_caches, &cache_pages, page_size, list, &extents, err);
  if (ck != ROPE_OK) return ck;
  const rope_tensor *ins[5] = {page_table, seq_lens, parents, grow, ref_counts};
  const rope_tensor *outs[4] = {page_table_out, seq_lens_out, ref_counts_out, shortage};
  for (const rope_tensor *o : outs) {
    if (count(o) == 0) continue;
    if (!injective(o))
      return reject(err, ROPE_ERR_PARAM_INVALID, "an output's strides reach an element twice");
    for (const rope_tensor *t : ins) {
      if (t == nullptr || count(t) == 0) continue;
      if (o == ref_counts_out && t == ref_counts && identical_view(o, t)) continue;
      if (!disjoint(o, t))
        return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
    }
    for (const rope_tensor *t : outs)
      if (t != o && count(t) > 0 && !disjoint(o, t))
        return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
  }
  for (const rope_tensor *t : {page_table, seq_lens, parents, grow, ref_counts, page_table_out,
                               seq_lens_out, ref_counts_out, shortage})
    if (meets_caches(t, extents))
      return reject(err, ROPE_ERR_PARAM_INVALID, "a cache overlaps another tensor");
  const int64_t need = fork_workspace(B, R, pages);
  if (workspace == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "workspace is NULL");
  if (workspace_bytes < need || !aligned16(workspace))
    return reject(err, ROPE_ERR_PARAM_INVALID, "workspace too small or not 16-byte aligned");
  for (const rope_tensor *t : {page_table, seq_lens, parents, grow, ref_counts, page_table_out,
                               seq_lens_out, ref_counts_out, shortage})
    if (touches(workspace, need, t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "workspace overlaps a tensor");
  if (in_caches(workspace, need, extents))
    return reject(err, ROPE_ERR_PARAM_INVALID, "workspace overlaps a tensor");

  ForkPlan &p = *plan;
  p.table = table_of(page_table);
  p.out = table_of(page_table_out);
  p.lens = i64(seq_lens);
  p.len_stride = seq_lens->stride[0];
  p.parents = i64(parents);
  p.parent_stride = parents->stride[0];
  if (grow != nullptr) {
    p.grow = i64(grow);
    p.grow_stride = grow->stride[0];
  }
  p.refs = i64(ref_counts);
  p.ref_stride = ref_counts->stride[0];
  p.lens_out = i64_out(seq_lens_out);
  p.len_out_stride = seq_lens_out->stride[0];
  p.refs_out = i64_out(ref_counts_out);
  p.ref_out_stride = ref_counts_out->stride[0];
  p.shortage = i64_out(shortage);
  p.num_pages = pages;
  p.page_size = page_size;
  p.chunks = (pages + kPageChunk - 1) / kPageChunk;
  const int64_t entries =  // the first one's thread writes the shortage, too
      std::max({int64_t(1), R * std::max<int64_t>(p.out.width, 1), B * p.table.width});
  p.table_blocks = std::min<int64_t>(1 << 16, (entries + kPageBlock - 1) / kPageBlock);
  char *w = static_cast<char *>(workspace);
  auto take = [&w](int64_t bytes) {
    char *at = w;
    w += up(bytes, 256);
    return at;
  };
  p.totals = reinterpret_cast<int64_t *>(take(256));
  p.first = reinterpret_cast<int32_t *>(take(B * 4));
  p.children = reinterpret_cast<int32_t *>(take(B * 4));
  p.kept = reinterpret_cast<int32_t *>(take(B * 4));
  p.base = reinterpret_cast<int64_t *>(take(R * 8));
  p.copies = reinterpret_cast<int64_t *>(take(R * 24));
  p.counts = reinterpret_cast<int32_t *>(take(p.chunks * 4));
  p.free = reinterpret_cast<int32_t *>(take(pages * 4));
  return ROPE_OK;
}

int64_t compact_workspace(int64_t pages) {
  if (pages < 0 || pages >= kIndexLimit) return 0;
  const int64_t chunks = (pages + kPageChunk - 1) / kPageChunk;
  return 256 + up((pages / 2 + 1) * 16, 256) + up(chunks * 4, 256);
}

int plan_compact_pages(const rope_tensor *page_table, const rope_tensor *ref_counts,
                       const rope_tensor *caches, int64_t num_caches,
                       const rope_tensor *page_table_out, const rope_tensor *ref_counts_out,
                       const rope_tensor *page_map, const rope_tensor *live, void *workspace,
                       int64_t workspace_bytes, CompactPlan *plan, std::vector<PageCache> *list,
                       std::string *err) {
  *plan = CompactPlan();
  for (const rope_tensor *t : {page_table, ref_counts, page_table_out, ref_counts_out, page_map,
                               live})
    if (t == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "a tensor argument is NULL");
  const int st = common_checks({page_table, ref_counts, page_table_out, ref_counts_out, page_map,
                                live}, err);
  if (st != ROPE_OK) return st;
  for (const rope_tensor *t : {page_table, page_table_out})
    if (t->dtype != ROPE_I64 || t->ndim != 2)
      return reject(err, ROPE_ERR_PARAM_INVALID, "page tables must be int64 and 2-D");
  for (const rope_tensor *t : {ref_counts, ref_counts_out, page_map, live})
    if (!is_i64_vector(t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "counts and page_map must be int64 and 1-D");
  const int64_t pages = ref_counts->shape[0];
  if (ref_counts_out->shape[0] != pages || page_map->shape[0] != pages || live->shape[0] != 1)
    return reject(err, ROPE_ERR_PARAM_INVALID,
                  "ref_counts_out and page_map must be [pages], live [1]");
  for (int d = 0; d < 2; ++d)
    if (page_table_out->shape[d] != page_table->shape[d])
      return reject(err, ROPE_ERR_PARAM_INVALID, "page_table_out shape differs from page_table");
  if (pages >= kIndexLimit || count(page_table) >= (int64_t(1) << 40))
    return reject(err, ROPE_ERR_PARAM_INVALID, "too many pages");
  int64_t cache_pages = pages;
  std::vector<Extent> extents;
  const int ck = check_caches(caches, num_caches, &cache_pages, 0, list, &extents, err);
  if (ck != ROPE_OK) return ck;
  const rope_tensor *ins[2] = {page_table, ref_counts};
  const rope_tensor *outs[4] = {page_table_out, ref_counts_out, page_map, live};
  for (int k = 0; k < 4; ++k) {
    const rope_tensor *o = outs[k];
    if (count(o) == 0) continue;
    if (!injective(o))
      return reject(err, ROPE_ERR_PARAM_INVALID, "an output's strides reach an element twice");
    for (int i = 0; i < 2; ++i) {
      if (count(ins[i]) == 0 || (k == i && identical_view(o, ins[i]))) continue;
      if (!disjoint(o, ins[i]))
        return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
    }
    for (const rope_tensor *t : outs)
      if (t != o && count(t) > 0 && !disjoint(o, t))
        return reject(err, ROPE_ERR_PARAM_INVALID, "an output overlaps another tensor");
  }
  for (const rope_tensor *t : {page_table, ref_counts, page_table_out, ref_counts_out, page_map,
                               live})
    if (meets_caches(t, extents))
      return reject(err, ROPE_ERR_PARAM_INVALID, "a cache overlaps another tensor");
  const int64_t need = compact_workspace(pages);
  if (workspace == nullptr) return reject(err, ROPE_ERR_PARAM_NULLPTR, "workspace is NULL");
  if (workspace_bytes < need || !aligned16(workspace))
    return reject(err, ROPE_ERR_PARAM_INVALID, "workspace too small or not 16-byte aligned");
  for (const rope_tensor *t : {page_table, ref_counts, page_table_out, ref_counts_out, page_map,
                               live})
    if (touches(workspace, need, t))
      return reject(err, ROPE_ERR_PARAM_INVALID, "workspace overlaps a tensor");
  if (in_caches(workspace, need, extents))
    return reject(err, ROPE_ERR_PARAM_INVALID, "workspace overlaps a tensor");

  CompactPlan &p = *plan;
  p.table = table_of(page_table);
  p.out = table_of(page_table_out);
  p.refs = i64(ref_counts);
  p.ref_stride = ref_counts->stride[0];
  p.refs_out = i64_out(ref_counts_out);
  p.ref_out_stride = ref_counts_out->stride[0];
  p.map = i64_out(page_map);
  p.map_stride = page_map->stride[0];
  p.live = i64_out(live);
  p.num_pages = pages;
  p.chunks = (pages + kPageChunk - 1) / kPageChunk;
  p.table_blocks = std::min<int64_t>(1 << 16, (std::max(count(page_table), pages / 2 + 1) +
                                               kPageBlock - 1) / kPageBlock);
  char *w = static_cast<char *>(workspace);
  p.totals = reinterpret_cast<int64_t *>(w);
  w += 256;
  p.moves = reinterpret_cast<int64_t *>(w);
  w += up((pages / 2 + 1) * 16, 256);
  p.counts = reinterpret_cast<int32_t *>(w);
  return ROPE_OK;
}

}  // namespace ropeamd
