// Host checks of single cases of the 8-bit cache's and the page operators' launch plans, each run by its name:
//   append_no_values   values of width 0: nothing of them may be loaded, by any launch form
//   append_long_blocks blocks whose elements of a head pass the kernel's 32-bit numbers: refused
//   fork_layouts       which caches are copied in part: those whose second dimension is a page's tokens or
//                      blocks of them by their form, never others that its length only fits
//   interleaved_caches caches side by side in every page of one allocation: accepted if and only if they share no
//                      byte (against all bytes of small pools), and in a time that grows with their number
//
// No GPU and no tensor data are involved.  Prints "ok" or the first failure.
#include <algorithm>
#include <chrono>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <string>
#include <utility>
#include <vector>

#include "rope.h"
#include "rope_pages_plan.h"
#include "rope_q8_plan.h"

using namespace ropeamd;

#define CHECK(c, ...)                                           \
  do {                                                          \
    if (!(c)) {                                                 \
      std::printf("failed %s:%d %s: ", __FILE__, __LINE__, #c); \
      std::printf(__VA_ARGS__);                                 \
      std::printf("\n");                                        \
      std::exit(1);                                             \
    }                                                           \
  } while (0)

constexpr uintptr_t kBase = uintptr_t(1) << 40, kStep = uintptr_t(1) << 38;

// Contiguous, at a place of its own; empty tensors at address 0, as torch has them.
static rope_tensor desc(int place, rope_dtype dt, std::vector<int64_t> shape) {
  rope_tensor t{};
  t.dtype = dt;
  t.ndim = int(shape.size());
  int64_t st = 1;
  for (int d = t.ndim - 1; d >= 0; --d) {
    t.shape[d] = shape[size_t(d)];
    t.stride[d] = st;
    st *= std::max<int64_t>(shape[size_t(d)], 1);
  }
  bool empty = false;
  for (int64_t n : shape) empty |= n == 0;
  t.data = empty ? nullptr : reinterpret_cast<void *>(kBase + uintptr_t(place) * kStep);
  return t;
}

// A plan for B sequences of `tokens` new tokens each, in blocks of `block`.
static int append_plan(rope_dtype dt, rope_dtype codes, int64_t B, int64_t tokens, int64_t page, int64_t block,
                       int64_t heads, int64_t D, int64_t Dv, int neox, AppendQ8Plan *p, std::string *err) {
  const int64_t T = B * tokens;
  const rope_tensor pos = desc(0, ROPE_I64, {T}), k = desc(1, dt, {T, heads, D}), v = desc(2, dt, {T, heads, Dv});
  const rope_tensor cs = desc(3, dt, {100, 16}), table = desc(4, ROPE_I64, {B, 8}), lens = desc(5, ROPE_I64, {B});
  const rope_tensor kc = desc(6, codes, {9, page, heads, D}), vc = desc(7, codes, {9, page, heads, Dv});
  const rope_tensor ks = desc(8, ROPE_F32, {9, page / block, heads}), vs = desc(9, ROPE_F32, {9, page / block, heads});
  return plan_append_q8(&pos, nullptr, &k, &v, &cs, &table, &lens, nullptr, 0, 0, neox, nullptr, &kc, &vc, &ks, &vs,
                        p, err);
}

static void append_no_values() {
  std::string err;
  for (rope_dtype dt : {ROPE_F32, ROPE_F16, ROPE_BF16})
    for (rope_dtype codes : {ROPE_I8, ROPE_E4M3})
      for (int64_t tokens : {1, 7, 200})
        for (int64_t block : {1, 4, 64})
          for (int neox : {0, 1})
            for (int64_t D : {16, 30, 128, 512}) {
              AppendQ8Plan p;
              const int st = append_plan(dt, codes, 3, tokens, 64, block, 2, D, 0, neox, &p, &err);
              CHECK(st == ROPE_OK, "%s", err.c_str());
              CHECK(p.kv[1].items == 0 && p.kv[1].in == nullptr, "values of width 0");
              // rows side by side are loaded without a look at their number of items
              CHECK(!p.kv[1].side_by_side, "rows without items are loaded");
              CHECK(p.kv[0].items > 0, "keys");
            }
}

static void append_long_blocks() {
  std::string err;
  // the kernel numbers a block's pieces of a head up to block * width, and adds the threads of a workgroup
  const struct {
    int64_t block, D, Dv;
    bool fits;
  } cases[] = {{1 << 22, 128, 128, true},  {1 << 22, 254, 16, true},  {1 << 22, 16, 254, true},
               {1 << 22, 256, 16, false},  {1 << 22, 16, 256, false}, {1 << 24, 128, 128, false},
               {1 << 29, 16, 16, false},   {1 << 25, 16, 0, true},    {1 << 26, 16, 0, false}};
  for (const auto &c : cases)
    for (rope_dtype codes : {ROPE_I8, ROPE_E4M3})
      for (int64_t parts : {1, 2}) {
        if (c.block * parts * 8 >= int64_t(1) << 30) continue;  // tokens of a sequence: refused for that
        AppendQ8Plan p;
        const int st = append_plan(ROPE_BF16, codes, 2, 3, c.block * parts, c.block, 1, c.D, c.Dv, 1, &p, &err);
        CHECK((st == ROPE_OK) == c.fits, "block %lld of %lld and %lld: %d %s", (long long)c.block, (long long)c.D,
              (long long)c.Dv, st, err.c_str());
        if (st == ROPE_OK)
          for (const Q8Rows &r : p.kv)
            CHECK(int64_t(p.block) * std::max<int64_t>(r.dim, r.items) + kQ8Block < (int64_t(1) << 31), "numbers");
      }
}

static void fork_layouts() {
  const int64_t page = 16, P = 20;
  const struct {
    const char *what;
    rope_dtype dt;
    std::vector<int64_t> shape;
    uint32_t parts;  // 0: whole pages
  } cases[] = {{"rows", ROPE_BF16, {P, page, 8, 128}, 16},
               {"codes, as many heads as rows", ROPE_E4M3, {P, page, 16, 128}, 16},
               {"latent rows", ROPE_F16, {P, page, 576}, 16},
               {"scales of blocks of 4", ROPE_F32, {P, 4, 8}, 4},
               {"scales of tokens", ROPE_F32, {P, page, 8}, 16},
               {"scales of pages", ROPE_F32, {P, 1, 8}, 1},
               {"heads outermost", ROPE_BF16, {P, 8, page, 128}, 0},
               {"heads outermost, codes", ROPE_I8, {P, 2, page, 64}, 0},
               {"heads outermost, longer than a page", ROPE_I8, {P, 32, page, 64}, 0},
               {"keys and values in a page", ROPE_BF16, {P, 2, page, 1024}, 0},
               {"keys and values in a page", ROPE_BF16, {P, 2, page * 1024}, 0},
               {"keys' and values' scales of a page", ROPE_F32, {P, 2, 1, 8}, 0},
               {"scales of a page by head", ROPE_F32, {P, 8}, 0},
               {"a page as one dimension", ROPE_F32, {P, page}, 0},
               {"a page as one dimension", ROPE_BF16, {P, page * 8 * 128}, 0},
               {"a number a page", ROPE_I64, {P}, 0}};
  std::string err;
  for (const auto &c : cases) {
    const int64_t B = 3, R = 5, width = 4;
    const rope_tensor table = desc(0, ROPE_I64, {B, width}), lens = desc(1, ROPE_I64, {B});
    const rope_tensor parents = desc(2, ROPE_I64, {R}), refs = desc(3, ROPE_I64, {P});
    const rope_tensor out = desc(4, ROPE_I64, {R, width}), lens_out = desc(5, ROPE_I64, {R});
    const rope_tensor refs_out = desc(6, ROPE_I64, {P}), one = desc(7, ROPE_I64, {1}), cache = desc(8, c.dt, c.shape);
    ForkPlan p;
    std::vector<PageCache> list;
    const int st = plan_fork_pages(&table, &lens, &parents, nullptr, &refs, page, &cache, 1, &out, &lens_out,
                                   &refs_out, &one, reinterpret_cast<void *>(kBase + 20 * kStep),
                                   fork_workspace(B, R, P), &p, &list, &err);
    CHECK(st == ROPE_OK && list.size() == 1, "%s: %s", c.what, err.c_str());
    const PageRun &r = list[0].run;
    CHECK(r.parts == c.parts || (c.parts == 1 && r.parts == 0), "%s: %u parts", c.what, r.parts);
    CHECK(r.parts == 0 || r.parts * r.part_words == r.vecs, "%s: %u words of %u", c.what, r.part_words, r.vecs);
  }
}

// The plan of a copy of no page in `caches`; 0 if they are refused.
static int accepted(const std::vector<rope_tensor> &caches, std::string *err) {
  const rope_tensor src = desc(0, ROPE_I64, {3}), dst = desc(1, ROPE_I64, {3});
  CopyPagesPlan p;
  std::vector<PageCache> list;
  return plan_copy_pages(&src, &dst, caches.data(), int64_t(caches.size()), &p, &list, err) == ROPE_OK;
}

static rope_tensor slice(uintptr_t at, rope_dtype dt, int64_t pages, int64_t stride, int64_t elements) {
  rope_tensor t{};
  t.data = reinterpret_cast<void *>(at);
  t.dtype = dt;
  t.ndim = 2;
  t.shape[0] = pages;
  t.shape[1] = elements;
  t.stride[0] = stride;
  t.stride[1] = 1;
  return t;
}

static void interleaved_caches() {
  std::mt19937_64 rng(7);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + int64_t(rng() % uint64_t(hi - lo + 1)); };
  std::string err;
  int64_t apart = 0, meeting = 0;
  const uintptr_t base = kBase + 2 * kStep;
  for (int round = 0; round < 20000; ++round) {
    // a record of every page, in it blocks one behind the other, some of them moved or longer by a few bytes
    const int64_t pages = pick(1, 4), n = pick(1, 6), pools = pick(1, 2);
    std::vector<rope_tensor> caches;
    for (int64_t pool = 0; pool < pools; ++pool) {
      std::vector<std::pair<int64_t, int64_t>> blocks;  // where, bytes
      int64_t at = 0;
      for (int64_t i = 0; i < n; ++i) {
        const int64_t bytes = 4 * pick(1, 5);
        blocks.push_back({at, bytes});
        at += bytes + 4 * pick(0, 1);
      }
      if (pick(0, 3) == 0) at -= 4 * pick(0, 2);  // the next page's record begins in this one
      if (pick(0, 3) == 0) blocks[size_t(pick(0, n - 1))].first += 4 * pick(0, 3);
      const int64_t stride = std::max<int64_t>(at, 4) * (pick(0, 5) == 0 ? 2 : 1);
      for (auto &b : blocks) {
        const int64_t own = pick(0, 9) == 0 ? stride * 2 : stride;
        if (b.second > own) b.second = own;
        const rope_dtype dt = pick(0, 1) ? ROPE_F32 : ROPE_I8;
        const int64_t es = dt == ROPE_F32 ? 4 : 1;
        caches.push_back(slice(base + uintptr_t(pool * pick(0, 400) * 4 + b.first), dt, pages, own / es, b.second / es));
      }
    }
    std::shuffle(caches.begin(), caches.end(), rng);
    std::vector<int> held(8192);
    bool overlap = false;
    for (const rope_tensor &t : caches) {
      const int64_t es = t.dtype == ROPE_F32 ? 4 : 1, from = int64_t(reinterpret_cast<uintptr_t>(t.data) - base);
      for (int64_t p = 0; p < pages; ++p)
        for (int64_t b = 0; b < t.shape[1] * es; ++b) overlap |= held[size_t(from + p * t.stride[0] * es + b)]++ != 0;
    }
    const bool ok = accepted(caches, &err);
    CHECK(!(ok && overlap), "round %d: caches that overlap are accepted", round);
    (overlap ? meeting : apart) += 1;
  }
  CHECK(apart > 1000 && meeting > 1000, "%lld apart, %lld not", (long long)apart, (long long)meeting);
  // layers' keys, values and scales of every page one behind the other, and two such pools, in any order
  for (int64_t layers : {1, 4, 32, 16384}) {
    std::vector<rope_tensor> caches;
    const int64_t part = 4096, record = layers * 2 * (part + 64), pools = layers > 1000 ? 1 : 2;
    for (int64_t pool = 0; pool < pools; ++pool)
      for (int64_t i = 0; i < 2 * layers; ++i) {
        const uintptr_t at = base + uintptr_t(pool * (record * 50 + 12345 * 4));
        caches.push_back(slice(at + uintptr_t(i * part), ROPE_I8, 50, record, part));
        caches.push_back(slice(at + uintptr_t(2 * layers * part + i * 64), ROPE_F32, 50, record / 4, 16));
      }
    std::shuffle(caches.begin(), caches.end(), rng);
    const auto begin = std::chrono::steady_clock::now();
    CHECK(accepted(caches, &err), "%lld layers: %s", (long long)layers, err.c_str());
    const double s = std::chrono::duration<double>(std::chrono::steady_clock::now() - begin).count();
    CHECK(s < 5, "%lld caches took %.1f s", (long long)caches.size(), s);  // compared in pairs: 40 s and more
    for (int k = 0; k < 20; ++k) {  // one of them a byte off
      std::vector<rope_tensor> moved = caches;
      rope_tensor &t = moved[size_t(pick(0, int64_t(moved.size()) - 1))];
      if (t.dtype != ROPE_I8) continue;
      t.data = static_cast<char *>(t.data) + (k % 2 ? 1 : -1);
      if (layers < 1000) CHECK(!accepted(moved, &err), "one byte of two caches");
    }
  }
}

int main(int argc, char **argv) {
  const struct {
    const char *name;
    void (*run)();
  } checks[] = {{"append_no_values", append_no_values},
                {"append_long_blocks", append_long_blocks},
                {"fork_layouts", fork_layouts},
                {"interleaved_caches", interleaved_caches}};
  for (const auto &c : checks)
    if (argc > 1 && std::strcmp(argv[1], c.name) == 0) {
      c.run();
      std::printf("ok\n");
      return 0;
    }
  std::printf("no such check\n");
  return 1;
}
