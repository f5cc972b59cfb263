// Host checks of single cases of the 8-bit cache's and the page operators' launch plans, each run by its name:
//   append_no_values   values of width 0: nothing of them may be loaded, by any launch form
//   append_long_blocks blocks whose elements of a head pass the kernel's 32-bit numbers: refused
//   fork_layouts       which caches are copied in part: those whose second dimension is a page's tokens or
//                      blocks of them by their form, never others that its length only fits
//
// No GPU and no tensor data are involved.  Prints "ok" or the first failure.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>
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

int main(int argc, char **argv) {
  const struct {
    const char *name;
    void (*run)();
  } checks[] = {{"append_no_values", append_no_values},
                {"append_long_blocks", append_long_blocks},
                {"fork_layouts", fork_layouts}};
  for (const auto &c : checks)
    if (argc > 1 && std::strcmp(argv[1], c.name) == 0) {
      c.run();
      std::printf("ok\n");
      return 0;
    }
  std::printf("no such check\n");
  return 1;
}
