// Host check of the 8-bit cache's launch plans (rope_q8_plan.cpp) with the device's walks over them written
// out here, and of all its and the page operators' plans under extreme descriptions.
//
// Append: every place of a plan is taken as a wavefront would; each block of each sequence's new tokens has to
// be found exactly once, under either numbering.
// Attention: the shares of all workgroups are walked; every step of every tile has to be taken once, every
// part has to lie where the joining kernel looks for it, and the cost has to fit what the plan says.
// All plans: descriptions of random extreme shapes, strides, ranks, types and addresses have to be refused, or
// planned within their limits, without undefined behaviour (the sanitizers' run of this program).
//
// No GPU and no tensor data are involved.  Prints "ok <places> <pieces> <accepted>" or the first failure.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <string>
#include <tuple>
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

static rope_tensor desc(uintptr_t addr, rope_dtype dt, std::vector<int64_t> shape) {
  rope_tensor t{};
  t.data = reinterpret_cast<void *>(addr);
  t.dtype = dt;
  t.ndim = int(shape.size());
  int64_t st = 1;
  for (int d = t.ndim - 1; d >= 0; --d) {
    t.shape[d] = shape[size_t(d)];
    t.stride[d] = st;
    st *= shape[size_t(d)];
  }
  return t;
}

static uint32_t div_by(const FastDiv &f, uint32_t n) {
  const uint32_t t = uint32_t((uint64_t(f.m) * n) >> 32);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}

static std::mt19937_64 rng(1);
static int64_t pick(int64_t lo, int64_t hi) { return lo + int64_t(rng() % uint64_t(hi - lo + 1)); }

constexpr uintptr_t kBase = uintptr_t(1) << 40, kStep = uintptr_t(1) << 36;

// ---- append ------------------------------------------------------------------------------------------
static int64_t walk_append() {
  const int64_t B = pick(1, 9), block = int64_t(1) << pick(0, 6), page = block * pick(1, 4);
  const int64_t heads = pick(1, 9), D = 16 * pick(1, 9), max_pages = pick(1, 6);
  const bool even = pick(0, 3) == 0;
  const int64_t each = pick(0, 1) ? pick(0, 3) : pick(0, 200);
  std::vector<int64_t> offsets = {even ? 0 : pick(0, 3)}, lens;
  for (int64_t b = 0; b < B; ++b) {
    const int64_t n = even ? each : pick(0, 2) ? pick(0, each) : 0;
    offsets.push_back(offsets.back() + n);
    lens.push_back(pick(0, 3) ? n + pick(0, 100) : pick(0, 2 * n));
  }
  const int64_t T = offsets.back() + (even ? 0 : pick(0, 3));
  if (T == 0) return 0;
  const rope_tensor pos = desc(kBase, ROPE_I64, {T}), k = desc(kBase + kStep, ROPE_F16, {T, heads, D});
  const rope_tensor v = desc(kBase + 2 * kStep, ROPE_F16, {T, heads, D});
  const rope_tensor cs = desc(kBase + 3 * kStep, ROPE_F16, {100, 16});
  const rope_tensor table = desc(kBase + 4 * kStep, ROPE_I64, {B, max_pages});
  const rope_tensor lt = desc(kBase + 5 * kStep, ROPE_I64, {B}), ot = desc(kBase + 6 * kStep, ROPE_I64, {B + 1});
  const rope_tensor kc = desc(kBase + 7 * kStep, ROPE_I8, {50, page, heads, D});
  const rope_tensor vc = desc(kBase + 8 * kStep, ROPE_I8, {50, page, heads, D});
  const rope_tensor ks = desc(kBase + 9 * kStep, ROPE_F32, {50, page / block, heads});
  const rope_tensor vs = desc(kBase + 10 * kStep, ROPE_F32, {50, page / block, heads});
  AppendQ8Plan p;
  std::string err;
  const int st = plan_append_q8(&pos, nullptr, &k, &v, &cs, &table, &lt, even ? nullptr : &ot, 0, 0, 1, nullptr,
                                &kc, &vc, &ks, &vs, &p, &err);
  CHECK(st == ROPE_OK, "%s", err.c_str());
  const int64_t units = kQ8Block / std::max(64, p.lanes);
  CHECK(p.kv_blocks * units >= p.places * p.head_groups, "too few wavefronts");
  CHECK(p.head_groups / 2 * std::max(1, 64 / p.lanes) >= heads, "heads left out");
  // wavefronts that meet are of one place, its keys or its values
  CHECK(p.lanes <= 64 || p.head_groups / 2 % units == 0, "a workgroup of keys and values");
  std::map<std::pair<int64_t, int64_t>, std::pair<int64_t, int64_t>> found;  // (b, block) -> first token, count
  auto first_place = [&](int64_t offset, int64_t i) {
    return p.by_token ? offset : int64_t(div_by(p.div_block, uint32_t(offset))) + 2 * i;
  };
  for (int64_t u = 0; u < p.places; ++u) {
    int64_t b = 0;
    while (b + 1 < B && first_place(offsets[size_t(b + 1)], b + 1) <= u) ++b;
    const int64_t o0 = offsets[size_t(b)], n = offsets[size_t(b + 1)] - o0;
    const int64_t len = std::min(lens[size_t(b)], max_pages * page);
    const int64_t start = len - n, first = std::max<int64_t>(start, 0), k0 = u - first_place(o0, b);
    if (n <= 0 || len <= first || k0 < 0) continue;
    int64_t lo;
    if (p.by_token) {
      lo = start + k0;
      const bool begins = lo == first || (lo > first && lo % block == 0);
      if (k0 >= n || !begins) continue;
    } else {
      lo = std::max(first, (first / block + k0) * block);
      if (lo >= len) continue;
    }
    const int64_t begin = lo / block * block, count = std::min(len, begin + block) - lo;
    CHECK(found.emplace(std::make_pair(b, begin), std::make_pair(o0 + lo - start, count)).second,
          "a block taken twice: sequence %lld", (long long)b);
  }
  size_t want = 0;
  for (int64_t b = 0; b < B; ++b) {
    const int64_t o0 = offsets[size_t(b)], n = offsets[size_t(b + 1)] - o0;
    const int64_t len = std::min(lens[size_t(b)], max_pages * page), start = len - n;
    for (int64_t at = std::max<int64_t>(start, 0); at < len;) {
      const int64_t begin = at / block * block, end = std::min(len, begin + block);
      const auto f = found.find({b, begin});
      CHECK(f != found.end() && f->second.first == o0 + at - start && f->second.second == end - at,
            "sequence %lld's block %lld left out", (long long)b, (long long)begin);
      ++want;
      at = end;
    }
  }
  CHECK(found.size() == want, "blocks of no sequence");
  return p.places;
}

// ---- attention ---------------------------------------------------------------------------------------
constexpr int32_t kItemCost = 2;

struct Sequence {
  int32_t len, first, count, tiles, cost;
};

struct Walk {
  const AttnQ8Plan &p;
  int32_t rows;
  int32_t visible(const Sequence &s, int32_t tile) const {
    const int32_t all = s.count * p.group;
    const int32_t tok = int32_t(div_by(p.div_group, uint32_t(std::min((tile + 1) * rows, all) - 1)));
    return std::max(0, s.len - s.count + 1 + tok);
  }
  int32_t steps(const Sequence &s, int32_t tile) const {
    return std::max(1, (visible(s, tile) + (1 << p.step_log2) - 1) >> p.step_log2);
  }
  Sequence sequence(int64_t len, int64_t first, int64_t count) const {
    Sequence s = {int32_t(len), int32_t(first), int32_t(count), 0, 0};
    s.tiles = (std::max(s.count, 0) * p.group + rows - 1) / rows;
    if (s.tiles > 0) {
      s.cost = steps(s, s.tiles - 1) + kItemCost;
      if (s.tiles > 1) s.cost += steps(s, 0) + kItemCost + (rows >> p.step_log2) + 2;
    }
    return s;
  }
};

static int64_t walk_attention() {
  const int64_t B = pick(1, 12), N = pick(1, 8), group = pick(1, 12), D = 64 << pick(0, 2);
  const int64_t page = int64_t(16) << pick(0, 2);
  std::vector<int64_t> lens, counts;
  int64_t T = 0;
  const int64_t most = pick(0, 1) ? 1 : pick(0, 1) ? 6 : 700;
  for (int64_t b = 0; b < B; ++b) {
    counts.push_back(pick(0, 4) ? pick(0, most) : 0);
    lens.push_back(pick(0, 3) ? pick(0, 200) + counts.back() : pick(0, 1) ? pick(0, 40000) : 0);
    T += counts.back();
  }
  if (T == 0) return 0;
  const int64_t max_pages = 40000 / page + 60;
  const rope_tensor q = desc(kBase, ROPE_BF16, {T, N * group, D}), out = desc(kBase + kStep, ROPE_BF16, {T, N * group, D});
  const rope_tensor kc = desc(kBase + 2 * kStep, ROPE_I8, {50, page, N, D}), vc = desc(kBase + 3 * kStep, ROPE_I8, {50, page, N, D});
  const rope_tensor ks = desc(kBase + 4 * kStep, ROPE_F32, {50, 1, N}), vs = desc(kBase + 5 * kStep, ROPE_F32, {50, 1, N});
  const rope_tensor table = desc(kBase + 6 * kStep, ROPE_I64, {B, max_pages}), lt = desc(kBase + 7 * kStep, ROPE_I64, {B});
  const rope_tensor ot = desc(kBase + 8 * kStep, ROPE_I64, {B + 1});
  const int64_t need = attention_q8_workspace(T, N * group, N, D, B);
  AttnQ8Plan p;
  std::string err;
  const int st = plan_attention_q8(&q, &kc, &vc, &ks, &vs, &table, &lt, &ot, 0.1, &out, nullptr,
                                   reinterpret_cast<void *>(kBase + 9 * kStep), need, &p, &err);
  CHECK(st == ROPE_OK, "%s", err.c_str());
  const char *end = reinterpret_cast<const char *>(p.parts + int64_t(p.groups) * 2 * p.abreast * p.rows * D);
  CHECK(end <= reinterpret_cast<const char *>(kBase + 9 * kStep) + need, "workspace");
  CHECK(p.head_sets * p.abreast == N, "sets");
  const Walk w = {p, p.rows};
  std::vector<Sequence> s;
  int64_t total = 0, first = 0;
  for (int64_t b = 0; b < B; ++b) {
    s.push_back(w.sequence(std::min(lens[size_t(b)], max_pages * page), first, counts[size_t(b)]));
    first += counts[size_t(b)];
    total += int64_t((s.back().tiles + 1) / 2) * p.head_sets * s.back().cost;
  }
  CHECK(!p.small || total < (int64_t(1) << 31), "cost %lld", (long long)total);
  const int64_t per = (total + p.groups - 1) / p.groups;
  using Tile = std::tuple<int64_t, int32_t, int32_t>;  // sequence, set, tile
  std::map<Tile, std::vector<std::pair<int32_t, int32_t>>> taken;
  std::map<std::pair<int64_t, int>, Tile> slots;  // workgroup, part -> tile
  struct Record {
    int64_t n, first, part;
  };
  std::map<Tile, std::vector<Record>> records;
  int64_t pieces = 0;
  for (int64_t me = 0; me < p.groups; ++me) {
    const int64_t w0 = me * per, w1 = std::min(total, w0 + per);
    if (w0 >= total) continue;
    int64_t at = w0, b = 0, before = 0;
    while (true) {
      const int64_t cost = int64_t((s[size_t(b)].tiles + 1) / 2) * p.head_sets * s[size_t(b)].cost;
      if (w0 < before + cost) break;
      before += cost;
      ++b;
    }
    int64_t item = (w0 - before) / s[size_t(b)].cost, x = (w0 - before) % s[size_t(b)].cost;
    while (at < w1) {
      const Sequence &q1 = s[size_t(b)];
      const int32_t pair = int32_t(item / p.head_sets), set = int32_t(item % p.head_sets);
      int32_t tile = q1.tiles - 1 - pair;
      int64_t from = 0, to = q1.cost;
      if (tile != pair) {
        const int64_t border = w.steps(q1, tile) + kItemCost;
        if (x < border) {
          to = border;
        } else {
          from = border;
          tile = pair;
        }
      }
      const int32_t steps = w.steps(q1, tile);
      CHECK(from + kItemCost + steps <= to, "a pair costs more than its share");
      const int64_t begin = at - (x - from), x1 = std::min(to, x + (w1 - at));
      const int32_t st0 = int32_t(std::min<int64_t>(std::max<int64_t>(0, x - from - kItemCost), steps));
      const int32_t st1 = int32_t(std::min<int64_t>(std::max<int64_t>(0, x1 - from - kItemCost), steps));
      const int part = at == w0 ? 0 : 1;
      at += x1 - x;
      x = x1;
      if (st0 < st1) {
        ++pieces;
        const Tile key = {b, set, tile};
        taken[key].push_back({st0, st1});
        if (!(st0 == 0 && st1 == steps)) {
          CHECK(slots.emplace(std::make_pair(me, part), key).second, "a slot written twice");
          const int64_t f = begin + kItemCost, g0 = f / per;
          records[key].push_back({(f + steps - 1) / per - g0 + 1, g0, begin <= g0 * per ? 0 : 1});
        }
      }
      if (at < w1 && x >= q1.cost) {
        x = 0;
        if (++item >= int64_t((q1.tiles + 1) / 2) * p.head_sets) {
          item = 0;
          do {
            ++b;
            CHECK(b < B, "past the last sequence");
          } while (s[size_t(b)].tiles == 0);
        }
      }
    }
  }
  for (int64_t b = 0; b < B; ++b)
    for (int32_t set = 0; set < p.head_sets; ++set)
      for (int32_t tile = 0; tile < s[size_t(b)].tiles; ++tile) {
        const Tile key = {b, set, tile};
        auto &t = taken[key];
        std::sort(t.begin(), t.end());
        int32_t next = 0;
        for (const auto &r : t) {
          CHECK(r.first == next, "steps of a tile left out or taken twice");
          next = r.second;
        }
        CHECK(next == w.steps(s[size_t(b)], tile), "steps at a tile's end left out");
        if (t.size() == 1) continue;
        CHECK(records[key].size() == t.size(), "parts without records");
        for (const Record &r : records[key]) {
          CHECK(r.n == int64_t(t.size()), "a record counts %lld parts of %zu", (long long)r.n, t.size());
          for (int64_t k = 0; k < r.n; ++k) {
            const auto f = slots.find({r.first + k, k == 0 ? int(r.part) : 0});
            CHECK(f != slots.end() && f->second == key, "a part lies elsewhere");
          }
        }
      }
  CHECK(taken.size() == size_t([&] {
          size_t n = 0;
          for (const Sequence &x : s) n += size_t(x.tiles) * size_t(p.head_sets);
          return n;
        }()), "tiles of no sequence");
  return pieces;
}

// ---- extremes ----------------------------------------------------------------------------------------
static int64_t extreme() {
  static const int64_t values[] = {0, 1, 2, 3, 7, 16, 64, 100, 128, 256, 257, 4096, (1 << 24) - 1, 1 << 24,
                                   (1 << 30) - 1, 1 << 30, int64_t(1) << 31, int64_t(1) << 32,
                                   int64_t(1) << 40, int64_t(1) << 52, int64_t(1) << 53, int64_t(1) << 62,
                                   INT64_MAX, -1, INT64_MIN};
  return values[rng() % (sizeof(values) / sizeof(values[0]))];
}

// A sensible description with some of its numbers replaced.
static rope_tensor bend(rope_tensor t) {
  const int n = int(rng() % 3);
  for (int i = 0; i < n; ++i) {
    switch (rng() % 6) {
      case 0: t.shape[rng() % 4] = extreme(); break;
      case 1: t.stride[rng() % 4] = extreme(); break;
      case 2: t.ndim = int(rng() % 7) - 1; break;
      case 3: t.dtype = rope_dtype(rng() % 6); break;
      case 4: t.data = reinterpret_cast<void *>(rng() % 3 ? uintptr_t(t.data) + rng() % 16 : rng()); break;
      default: t.data = rng() % 4 ? t.data : nullptr;
    }
  }
  return t;
}

static int64_t extremes() {
  const int64_t T = pick(0, 40), B = pick(0, 9), N = pick(0, 8), G = pick(1, 4), D = 64 << pick(0, 2);
  const int64_t page = pick(0, 40), pages = pick(0, 99), width = pick(0, 9), R = pick(0, 9);
  int n = 0;
  auto make = [&](rope_dtype dt, std::vector<int64_t> shape) { return bend(desc(kBase + uintptr_t(n++) * kStep, dt, shape)); };
  const rope_tensor pos = make(ROPE_I64, {T}), q = make(ROPE_BF16, {T, N * G, D}), k = make(ROPE_BF16, {T, N, D});
  const rope_tensor v = make(ROPE_BF16, {T, N, D}), cs = make(ROPE_BF16, {100, 32}), qo = make(ROPE_BF16, {T, N * G, D});
  const rope_tensor table = make(ROPE_I64, {B, width}), lens = make(ROPE_I64, {B}), off = make(ROPE_I64, {B + 1});
  const rope_tensor kc = make(ROPE_E4M3, {pages, page, N, D}), vc = make(ROPE_E4M3, {pages, page, N, D});
  const rope_tensor ks = make(ROPE_F32, {pages, std::min<int64_t>(page, 1), N}), vs = make(ROPE_F32, {pages, std::min<int64_t>(page, 1), N});
  const rope_tensor lse = make(ROPE_F32, {T, N * G});
  auto maybe = [&](const rope_tensor &t) { return rng() % 30 ? &t : nullptr; };
  int64_t accepted = 0;
  std::string err;
  {
    AppendQ8Plan p;
    const int st = plan_append_q8(maybe(pos), maybe(q), maybe(k), maybe(v), maybe(cs), maybe(table), maybe(lens),
                                  rng() % 2 ? &off : nullptr, rng() % 9 ? 0 : extreme(), rng() % 9 ? 0 : extreme(),
                                  int(rng() % 2), maybe(qo), maybe(kc), maybe(vc), maybe(ks), maybe(vs), &p, &err);
    if (st == ROPE_OK && !p.noop) {
      ++accepted;
      CHECK(p.kv_blocks >= 0 && p.query_blocks >= 0 && p.places >= 0 && p.head_groups > 0, "append");
      CHECK(p.kv_blocks < (int64_t(1) << 56) && p.query_blocks < (int64_t(1) << 56), "append grid");
    }
  }
  {
    AttnQ8Plan p;
    const int64_t need = rng() % 9 ? attention_q8_workspace(T, N * G, N, D, B) : extreme();
    attention_q8_workspace(extreme(), extreme(), extreme(), extreme(), extreme());
    const int st = plan_attention_q8(maybe(q), maybe(kc), maybe(vc), maybe(ks), maybe(vs), maybe(table), maybe(lens),
                                     rng() % 2 ? &off : nullptr, rng() % 9 ? 0.1 : double(extreme()), maybe(qo),
                                     maybe(lse), rng() % 30 ? reinterpret_cast<void *>(kBase + 60 * kStep) : nullptr,
                                     need, &p, &err);
    if (st == ROPE_OK && !p.noop) {
      ++accepted;
      CHECK(p.groups > 0 && p.groups <= 1024 && p.head_sets > 0 && p.rows >= 16, "attention");
    }
  }
  const rope_tensor src = make(ROPE_I64, {R}), dst = make(ROPE_I64, {R}), refs = make(ROPE_I64, {pages});
  const rope_tensor out = make(ROPE_I64, {R, width}), lo = make(ROPE_I64, {R}), ro = make(ROPE_I64, {pages});
  const rope_tensor one = make(ROPE_I64, {1}), map = make(ROPE_I64, {pages}), to = make(ROPE_I64, {B, width});
  const rope_tensor list[4] = {kc, vc, ks, vs};
  const int64_t caches = rng() % 20 ? pick(0, 4) : extreme() < 0 ? -1 : 4;
  std::vector<PageCache> left;
  auto units = [&](const std::vector<PageCache> &l) {
    PageCaches c;
    for (size_t at = 0; at < l.size();) {
      at = take_caches(l, at, kPageWords, &c);
      CHECK(c.units(1) >= 0 && c.units(1) < (int64_t(1) << 56), "units");
    }
  };
  {
    CopyPagesPlan p;
    if (plan_copy_pages(maybe(src), maybe(dst), list, caches, &p, &left, &err) == ROPE_OK) ++accepted, units(left);
  }
  left.clear();
  {
    ForkPlan p;
    fork_workspace(extreme(), extreme(), extreme());
    const int64_t need = rng() % 9 ? fork_workspace(B, R, pages) : extreme();
    if (plan_fork_pages(maybe(table), maybe(lens), maybe(src), rng() % 2 ? &dst : nullptr, maybe(refs),
                        rng() % 9 ? page : extreme(), list, caches, maybe(out), maybe(lo), maybe(ro), maybe(one),
                        reinterpret_cast<void *>(kBase + 60 * kStep), need, &p, &left, &err) == ROPE_OK) {
      ++accepted;
      CHECK(p.table_blocks >= 1 && p.table_blocks <= 65536 && p.chunks >= 0, "fork");
      units(left);
    }
  }
  left.clear();
  {
    CompactPlan p;
    compact_workspace(extreme());
    const int64_t need = rng() % 9 ? compact_workspace(pages) : extreme();
    if (plan_compact_pages(maybe(table), maybe(refs), list, caches, maybe(to), maybe(ro), maybe(map), maybe(one),
                           reinterpret_cast<void *>(kBase + 60 * kStep), need, &p, &left, &err) == ROPE_OK) {
      ++accepted;
      CHECK(p.table_blocks >= 1 && p.table_blocks <= 65536 && p.chunks >= 0, "compact");
      units(left);
    }
  }
  return accepted;
}

int main(int argc, char **argv) {
  const int64_t rounds = argc > 1 ? std::atoll(argv[1]) : 2000;
  int64_t places = 0, pieces = 0, accepted = 0;
  for (int64_t i = 0; i < rounds; ++i) places += walk_append();
  for (int64_t i = 0; i < rounds / 4; ++i) pieces += walk_attention();
  for (int64_t i = 0; i < rounds * 20; ++i) accepted += extremes();
  CHECK(places > 0 && pieces > 0 && accepted > rounds, "nothing checked: %lld", (long long)accepted);
  std::printf("ok %lld %lld %lld\n", (long long)places, (long long)pieces, (long long)accepted);
}
