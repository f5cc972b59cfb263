// Host check of the paged append's launch plan (rope_append_plan.cpp) with the work-item decode
// that append_paged_kernel applies to it, written out here for the host, and of the latent
// attention plans (rope_latent_plan.cpp) under extreme descriptions.
//
// Append: for each plan every item of every group is walked as a lane would; every element of
// query_out and of every used slot's rows has to be written exactly once, from the input element
// the formulas name, and nothing else; every rotated element has to be paired with its partner
// and its own column of the table.  Both styles, every dtype, vector and element paths, one to
// many heads, slices inside a head, caches that are contiguous, padded, or keep heads before rows,
// slots out of range, the query in place.
//
// All plans: descriptions of random extreme shapes, strides, ranks, types and addresses have to be
// refused, or planned within their limits (grids, 31-bit counts, workspace), without undefined
// behaviour (the sanitizers' run of this program).
//
// No GPU and no tensor data are involved: descriptors carry made-up, suitably aligned addresses.
// Prints "ok <plans> <items> <accepted>" or the first failure; exit status 1 on failure.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <string>
#include <vector>

#include "rope.h"
#include "rope_append_plan.h"
#include "rope_latent_plan.h"

using namespace ropeamd;

#define CHECK(c, ...)                                                    \
  do {                                                                   \
    if (!(c)) {                                                          \
      std::printf("failed %s:%d %s: ", __FILE__, __LINE__, #c);          \
      std::printf(__VA_ARGS__);                                          \
      std::printf("\n");                                                 \
      std::exit(1);                                                      \
    }                                                                    \
  } while (0)

static rope_tensor desc(uintptr_t addr, rope_dtype dt, std::vector<int64_t> shape,
                        std::vector<int64_t> stride = {}) {
  rope_tensor t{};
  t.data = reinterpret_cast<void *>(addr);
  t.dtype = dt;
  t.ndim = int(shape.size());
  int64_t st = 1;
  for (int d = t.ndim - 1; d >= 0; --d) {
    t.shape[d] = shape[size_t(d)];
    t.stride[d] = stride.empty() ? st : stride[size_t(d)];
    st = int64_t(uint64_t(st) * uint64_t(shape[size_t(d)]));
  }
  return t;
}

static int64_t esize(rope_dtype dt) { return dt == ROPE_F32 ? 4 : dt == ROPE_I64 ? 8 : 2; }

static uint32_t div_by(const FastDiv &f, uint32_t n) {
  const uint32_t t = uint32_t((uint64_t(f.m) * n) >> 32);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}

// What an output element is made of: input element, partner (-1: a copy), table column.
struct Source {
  int64_t in, partner, column;
  bool first;
};

struct Shape {
  int64_t T, nq, nk, Dq, D, Dv, rd, q_start, k_start, pages, page;
  int layout;  // 0 contiguous caches, 1 padded rows and pages, 2 heads before rows
  bool in_place, query, value;
};

static int64_t walk(const Shape &s, rope_dtype dt, bool neox, int64_t shift) {
  const int64_t V16 = 16 / esize(dt);
  const uintptr_t base = uintptr_t(1) << 40, step = uintptr_t(1) << 36;
  const uintptr_t off = uintptr_t(shift * esize(dt));
  const rope_tensor pos = desc(base, ROPE_I64, {s.T}), slots = desc(base + step, ROPE_I64, {s.T});
  const rope_tensor q = desc(base + 2 * step + off, dt, {s.T, s.nq, s.Dq});
  const rope_tensor k = desc(base + 3 * step + off, dt, {s.T, s.nk, s.D});
  const rope_tensor v = desc(base + 4 * step + off, dt, {s.T, s.nk, s.Dv});
  const rope_tensor table = desc(base + 5 * step, dt, {100, s.rd});
  const rope_tensor qo = s.in_place ? q : desc(base + 6 * step + off, dt, {s.T, s.nq, s.Dq});
  auto cache = [&](int n, int64_t width) {
    const std::vector<int64_t> shape = {s.pages, s.page, s.nk, width};
    const uintptr_t at = base + uintptr_t(n) * step + off;
    if (s.layout == 0) return desc(at, dt, shape);
    if (s.layout == 1) {
      const int64_t row = s.nk * width + V16;
      return desc(at, dt, shape, {s.page * row + 2 * V16, row, width, 1});
    }
    return desc(at, dt, shape, {s.page * s.nk * width, width, s.page * width, 1});
  };
  const rope_tensor kc = cache(7, s.D), vc = cache(8, s.Dv);
  AppendPlan p;
  std::string err;
  const int st = plan_append(&pos, &slots, s.query ? &q : nullptr, &k, s.value ? &v : nullptr,
                             &table, s.q_start, s.k_start, neox, s.query ? &qo : nullptr, &kc,
                             s.value ? &vc : nullptr, &p, &err);
  CHECK(st == ROPE_OK, "%s", err.c_str());
  if (p.noop) return 0;
  const int64_t V = p.vector_io ? V16 : 1;
  auto slot_of = [&](int64_t t) {  // distinct in range; every fifth token's is out of range
    if (t % 5 == 4) return t % 2 ? int64_t(-1 - t) : s.pages * s.page + t;
    return (t * 11 + 3) % (s.pages * s.page);
  };
  const rope_tensor *ins[3] = {&q, &k, &v}, *outs[3] = {&qo, &kc, &vc};
  const int64_t starts[3] = {s.q_start, s.k_start, 0};
  int64_t items = 0;
  for (int g = 0; g < 3; ++g) {
    const AppendRows &r = p.rows[g];
    std::map<int64_t, Source> seen;  // output offset -> source
    auto put = [&](int64_t out, const Source &src) {
      CHECK(seen.emplace(out, src).second, "group %d: element %lld written twice", g, (long long)out);
    };
    CHECK(r.blocks * kAppendBlock >= r.all, "blocks");
    for (int64_t it = 0; it < r.all; ++it, ++items) {
      int64_t t;
      uint32_t i;
      if (p.idx32) {
        const uint32_t n = div_by(r.div_total, uint32_t(it));
        t = n;
        i = uint32_t(it) - n * r.total;
      } else {
        t = it / r.total;
        i = uint32_t(it - t * r.total);
      }
      const uint32_t h = div_by(r.div_items, i), unit = i - h * r.items;
      const int64_t in = t * r.in_tok + int64_t(h) * r.in_head;
      const bool turn = unit < r.rot_items;
      int64_t e;
      if (turn) {
        e = r.rot_start + int64_t(unit) * (V == 1 && !neox ? 2 : V);
      } else {
        e = int64_t(unit - r.rot_items) * V;
        if (e >= r.rot_start && r.rot_items != 0) e += 2 * p.half;
      }
      const bool pair = neox || V == 1;
      const int64_t partner = neox ? p.half : 1;
      const int64_t slot = g != 0 ? slot_of(t) : 0;
      int64_t out = int64_t(h) * r.out_head;
      if (g == 0) {
        out += t * r.out_tok;
      } else {
        const int64_t page = slot / p.page_size;
        out += page * r.out_page + (slot - page * p.page_size) * r.out_tok;
      }
      if (g != 0 && (slot < 0 || slot >= p.num_slots)) continue;
      for (int64_t m = 0; m < V; ++m) {
        if (!turn) {
          put(out + e + m, {in + e + m, -1, -1, true});
        } else if (pair) {
          const int64_t c = int64_t(unit) * V + m;
          put(out + e + m, {in + e + m, in + e + m + partner, c, true});
          put(out + e + m + partner, {in + e + m + partner, in + e + m, c, false});
        } else {
          const int64_t c = int64_t(unit) * (V / 2) + m / 2;
          put(out + e + m, {in + e + m, in + e + (m ^ 1), c, m % 2 == 0});
        }
      }
    }
    // what has to have been written
    size_t want = 0;
    if ((g == 0 && !s.query) || (g == 2 && !s.value)) {
      CHECK(seen.empty(), "absent group");
      continue;
    }
    const int64_t heads = g == 0 ? s.nq : s.nk, width = ins[g]->shape[2];
    const int64_t rd = g == 2 ? 0 : s.rd, start = starts[g];
    for (int64_t t = 0; t < s.T; ++t) {
      const int64_t slot = g == 0 ? 0 : slot_of(t);
      if (g != 0 && (slot < 0 || slot >= s.pages * s.page)) continue;
      for (int64_t h = 0; h < heads; ++h)
        for (int64_t e = 0; e < width; ++e) {
          const bool turned = e >= start && e < start + rd;
          if (g == 0 && s.in_place && !turned) continue;
          const int64_t in = t * ins[g]->stride[0] + h * ins[g]->stride[1];
          const int64_t out = g == 0 ? t * qo.stride[0] + h * qo.stride[1] + e
                                     : slot / s.page * outs[g]->stride[0] +
                                           slot % s.page * outs[g]->stride[1] +
                                           h * outs[g]->stride[2] + e;
          const auto f = seen.find(out);
          CHECK(f != seen.end(), "group %d token %lld element %lld not written", g, (long long)t,
                (long long)e);
          ++want;
          int64_t other = -1, column = -1;
          bool first = true;
          if (turned) {
            const int64_t x = e - start;
            first = neox ? x < rd / 2 : x % 2 == 0;
            other = in + start + (neox ? (x + rd / 2) % rd : x ^ 1);
            column = neox ? x % (rd / 2) : x / 2;
          }
          const Source &src = f->second;
          CHECK(src.in == in + e && src.partner == other && src.column == column &&
                    src.first == first,
                "group %d token %lld head %lld element %lld", g, (long long)t, (long long)h,
                (long long)e);
        }
    }
    CHECK(want == seen.size(), "group %d: %zu written, %zu wanted", g, seen.size(), want);
  }
  return items;
}

// ---- extreme descriptions ---------------------------------------------------------------------

static std::mt19937_64 rng(1);

static int64_t pick(std::initializer_list<int64_t> of) { return of.begin()[rng() % of.size()]; }

static int64_t wild() {
  switch (rng() % 6) {
    case 0: return int64_t(rng());
    case 1: return int64_t(1) << (rng() % 63);
    case 2: return -(int64_t(1) << (rng() % 63));
    case 3: return INT64_MAX - int64_t(rng() % 3);
    case 4: return INT64_MIN + int64_t(rng() % 3);
    default: return int64_t(rng() % 1000);
  }
}

// A description near a sound one: each number is replaced by a wild one now and then.
static void shake(rope_tensor *t, unsigned odds) {
  for (int d = 0; d < 4; ++d) {
    if (rng() % odds == 0) t->shape[d] = wild();
    if (rng() % odds == 0) t->stride[d] = wild();
  }
  if (rng() % (8 * odds) == 0) t->ndim = int(wild());
  if (rng() % (8 * odds) == 0) t->dtype = rope_dtype(rng() % 4);
  if (rng() % (8 * odds) == 0) t->data = reinterpret_cast<void *>(uintptr_t(wild()));
}

static int64_t fuzz(int64_t rounds) {
  int64_t accepted = 0;
  const uintptr_t base = uintptr_t(1) << 40, step = uintptr_t(1) << 42;
  for (int64_t n = 0; n < rounds; ++n) {
    const unsigned odds = unsigned(pick({4, 20, 100, 1000}));
    const int64_t big = int64_t(1) << (rng() % 32);
    const int64_t T = pick({0, 1, 7, big}), H = pick({0, 1, 16, 128, big}), B = pick({0, 1, 3, big});
    const int64_t L = pick({128, 256, 512}), P = pick({0, 1, 9, big}), S = pick({0, 1, 64, big});
    std::string err;
    {
      rope_tensor q = desc(base, ROPE_BF16, {T, H, L + 64});
      rope_tensor c = desc(base + step, ROPE_BF16, {P, S, L + 64});
      rope_tensor table = desc(base + 2 * step, ROPE_I64, {B, pick({0, 1, 100, big})});
      rope_tensor lens = desc(base + 3 * step, ROPE_I64, {B});
      rope_tensor offs = desc(base + 4 * step, ROPE_I64, {B + 1});
      rope_tensor out = desc(base + 5 * step, ROPE_BF16, {T, H, L});
      rope_tensor lse = desc(base + 6 * step, ROPE_F32, {T, H});
      for (rope_tensor *t : {&q, &c, &table, &lens, &offs, &out, &lse}) shake(t, odds);
      const int64_t bytes = pick({0, int64_t(1) << 30, wild()});
      PagedPlan p;
      if (plan_paged(&q, &c, &table, &lens, rng() % 2 ? &offs : nullptr, L, 0.1, &out,
                     rng() % 2 ? &lse : nullptr, reinterpret_cast<void *>(base + 7 * step), bytes,
                     &p, &err) == ROPE_OK &&
          !p.noop) {
        ++accepted;
        const int64_t rows = 32 * p.row_blocks * p.cluster;
        CHECK(p.clusters > 0 && p.clusters * p.cluster <= kPagedGroups, "clusters");
        CHECK(p.clusters % kXcds == 0, "whole rounds of the XCDs");
        const int64_t steps = (p.max_pages * p.page_size + kPagedStep - 1) / kPagedStep;
        // items of all sequences together, each with its beginning
        const __int128 total = (__int128(p.B) + p.T * p.heads / rows) * (steps + 8);
        CHECK(total < (__int128(1) << 31), "31 bits");
        const char *w = reinterpret_cast<const char *>(base + 7 * step);
        const int64_t end = reinterpret_cast<const char *>(p.parts) - w +
                            2 * int64_t(p.clusters) * p.cluster * 32 * p.row_blocks * p.latent * 4;
        CHECK(end <= bytes && end <= paged_workspace(p.T, p.heads, p.latent, p.B), "workspace");
        CHECK(reinterpret_cast<const char *>(p.stats) - w >=
                  int64_t(p.clusters) * 2 * kJoinWords * 4, "joins");
        CHECK(reinterpret_cast<const char *>(p.parts) - reinterpret_cast<const char *>(p.stats) >=
                  2 * int64_t(p.clusters) * p.cluster * 32 * p.row_blocks * 8, "stats");
      }
    }
    {
      const int64_t dim = pick({64, 128}), Tk = pick({0, 1, 9, big});
      rope_tensor q = desc(base, ROPE_F16, {T, H, dim + 64}), k = desc(base + step, ROPE_F16, {Tk, H, dim});
      rope_tensor kr = desc(base + 2 * step, ROPE_F16, {Tk, 64});
      rope_tensor v = desc(base + 3 * step, ROPE_F16, {Tk, H, dim});
      rope_tensor qo = desc(base + 4 * step, ROPE_I64, {B + 1}), ko = desc(base + 5 * step, ROPE_I64, {B + 1});
      rope_tensor out = desc(base + 6 * step, ROPE_F16, {T, H, dim}), lse = desc(base + 7 * step, ROPE_F32, {T, H});
      rope_tensor grad = desc(base + 8 * step, ROPE_F16, {T, H, dim});
      rope_tensor dq = desc(base + 9 * step, ROPE_F16, {T, H, dim + 64}), dk = desc(base + 10 * step, ROPE_F16, {Tk, H, dim});
      rope_tensor dkr = desc(base + 11 * step, ROPE_F16, {Tk, 64}), dv = desc(base + 12 * step, ROPE_F16, {Tk, H, dim});
      for (rope_tensor *t : {&q, &k, &kr, &v, &qo, &ko, &out, &lse, &grad, &dq, &dk, &dkr, &dv})
        shake(t, 2 * odds);
      const bool offsets = rng() % 2;
      const int64_t bytes = pick({0, int64_t(1) << 42, wild()});
      ExpandedPlan p;
      if (plan_expanded_backward(&grad, &q, &k, &kr, &v, &out, &lse, offsets ? &qo : nullptr,
                                 offsets ? &ko : nullptr, offsets ? 0 : B, 0.1, 1, &dq, &dk, &dkr,
                                 &dv, reinterpret_cast<void *>(base + 13 * step), bytes, &p,
                                 &err) == ROPE_OK &&
          !p.noop) {
        ++accepted;
        CHECK(p.heads * p.q_tiles + kXcds < (int64_t(1) << 31), "grid");
        CHECK(p.heads * p.k_tiles + kXcds < (int64_t(1) << 31), "grid");
        CHECK((p.Tq + p.Tk) * 16 / 256 + 1 < (int64_t(1) << 31), "grid of the shared part");
        const char *w = reinterpret_cast<const char *>(base + 13 * step);
        CHECK(reinterpret_cast<const char *>(p.dkr_part) + p.heads * p.Tk * 64 * 4 - w <= bytes ||
                  p.heads == 0, "workspace");
      }
    }
    {
      const int64_t D = pick({2, 64, 576, big}), rd = pick({2, 64, D}), nk = pick({1, 8, big});
      rope_tensor pos = desc(base, ROPE_I64, {T}), slots = desc(base + step, ROPE_I64, {T});
      rope_tensor q = desc(base + 2 * step, ROPE_F32, {T, H, D}), k = desc(base + 3 * step, ROPE_F32, {T, nk, D});
      rope_tensor v = desc(base + 4 * step, ROPE_F32, {T, nk, D}), t = desc(base + 5 * step, ROPE_F32, {100, rd});
      rope_tensor qo = desc(base + 6 * step, ROPE_F32, {T, H, D});
      rope_tensor kc = desc(base + 7 * step, ROPE_F32, {P, S, nk, D}), vc = desc(base + 8 * step, ROPE_F32, {P, S, nk, D});
      for (rope_tensor *x : {&pos, &slots, &q, &k, &v, &t, &qo, &kc, &vc}) shake(x, odds);
      AppendPlan p;
      if (plan_append(&pos, &slots, &q, &k, &v, &t, rng() % odds == 0 ? wild() : 0,
                      rng() % odds == 0 ? wild() : 0, 1, &qo, &kc, &vc, &p, &err) == ROPE_OK &&
          !p.noop) {
        ++accepted;
        for (const AppendRows &r : p.rows) {
          CHECK(r.all == 0 || (r.all > 0 && r.all == p.T * int64_t(r.total)), "items");
          CHECK(!p.idx32 || r.blocks * kAppendBlock < (int64_t(1) << 32), "32-bit items");
          CHECK(r.rot_start >= 0, "slice");
        }
      }
    }
  }
  return accepted;
}

int main(int argc, char **argv) {
  const int64_t rounds = argc > 1 ? std::atoll(argv[1]) : 200000;
  int64_t plans = 0, items = 0;
  const Shape shapes[] = {
      // T, nq, nk, Dq, D, Dv, rd, q_start, k_start, pages, page, layout, in place, query, value
      {13, 4, 2, 128, 128, 64, 64, 0, 0, 3, 16, 0, false, true, true},
      {13, 4, 2, 96, 128, 64, 64, 32, 64, 3, 16, 1, true, true, true},
      {9, 3, 1, 192, 576, 8, 64, 128, 512, 5, 7, 2, true, true, false},
      {20, 5, 3, 34, 30, 13, 6, 3, 11, 40, 1, 0, false, true, true},
      {20, 5, 3, 34, 30, 13, 30, 4, 0, 7, 5, 2, true, true, true},
      {1, 1, 1, 64, 64, 1, 64, 0, 0, 1, 1, 0, false, false, true},
      {7, 1, 8, 64, 72, 72, 2, 62, 70, 2, 64, 1, false, true, true},
  };
  for (const Shape &s : shapes)
    for (rope_dtype dt : {ROPE_F32, ROPE_F16, ROPE_BF16})
      for (bool neox : {true, false})
        for (int64_t shift : {0, 1}) {
          items += walk(s, dt, neox, shift);
          ++plans;
        }
  const int64_t accepted = fuzz(rounds);
  CHECK(accepted > rounds / 10, "only %lld accepted", (long long)accepted);
  std::printf("ok %lld %lld %lld\n", (long long)plans, (long long)items, (long long)accepted);
  return 0;
}
