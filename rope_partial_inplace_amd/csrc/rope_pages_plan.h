// rope_pages_plan.h -- launch plans of the operators on a cache's pages (library-internal).
#pragma once

#include <cstdint>
#include <string>
#include <vector>

#include "rope.h"
#include "rope_plan.h"

namespace ropeamd {

// Caches whose pages are alike: `vecs` words of 2^width bytes each.  Where a page's outermost dimension
// is its tokens (or blocks of them), the first tokens of a page are its first words: part_words of them
// for each of `parts` equal parts of a page's tokens.
//
// A run's work is numbered cache by cache, in it move by move, in that piece by piece (move by move and
// then cache by cache, 500 pages of 16 KiB in 64 caches took 207 us in place of 175).  Pages of at least
// 64 words are cut into pieces that a wavefront copies, so that its page numbers are scalars; of
// smaller ones a wavefront takes several, 2^lanes_log2 lanes each.
struct PageRun {
  int32_t first = 0, count = 0;  // caches
  uint32_t vecs = 0, pieces = 1, part_words = 0, parts = 0;
  int32_t width = 0, lanes_log2 = 6;
  FastDiv div_pieces;
};

constexpr int kPageBlock = 64;  // threads of a copying workgroup
constexpr int kPageWords = 2;  // words of a lane
constexpr int kForkWords = 8;  // the same where the way to a word is longer
constexpr int64_t kPageChunk = 4096;  // pages that a workgroup counts
constexpr int kCountBlock = 1024;

// What a launch copies between.
constexpr int kPageCaches = 160;
constexpr int kPageRuns = 4;
struct PageCaches {
  int32_t runs = 0, count = 0;
  PageRun run[kPageRuns];
  char *base[kPageCaches];
  int64_t page[kPageCaches];  // bytes from one page to the next
  // wavefronts that `moves` moves take
  int64_t units(int64_t moves) const {
    int64_t n = 0;
    for (int r = 0; r < runs; ++r) {
      const int64_t per = int64_t(1) << (6 - run[r].lanes_log2);
      n += (moves * run[r].count * run[r].pieces + per - 1) / per;
    }
    return n;
  }
};

// A cache as the checks leave it.
struct PageCache {
  PageRun run;
  char *base = nullptr;
  int64_t page = 0;
};

// As many of the caches from `at` on as a launch takes, in pieces of `words` words a lane; returns where
// the next launch's begin.
size_t take_caches(const std::vector<PageCache> &list, size_t at, int words, PageCaches *to);

// ---- copy ------------------------------------------------------------------------------------------
struct CopyPagesPlan {
  PageCaches caches;
  const int64_t *sources = nullptr, *targets = nullptr;
  int64_t source_stride = 0, target_stride = 0, moves = 0, num_pages = 0;
  int64_t table_blocks = 0;  // no tables to write
};

// ---- fork and compact ------------------------------------------------------------------------------
struct PageTable {
  int64_t *data = nullptr;
  int64_t rows = 0, width = 0, row = 0, col = 0;  // sizes and strides
};

struct ForkPlan {
  PageCaches caches;
  PageTable table, out;
  const int64_t *lens = nullptr, *parents = nullptr, *grow = nullptr, *refs = nullptr;
  int64_t *lens_out = nullptr, *refs_out = nullptr, *shortage = nullptr;
  int64_t len_stride = 0, parent_stride = 0, grow_stride = 0, ref_stride = 0, len_out_stride = 0,
          ref_out_stride = 0;
  int64_t num_pages = 0, page_size = 1;
  int64_t chunks = 0;
  int64_t table_blocks = 0;  // workgroups of the last launch that write tables and holds
  // workspace
  int64_t *totals = nullptr;  // pages wanted, copies, free pages
  int32_t *first = nullptr, *children = nullptr, *kept = nullptr;  // [B]
  int64_t *base = nullptr;    // [R] rank of the row's first new page
  int64_t *copies = nullptr;  // [R][3] source page, rank of the target, tokens
  int32_t *counts = nullptr;  // [chunks] free pages
  int32_t *free = nullptr;    // [pages] free pages in order, as many as are wanted
};

struct CompactPlan {
  PageCaches caches;
  PageTable table, out;
  const int64_t *refs = nullptr;
  int64_t *refs_out = nullptr, *map = nullptr, *live = nullptr;
  int64_t ref_stride = 0, ref_out_stride = 0, map_stride = 0;
  int64_t num_pages = 0, chunks = 0, table_blocks = 0;
  // workspace
  int64_t *totals = nullptr;  // moves
  int64_t *moves = nullptr;   // [pages / 2 + 1][2] from, to
  int32_t *counts = nullptr;  // [chunks] pages in use
};

int64_t fork_workspace(int64_t sequences, int64_t rows, int64_t pages);
int64_t compact_workspace(int64_t pages);

// The plans hold no caches: those follow in `caches`, checked, kPageCaches at a time for a launch.
int plan_copy_pages(const rope_tensor *sources, const rope_tensor *targets,
                    const rope_tensor *caches, int64_t num_caches, CopyPagesPlan *plan,
                    std::vector<PageCache> *list, std::string *err);
int plan_fork_pages(const rope_tensor *page_table, const rope_tensor *seq_lens,
                    const rope_tensor *parents, const rope_tensor *grow,
                    const rope_tensor *ref_counts, int64_t page_size, const rope_tensor *caches,
                    int64_t num_caches, const rope_tensor *page_table_out,
                    const rope_tensor *seq_lens_out, const rope_tensor *ref_counts_out,
                    const rope_tensor *shortage, void *workspace, int64_t workspace_bytes,
                    ForkPlan *plan, std::vector<PageCache> *list, std::string *err);
int plan_compact_pages(const rope_tensor *page_table, const rope_tensor *ref_counts,
                       const rope_tensor *caches, int64_t num_caches,
                       const rope_tensor *page_table_out, const rope_tensor *ref_counts_out,
                       const rope_tensor *page_map, const rope_tensor *live, void *workspace,
                       int64_t workspace_bytes, CompactPlan *plan, std::vector<PageCache> *list,
                       std::string *err);

}  // namespace ropeamd
