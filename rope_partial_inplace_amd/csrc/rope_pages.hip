// rope_pages.hip -- copying, forking and compacting the pages of a cache (gfx950).
//
// Copy: page targets[i] of every cache becomes a copy of page sources[i].
//
// Fork: new row i continues sequence parents[i].  Full pages are shared; the last page, if it is not
// full, goes to the first row that continues the sequence when nothing else holds it, and is copied
// to a new page for the others; new pages are taken for the tokens to come.  New pages are the lowest
// free ones, dealt in the order of the rows, so the result does not depend on timing: ranks are sums
// over the rows and over the pages before.  Pages that this call frees are not handed out by it: none
// of them can then be read by one copy and written by another.
//   1. one workgroup: which row continues a sequence first, what each row wants, and the sums of
//      that; the others count the free pages of 4096 each
//   2. the free pages' numbers; the holds as they were
//   3. tables, holds and copies
//
// Compact: with n pages in use, the k-th one at or behind place n goes to the k-th free place before.
//   1. pages in use of 4096 each; 2. the map and the list of moves; 3. tables, holds and copies
//
// Of small pools launches 1 and 2 are one: each workgroup counts the pages before its own by itself.
//
// Copies move bytes; all else is a few sums, bound by the way from one launch to the next.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <vector>

#include "rope.h"
#include "rope_launch.h"
#include "rope_pages_plan.h"
#include "rope_q8.h"

namespace ropeamd {
namespace {

// Wavefronts at most where the host does not know the copies: they take pieces in turns.  A turn costs its
// reads of page numbers, an idle wavefront its launch (355000 pieces of a compacted pool: 271 us with
// 65536 wavefronts, 252 with 262144, 332 with one for every piece that could be).
constexpr int64_t kForkGroups = 8192, kCompactGroups = 262144;

// Chunks of pages that every workgroup counts for itself, at most.  That saves the launch that would tell it, and
// costs it a turn for each chunk: fork 14.4 -> 11.0 us with one chunk, 14.0 -> 12.1 with four, 14.0 -> 14.4
// with eight; compaction, which counts twice, 12.0 -> 10.3 with one, 16.3 -> 18.8 with four.
constexpr int64_t kFewFork = 4, kFewCompact = 2;

typedef uint32_t words4 __attribute__((ext_vector_type(4)));
typedef uint32_t words2 __attribute__((ext_vector_type(2)));

// 16 bytes past the caches, from a base that is the same for all lanes: buffer stores with the
// device-scope and streaming bits.
__device__ inline void store_streamed(char *base, int offset, words4 v) {
  const auto buffer = __builtin_amdgcn_make_buffer_rsrc(base, 0, int(0xffffffff), 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b128(v, buffer, offset, 0, 16 | 2);
}

// What to copy: pages `from` to `to`, the first `tokens` of page_size tokens (0: whole pages).
struct Move {
  int64_t from, to, tokens;
};

__device__ inline int64_t wave_sum_before(int64_t x, int64_t *total) {
  const int lane = int(threadIdx.x) & 63;
  int64_t incl = x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  *total = __shfl(incl, 63);
  return incl - x;
}

// How many of a page's words a move takes.
__device__ inline uint32_t words_of(const PageRun &r, const Move &m, int64_t num_pages,
                                    int64_t page_size) {
  if (m.from < 0 || m.from >= num_pages || m.to < 0 || m.to >= num_pages) return 0;
  if (m.tokens <= 0 || r.parts == 0) return r.vecs;
  // the parts that hold the tokens, the last one whole
  return uint32_t((m.tokens * r.parts + page_size - 1) / page_size) * r.part_words;
}

// Unit `u` of a run: words of 2^width bytes as type W.
template <int WORDS, typename W, typename Moves>
__device__ inline void copy_unit(const PageCaches &p, const PageRun &r, int64_t u, int64_t count,
                                 int64_t num_pages, int64_t page_size, Moves moves) {
  const int lane = int(threadIdx.x) & 63;
  const bool small = count * r.count * r.pieces < (int64_t(1) << 31);
  if (r.lanes_log2 == 6) {
    const int64_t mc = small ? int64_t(div_by(r.div_pieces, uint32_t(u))) : u / r.pieces;
    const uint32_t piece = uint32_t(u - mc * r.pieces);
    const int64_t k = small ? int64_t(uint32_t(mc) / uint32_t(count)) : mc / count;
    const int64_t i = mc - k * count;
    const int c = r.first + int(k);
    const Move m = moves(i);
    const uint32_t all = words_of(r, m, num_pages, page_size), w0 = piece * (64 * WORDS);
    const char *from = p.base[c] + m.from * p.page[c] + int64_t(w0) * int64_t(sizeof(W));
    char *to = p.base[c] + m.to * p.page[c] + int64_t(w0) * int64_t(sizeof(W));
    W word[WORDS];
#pragma unroll
    for (int k = 0; k < WORDS; ++k)
      if (w0 + 64 * k + lane < all)
        word[k] = __builtin_nontemporal_load(reinterpret_cast<const W *>(from) + (64 * k + lane));
#pragma unroll
    for (int k = 0; k < WORDS; ++k)
      if (w0 + 64 * k + lane < all) {
        if constexpr (sizeof(W) == 16) store_streamed(to, 16 * (64 * k + lane), word[k]);
        else __builtin_nontemporal_store(word[k], reinterpret_cast<W *>(to) + (64 * k + lane));
      }
  } else {
    const int64_t mc = u * (64 >> r.lanes_log2) + (lane >> r.lanes_log2);
    const int64_t k = small ? int64_t(uint32_t(mc) / uint32_t(count)) : mc / count;
    if (k >= r.count) return;
    const int64_t i = mc - k * count;
    const int c = r.first + int(k);
    const uint32_t w = uint32_t(lane) & ((1u << r.lanes_log2) - 1);
    const Move m = moves(i);
    if (w >= words_of(r, m, num_pages, page_size)) return;
    const W word = reinterpret_cast<const W *>(p.base[c] + m.from * p.page[c])[w];
    reinterpret_cast<W *>(p.base[c] + m.to * p.page[c])[w] = word;
  }
}

// All words of `count` moves in all caches, shared by `groups` wavefronts, of which this is `group`.
template <int WORDS, typename Moves>
__device__ inline void copy_pages(const PageCaches &p, int64_t count, int64_t group, int64_t groups,
                                  int64_t num_pages, int64_t page_size, Moves moves) {
  int64_t end[kPageRuns], total = 0;
#pragma unroll
  for (int r = 0; r < kPageRuns; ++r) {
    if (r < p.runs) {
      const int per = 64 >> p.run[r].lanes_log2;
      total += (count * p.run[r].count * p.run[r].pieces + per - 1) / per;
    }
    end[r] = total;
  }
  for (int64_t u = group; u < total; u += groups) {
    int r = 0;
    int64_t begin = 0;
#pragma unroll
    for (int k = 0; k + 1 < kPageRuns; ++k)
      if (u >= end[k]) {
        r = k + 1;
        begin = end[k];
      }
    const PageRun &run = p.run[r];
    const int64_t at = u - begin;
    switch (run.width) {
      case 4: copy_unit<WORDS, words4>(p, run, at, count, num_pages, page_size, moves); break;
      case 3: copy_unit<WORDS, words2>(p, run, at, count, num_pages, page_size, moves); break;
      case 2: copy_unit<WORDS, uint32_t>(p, run, at, count, num_pages, page_size, moves); break;
      case 1: copy_unit<WORDS, uint16_t>(p, run, at, count, num_pages, page_size, moves); break;
      default: copy_unit<WORDS, uint8_t>(p, run, at, count, num_pages, page_size, moves); break;
    }
  }
}

__global__ __launch_bounds__(kPageBlock) void copy_pages_kernel(CopyPagesPlan p) {
  copy_pages<kPageWords>(p.caches, p.moves, blockIdx.x, gridDim.x, p.num_pages, 1, [&](int64_t i) {
    return Move{p.sources[i * p.source_stride], p.targets[i * p.target_stride], 0};
  });
}

// ---- counting over a workgroup of 1024 -------------------------------------------------------------
// Sum of x over the threads before this one, and over all.
__device__ inline int64_t scan_block(int64_t x, int64_t *lds, int64_t *total) {
  const int wave = int(threadIdx.x) >> 6, lane = int(threadIdx.x) & 63;
  int64_t sum;
  const int64_t before = wave_sum_before(x, &sum);
  __syncthreads();
  if (lane == 0) lds[wave] = sum;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int v = 0; v < kCountBlock / 64; ++v) {
    if (v < wave) base += lds[v];
    all += lds[v];
  }
  *total = all;
  return base + before;
}

constexpr int kPerThread = int(kPageChunk) / kCountBlock;

// How many of this thread's pages of a chunk (kPerThread neighbours) below `end` have (USED) or
// have no (!USED) holds; bit k of the flags: page k.
template <bool USED>
__device__ inline int32_t chunk_flags(const int64_t *refs, int64_t stride, int64_t chunk,
                                      int64_t end, uint32_t *flags) {
  *flags = 0;
  const int64_t first = chunk * kPageChunk + int64_t(threadIdx.x) * kPerThread;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k)
    if (first + k < end && (refs[(first + k) * stride] > 0) == USED) *flags |= 1u << k;
  return __popc(*flags);
}

// Sum of the chunks' counts before `chunk`, and of all.  At most 2^30 pages: both fit one scan.
__device__ inline int64_t chunks_before(const int32_t *counts, int64_t chunks, int64_t chunk,
                                        int64_t *lds, int64_t *total) {
  int64_t mine = 0, sum;
  for (int64_t i = threadIdx.x; i < chunks; i += kCountBlock)
    mine += int64_t(counts[i]) << 32 | int64_t(i < chunk ? counts[i] : 0);
  scan_block(mine, lds, &sum);
  *total = sum >> 32;
  return sum & 0xffffffff;
}

// The same, counted here: pages with (USED) or without holds before `chunk`, and all of them (ALL) or
// those up to `chunk`.
template <bool USED, bool ALL>
__device__ inline int64_t count_before(const int64_t *refs, int64_t stride, int64_t num_pages,
                                       int64_t chunks, int64_t chunk, int64_t *lds, int64_t *total) {
  int64_t mine = 0, sum;
  for (int64_t c = 0; c < (ALL ? chunks : chunk + 1); ++c) {
    uint32_t flags;
    const int64_t n = chunk_flags<USED>(refs, stride, c, num_pages, &flags);
    mine += n << 32 | (c < chunk ? n : 0);
  }
  scan_block(mine, lds, &sum);
  *total = sum >> 32;
  return sum & 0xffffffff;
}

// ---- fork ------------------------------------------------------------------------------------------
// The numbers of a chunk's free pages, `rank` of which lie before it, and the holds as they were.
__device__ inline void list_free(const ForkPlan &p, int64_t chunk, int64_t rank, int64_t *lds) {
  uint32_t flags;
  int64_t sum;
  const int32_t n = chunk_flags<false>(p.refs, p.ref_stride, chunk, p.num_pages, &flags);
  rank += scan_block(n, lds, &sum);
  const int64_t first = chunk * kPageChunk + int64_t(threadIdx.x) * kPerThread;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    if (first + k >= p.num_pages) break;
    if (flags >> k & 1u) p.free[rank++] = int32_t(first + k);
    p.refs_out[(first + k) * p.ref_out_stride] = p.refs[(first + k) * p.ref_stride];
  }
}

__device__ inline int64_t clamped_len(const ForkPlan &p, int64_t b) {
  return min(max(p.lens[b * p.len_stride], int64_t(0)), p.table.width * p.page_size);
}

__device__ inline int64_t pages_of(const ForkPlan &p, int64_t tokens) {
  return int64_t((uint32_t(tokens) + uint32_t(p.page_size) - 1) / uint32_t(p.page_size));
}

// What row i continues and how long it gets.
struct Row {
  int64_t parent, len, grown;  // parent -1: an empty row
};

__device__ inline Row row_of(const ForkPlan &p, int64_t i) {
  Row r = {p.parents[i * p.parent_stride], 0, 0};
  if (r.parent < 0 || r.parent >= p.table.rows) return {-1, 0, 0};
  r.len = clamped_len(p, r.parent);
  const int64_t g = p.grow != nullptr ? max(p.grow[i * p.grow_stride], int64_t(0)) : 0;
  r.grown = r.len + min(g, p.out.width * p.page_size - r.len);
  return r;
}

template <typename X>
__device__ inline X fresh(const X *p) {  // as the other threads' atomics left it
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// LOCAL: what the rows' threads tell each other about the sequences goes through LDS, which holds
// kLocalRows of them; else through global memory.
constexpr int64_t kLocalRows = 4096;

// FEW: the other workgroups list their chunk's free pages, too.
template <bool LOCAL, bool FEW>
__global__ __launch_bounds__(kCountBlock) void fork_count_kernel(ForkPlan p) {
  __shared__ int64_t lds[kCountBlock / 64];
  __shared__ int32_t local[LOCAL ? 2 * kLocalRows : 1];
  const int64_t B = p.table.rows, R = p.out.rows;
  int64_t sum;
  if (blockIdx.x > 0) {
    const int64_t chunk = int64_t(blockIdx.x) - 1;
    if constexpr (FEW) {
      const int64_t rank = count_before<false, false>(p.refs, p.ref_stride, p.num_pages, p.chunks,
                                                      chunk, lds, &sum);
      if (chunk == p.chunks - 1 && threadIdx.x == 0) p.totals[2] = sum;
      list_free(p, chunk, rank, lds);
    } else {
      uint32_t flags;
      const int32_t n = chunk_flags<false>(p.refs, p.ref_stride, chunk, p.num_pages, &flags);
      scan_block(n, lds, &sum);
      if (threadIdx.x == 0) p.counts[chunk] = int32_t(sum);
    }
    return;
  }
  int32_t *first = LOCAL ? local : p.first, *children = LOCAL ? local + kLocalRows : p.children;
  constexpr int kScope = LOCAL ? __HIP_MEMORY_SCOPE_WORKGROUP : __HIP_MEMORY_SCOPE_AGENT;
  for (int64_t b = threadIdx.x; b < B; b += kCountBlock) {
    __hip_atomic_store(&first[b], 0x7fffffff, __ATOMIC_RELAXED, kScope);
    __hip_atomic_store(&children[b], 0, __ATOMIC_RELAXED, kScope);
    p.kept[b] = 0;
  }
  if (!LOCAL) __threadfence();
  __syncthreads();
  for (int64_t i = threadIdx.x; i < R; i += kCountBlock) {
    const int64_t b = p.parents[i * p.parent_stride];
    if (b < 0 || b >= B) continue;
    __hip_atomic_fetch_min(&first[b], int32_t(i), __ATOMIC_RELAXED, kScope);
    __hip_atomic_fetch_add(&children[b], 1, __ATOMIC_RELAXED, kScope);
  }
  if (!LOCAL) __threadfence();
  __syncthreads();
  if (LOCAL)
    for (int64_t b = threadIdx.x; b < B; b += kCountBlock) {
      p.first[b] = first[b];
      p.children[b] = children[b];
    }
  int64_t wanted = 0, copies = 0;
  for (int64_t i0 = 0; i0 < R; i0 += kCountBlock) {
    const int64_t i = i0 + threadIdx.x;
    int64_t need = 0, last = -1;
    Row r = {-1, 0, 0};
    bool copy = false;
    if (i < R) r = row_of(p, i);
    if (r.parent >= 0) {
      const int64_t used = pages_of(p, r.len);
      need = pages_of(p, r.grown) - used;
      if (r.len % p.page_size != 0) {
        last = p.table.data[r.parent * p.table.row + (used - 1) * p.table.col];
        if (last >= 0 && last < p.num_pages) {
          const bool keep = __hip_atomic_load(&first[r.parent], __ATOMIC_RELAXED, kScope) == i &&
                            p.refs[last * p.ref_stride] <= 1;
          if (keep) p.kept[r.parent] = 1;
          copy = !keep;
          need += copy;
        }
      }
    }
    // both sums in one scan: at most 2^30 new pages a row's table holds, and 1024 rows' at a time
    int64_t all;
    const int64_t before = scan_block(need << 11 | int64_t(copy), lds, &all);
    const int64_t base = wanted + (before >> 11), k = copies + (before & 2047);
    wanted += all >> 11;
    copies += all & 2047;
    if (i < R) p.base[i] = base;
    if (copy) {
      p.copies[3 * k] = last;
      p.copies[3 * k + 1] = base;
      p.copies[3 * k + 2] = r.len % p.page_size;
    }
  }
  if (threadIdx.x == 0) {
    p.totals[0] = wanted;
    p.totals[1] = copies;
    if (p.chunks == 0) p.totals[2] = 0;
  }
}

__global__ __launch_bounds__(kCountBlock) void fork_free_kernel(ForkPlan p) {
  __shared__ int64_t lds[kCountBlock / 64];
  int64_t total;
  const int64_t rank = chunks_before(p.counts, p.chunks, blockIdx.x, lds, &total);
  if (blockIdx.x == 0 && threadIdx.x == 0) p.totals[2] = total;
  list_free(p, blockIdx.x, rank, lds);
}

__device__ inline int64_t new_page(const ForkPlan &p, int64_t rank) {
  return rank < p.totals[2] ? int64_t(p.free[rank]) : -1;
}

__device__ inline void add_holds(const ForkPlan &p, int64_t page, int64_t n) {
  if (n != 0 && page >= 0 && page < p.num_pages)
    atomicAdd(reinterpret_cast<unsigned long long *>(p.refs_out + page * p.ref_out_stride),
              static_cast<unsigned long long>(n));  // modulo 2^64: n may be negative
}

__device__ inline void fork_tables(const ForkPlan &p, int64_t at, int64_t step) {
  if (at == 0) p.shortage[0] = max(p.totals[0] - p.totals[2], int64_t(0));
  const int64_t wide = max(p.out.width, int64_t(1));
  for (int64_t e = at; e < p.out.rows * wide; e += step) {
    const int64_t i = e / wide, j = e - i * wide;
    const Row r = row_of(p, i);
    if (j == 0) p.lens_out[i * p.len_out_stride] = r.grown;
    if (j >= p.out.width) continue;
    int64_t page = -1;
    const int64_t used = pages_of(p, r.len);
    if (j < pages_of(p, r.grown)) {
      const int64_t *from = p.table.data + r.parent * p.table.row;
      int64_t own = used;  // the row's first new page
      if (r.len % p.page_size != 0) {
        const int64_t last = from[(used - 1) * p.table.col];
        if (last >= 0 && last < p.num_pages &&
            !(p.first[r.parent] == i && p.kept[r.parent] != 0))
          own = used - 1;
      }
      if (j < own) {
        page = from[j * p.table.col];
      } else {
        page = new_page(p, p.base[i] + (j - own));
        add_holds(p, page, 1);
      }
    }
    p.out.data[i * p.out.row + j * p.out.col] = page;
  }
  // holds of the sequences: full pages go on once for every row, the last one if a row keeps it
  for (int64_t e = at; e < p.table.rows * p.table.width; e += step) {
    const int64_t b = e / p.table.width, j = e - b * p.table.width;
    const int64_t len = clamped_len(p, b), held = pages_of(p, len);
    if (j >= held) continue;
    const int64_t page = p.table.data[b * p.table.row + j * p.table.col];
    const bool tail = j == held - 1 && len % p.page_size != 0;
    add_holds(p, page, (tail ? p.kept[b] : p.children[b]) - 1);
  }
}

__global__ __launch_bounds__(kPageBlock) void fork_write_kernel(ForkPlan p) {
  const int64_t block = blockIdx.x;
  if (block < p.table_blocks) {
    fork_tables(p, block * kPageBlock + threadIdx.x, p.table_blocks * kPageBlock);
    return;
  }
  copy_pages<kForkWords>(p.caches, p.totals[1], block - p.table_blocks, gridDim.x - p.table_blocks, p.num_pages,
             p.page_size, [&](int64_t i) {
               const int64_t *c = p.copies + 3 * i;
               return Move{c[0], new_page(p, c[1]), c[2]};
             });
}

// ---- compact ---------------------------------------------------------------------------------------
__global__ __launch_bounds__(kCountBlock) void compact_count_kernel(CompactPlan p) {
  __shared__ int64_t lds[kCountBlock / 64];
  uint32_t flags;
  int64_t sum;
  scan_block(chunk_flags<true>(p.refs, p.ref_stride, blockIdx.x, p.num_pages, &flags), lds, &sum);
  if (threadIdx.x == 0) p.counts[blockIdx.x] = int32_t(sum);
}

template <bool FEW>
__global__ __launch_bounds__(kCountBlock) void compact_map_kernel(CompactPlan p) {
  __shared__ int64_t lds[kCountBlock / 64];
  const int64_t chunk = blockIdx.x;
  int64_t n, sum, below;
  uint32_t flags;
  auto before = [&](int64_t c, int64_t *all) {
    if constexpr (FEW)
      return count_before<true, true>(p.refs, p.ref_stride, p.num_pages, p.chunks, c, lds, all);
    else
      return chunks_before(p.counts, p.chunks, c, lds, all);
  };
  int64_t rank = before(chunk, &n);
  // pages in use before place n: of the whole chunks before it, and of its own
  const int64_t border = n / kPageChunk;
  const int64_t whole = before(border, &sum);
  scan_block(chunk_flags<true>(p.refs, p.ref_stride, border, min(n, p.num_pages), &flags), lds, &below);
  const int64_t moves = n - whole - below;
  if (chunk == 0 && threadIdx.x == 0) {
    p.totals[0] = moves;
    p.live[0] = n;
  }
  if (chunk >= p.chunks) return;  // no pages at all
  rank += scan_block(chunk_flags<true>(p.refs, p.ref_stride, chunk, p.num_pages, &flags), lds, &sum);
  const int64_t first = chunk * kPageChunk + int64_t(threadIdx.x) * kPerThread;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int64_t page = first + k;
    if (page >= p.num_pages) break;
    const bool used = flags >> k & 1u;
    if (used && page >= n) p.moves[2 * (rank - (n - moves))] = page;
    if (!used && page < n) p.moves[2 * (page - rank) + 1] = page;
    // a moved page's entry: the number of its move, until the next launch has its place
    p.map[page * p.map_stride] = !used ? -1 : page < n ? page : -2 - (rank - (n - moves));
    p.refs_out[page * p.ref_out_stride] = p.refs[page * p.ref_stride];
    rank += used;
  }
}

// A page's new number from its map entry: below -1 the number of its move (launch 2), or the new number
// already (another thread of launch 3 may have written it).
__device__ inline int64_t moved_to(const CompactPlan &p, int64_t entry) {
  return entry < -1 ? p.moves[2 * (-2 - entry) + 1] : entry;
}

__device__ inline void compact_tables(const CompactPlan &p, int64_t at, int64_t step) {
  const int64_t moves = p.totals[0];
  for (int64_t k = at; k < moves; k += step) {
    const int64_t from = p.moves[2 * k], to = p.moves[2 * k + 1];
    __hip_atomic_store(&p.map[from * p.map_stride], to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    p.refs_out[to * p.ref_out_stride] = p.refs_out[from * p.ref_out_stride];
    p.refs_out[from * p.ref_out_stride] = 0;
  }
  for (int64_t e = at; e < p.table.rows * p.table.width; e += step) {
    const int64_t b = e / p.table.width, j = e - b * p.table.width;
    int64_t page = p.table.data[b * p.table.row + j * p.table.col];
    if (page >= 0 && page < p.num_pages) page = moved_to(p, fresh(&p.map[page * p.map_stride]));
    p.out.data[b * p.out.row + j * p.out.col] = page;
  }
}

__global__ __launch_bounds__(kPageBlock) void compact_write_kernel(CompactPlan p) {
  const int64_t block = blockIdx.x;
  if (block < p.table_blocks) {
    compact_tables(p, block * kPageBlock + threadIdx.x, p.table_blocks * kPageBlock);
    return;
  }
  copy_pages<kPageWords>(p.caches, p.totals[0], block - p.table_blocks, gridDim.x - p.table_blocks, p.num_pages,
             1, [&](int64_t i) { return Move{p.moves[2 * i], p.moves[2 * i + 1], 0}; });
}

// The last launch of a plan: tables, and the copies in the first caches; then the other caches' copies,
// as many at a time as a launch holds.  `copies`: workgroups for a launch's copies.
template <typename Plan, typename Groups>
int run_writes(const void *fn, Plan &p, const std::vector<PageCache> &list, int words,
               Groups copies, void *stream) {
  size_t at = 0;
  do {
    at = take_caches(list, at, words, &p.caches);
    const int64_t blocks = p.table_blocks + (p.caches.count > 0 ? copies(p) : 0);
    if (blocks > 0) {
      const int st = launch_kernel(fn, dim3(uint32_t(blocks)), kPageBlock, 0, stream, &p);
      if (st != ROPE_OK) return st;
    }
    p.table_blocks = 0;
  } while (at < list.size());
  return ROPE_OK;
}

}  // namespace
}  // namespace ropeamd

using namespace ropeamd;

ROPE_API int rope_copy_pages(const rope_tensor *sources, const rope_tensor *targets,
                             const rope_tensor *caches, int64_t num_caches, void *stream) {
  CopyPagesPlan p;
  std::vector<PageCache> list;
  std::string err;
  const int st = plan_copy_pages(sources, targets, caches, num_caches, &p, &list, &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
  return run_writes(reinterpret_cast<const void *>(&copy_pages_kernel), p, list, kPageWords,
                    [](const CopyPagesPlan &q) {
                      return std::min(q.caches.units(q.moves), int64_t(1) << 25);
                    }, stream);
}

ROPE_API int64_t rope_fork_pages_workspace(int64_t num_sequences, int64_t num_rows,
                                           int64_t num_pages) {
  return fork_workspace(num_sequences, num_rows, num_pages);
}

ROPE_API int rope_fork_pages(const rope_tensor *page_table, const rope_tensor *seq_lens,
                             const rope_tensor *parents, const rope_tensor *grow,
                             const rope_tensor *ref_counts, int64_t page_size,
                             const rope_tensor *caches, int64_t num_caches,
                             const rope_tensor *page_table_out, const rope_tensor *seq_lens_out,
                             const rope_tensor *ref_counts_out, const rope_tensor *shortage,
                             void *workspace, int64_t workspace_bytes, void *stream) {
  ForkPlan p;
  std::vector<PageCache> list;
  std::string err;
  int st = plan_fork_pages(page_table, seq_lens, parents, grow, ref_counts, page_size, caches,
                           num_caches, page_table_out, seq_lens_out, ref_counts_out, shortage,
                           workspace, workspace_bytes, &p, &list, &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
#define ROPE_FC(L, F) reinterpret_cast<const void *>(&fork_count_kernel<L, F>)
  const bool few = p.chunks <= kFewFork;
  const void *count = p.table.rows <= kLocalRows ? (few ? ROPE_FC(true, true) : ROPE_FC(true, false))
                                                 : (few ? ROPE_FC(false, true) : ROPE_FC(false, false));
#undef ROPE_FC
  st = launch_kernel(count, dim3(uint32_t(1 + p.chunks)), kCountBlock, 0, stream, &p);
  if (st != ROPE_OK) return st;
  if (!few) {
    st = launch_kernel(reinterpret_cast<const void *>(&fork_free_kernel), dim3(uint32_t(p.chunks)),
                       kCountBlock, 0, stream, &p);
    if (st != ROPE_OK) return st;
  }
  return run_writes(reinterpret_cast<const void *>(&fork_write_kernel), p, list, kForkWords,
                    [](const ForkPlan &q) {
                      return std::min(q.caches.units(q.out.rows), kForkGroups);
                    }, stream);
}

ROPE_API int64_t rope_compact_pages_workspace(int64_t num_pages) {
  return compact_workspace(num_pages);
}

ROPE_API int rope_compact_pages(const rope_tensor *page_table, const rope_tensor *ref_counts,
                                const rope_tensor *caches, int64_t num_caches,
                                const rope_tensor *page_table_out,
                                const rope_tensor *ref_counts_out, const rope_tensor *page_map,
                                const rope_tensor *live, void *workspace, int64_t workspace_bytes,
                                void *stream) {
  CompactPlan p;
  std::vector<PageCache> list;
  std::string err;
  int st = plan_compact_pages(page_table, ref_counts, caches, num_caches, page_table_out,
                              ref_counts_out, page_map, live, workspace, workspace_bytes, &p, &list,
                              &err);
  if (st != ROPE_OK) {
    g_last_error = err;
    return st;
  }
  g_last_error.clear();
  const bool few = p.chunks <= kFewCompact;
  if (!few) {
    st = launch_kernel(reinterpret_cast<const void *>(&compact_count_kernel),
                       dim3(uint32_t(p.chunks)), kCountBlock, 0, stream, &p);
    if (st != ROPE_OK) return st;
  }
  st = launch_kernel(few ? reinterpret_cast<const void *>(&compact_map_kernel<true>)
                         : reinterpret_cast<const void *>(&compact_map_kernel<false>),
                     dim3(uint32_t(std::max<int64_t>(1, p.chunks))), kCountBlock, 0, stream, &p);
  if (st != ROPE_OK) return st;
  return run_writes(reinterpret_cast<const void *>(&compact_write_kernel), p, list, kPageWords,
                    [](const CompactPlan &q) {
                      return std::min(q.caches.units(q.num_pages / 2), kCompactGroups);
                    }, stream);
}
