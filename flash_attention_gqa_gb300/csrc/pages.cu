// Pages of the key-value cache between steps: requests end, give tokens back, or go on as several
// requests that share their pages; a pool is made dense; pages are copied.
//
// Tables.  What these operators change hangs together (share counts, free list, lengths), and each
// call is one cluster of 8 CTAs: work is spread over 8192 threads, and the cluster's barrier stands
// between reading what is to be replaced and replacing it, and between counting pages and placing
// them.  A call that cannot be met finds that out before its first change.  Atomics are on whole
// numbers and on bits of a set of pages, kept in the CTAs' shared memory (each CTA the bits of one
// stretch of ids): their order never shows, and pages come back in the order of their ids.
// Latency bounds them.
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "pages.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace fa {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32, kCtas = 8;

__device__ __forceinline__ int pages_of(long long n, int shift) {
  return (int)((n + (1 << shift) - 1) >> shift);
}

// Sum over the CTA's threads before this one, and in all.  Every thread calls it.
__device__ __forceinline__ int scan_before(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();   // (of an earlier call's sums)
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int sums = lane < kWarps ? warp_sums[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, sums, d);
    if (lane >= d) sums += y;
  }
  total = __shfl_sync(~0u, sums, 31);
  const int before = __shfl_sync(~0u, sums, (warp + 31) & 31);
  return inc - x + (warp ? before : 0);
}

// A set of pages: CTA c of the cluster holds words [c * words, (c + 1) * words) of its bits.
struct PageSet {
  cg::cluster_group cluster;
  uint32_t* mine;
  int words;
  __device__ __forceinline__ uint32_t* word(int page) const {
    const int w = page >> 5, c = w / words;
    return cluster.map_shared_rank(mine, c) + (w - c * words);
  }
  // Whether it was there before.
  __device__ __forceinline__ bool put(int page) const {
    const uint32_t bit = 1u << (page & 31);
    return (atomicOr(word(page), bit) & bit) != 0;
  }
};

__host__ __device__ inline int set_words(int n_pages) { return ((n_pages + 31) / 32 + kCtas - 1) / kCtas; }

// The warps of the cluster over the columns [first, last) of rows 0 .. n - 1: `S` warps a row, the
// row's columns dealt to their lanes, four of a lane at a time: `load(row, column)` of all four, then
// `take(what it gave)` of all four, then `use(row, column, what the one and the other gave)`.
// `range(row, first, last)` says false for rows to be left out.  `barrier()` is called once by all
// threads, before the first take.
template <class Range, class Load, class Take, class Use, class Barrier>
__device__ __forceinline__ void over_entries(int rank, int n, Range range, Load load, Take take, Use use,
                                             Barrier barrier) {
  const int lane = threadIdx.x & 31, warp = rank * kWarps + (threadIdx.x >> 5);
  constexpr int all = kCtas * kWarps;
  const int S = n >= all ? 1 : all / max(n, 1);   // warps a row
  bool passed = false;
  for (int i = warp / S; i < n; i += all) {   // (several rows a warp: only with one warp a row)
    int first, last;
    if (!range(i, first, last)) continue;
    for (int j = first + warp % S * 32; j < last; j += 4 * S * 32) {
      int x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int column = j + k * S * 32 + lane;
        if (column < last) x[k] = load(i, column);
      }
      __syncwarp();   // (a warp comes to it as one)
      if (!passed) barrier();
      passed = true;
      int y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + k * S * 32 + lane < last) y[k] = take(x[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int column = j + k * S * 32 + lane;
        if (column < last) use(i, column, x[k], y[k]);
      }
    }
  }
  __syncwarp();
  if (!passed) barrier();
}
struct Nothing {
  __device__ int operator()(int) const { return 0; }
};
// Rows of a call that stay in shared memory; more of them are looked up again.
constexpr int kRowsKept = 1024;
struct KeptRow {
  int row, first, last;
};

// ------------------------------------------------------------------- free

// Decrement the share counts of the pages given back; who meets a count of zero was the last
// holder, and its page joins the set.  Counts, places by a sum over the set, pages to the list.
// 256 requests that drop 8 tokens 7.5 us, three barriers of the cluster and six of its CTAs with dependent loads
// between them; 128 rows of 512 pages 18 us, by 65536 atomics that return.
__global__ void __launch_bounds__(kThreads, 1) pages_free_kernel(const __grid_constant__ PagesFreeArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ uint32_t seen[kMaxPagedBatch / 32];   // rows of the call
  __shared__ KeptRow kept[kRowsKept];
  __shared__ int warp_sums[32], totals[kCtas];
  const cg::cluster_group cluster = cg::this_cluster();
  const PagesPool& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster.block_rank();
  const PageSet set{cluster, bits, set_words(p.n_pages)};
  for (int i = tid; i < set.words; i += kThreads) bits[i] = 0;
  for (int i = tid; i < kMaxPagedBatch / 32; i += kThreads) seen[i] = 0;
  __syncthreads();
  const int used = *p.free_used;
  const long long most = (long long)p.max_pages << p.page_shift;

  bool bad = used < 0 || used > p.n_free, odd = false;
  for (int i = tid; i < a.N; i += kThreads) {
    const int row = a.rows[i], keep = a.keep ? a.keep[i] : 0;
    if (i < kRowsKept) kept[i] = KeptRow{row, 0, 0};
    if (row < 0) continue;
    if (row >= p.B) { bad = true; continue; }
    const int len = p.lens[row];
    bad |= (atomicOr(&seen[row >> 5], 1u << (row & 31)) >> (row & 31) & 1) != 0;
    if (i < kRowsKept) kept[i] = KeptRow{row, pages_of(keep, p.page_shift), pages_of(len, p.page_shift)};
    if (len < 0 || len > most || keep < 0 || keep > len) { bad = true; continue; }
    // the last page kept gets new tokens, which other requests would see
    if (keep < len && (keep & ((1 << p.page_shift) - 1)) != 0) {
      const int page = p.block_table[(int64_t)row * p.max_pages + (keep >> p.page_shift)];
      if (page >= 0 && page < p.n_pages) bad |= p.shares[page] > 0;
    }
  }
  // All CTAs have looked at everything, and agree.
  const bool fail = __syncthreads_or(bad);
  auto row_of = [&](int i) { return i < kRowsKept ? kept[i].row : a.rows[i]; };
  auto range = [&](int i, int& first, int& last) {
    if (i < kRowsKept) {
      first = kept[i].first;
      last = kept[i].last;
      return true;
    }
    const int row = a.rows[i];
    if (row < 0) return false;
    first = pages_of(a.keep ? a.keep[i] : 0, p.page_shift);
    last = pages_of(p.lens[row], p.page_shift);
    return true;
  };
  auto entry = [&](int i, int j) { return p.block_table[(int64_t)row_of(i) * p.max_pages + j]; };
  auto known = [&](int page) { return page >= 0 && page < p.n_pages; };
  // (behind the barrier: the sets are empty, the counts have been looked at)
  over_entries(rank, fail ? 0 : a.N, range, entry, [&](int page) {
    return known(page) ? atomicSub(&p.shares[page], 1) : 0;
  }, [&](int, int, int page, int others) {
    if (!known(page)) { odd = true; return; }
    if (others <= 0) odd |= set.put(page) || others < 0;   // (below zero: given back before)
  }, [&] { cluster.sync(); });
  cluster.sync();
  int count = 0;
  const int per = (set.words + kThreads - 1) / kThreads;
  for (int w = tid * per; w < min((tid + 1) * per, set.words); ++w) count += __popc(bits[w]);
  int here;
  scan_before(count, warp_sums, here);
  if (tid < kCtas) cluster.map_shared_rank(totals, tid)[rank] = here;
  cluster.sync();   // (behind it, each CTA reads what is its own)
  int all = 0, before = 0;
  for (int c = 0; c < kCtas; ++c) {
    if (c < rank) before += totals[c];
    all += totals[c];
  }
  const bool over = !fail && all > used;   // more pages than the list has given out
  if (over) {
    over_entries(rank, a.N, range, entry, Nothing{}, [&](int, int, int page, int) {
      if (known(page)) atomicAdd(&p.shares[page], 1);
    }, [] {});
  } else if (!fail) {
    // a warp a word, a lane a page
    int at = used - all + before;
    for (int w0 = 0; w0 < set.words; w0 += kThreads) {   // in order, a word a thread
      const uint32_t word = w0 + tid < set.words ? bits[w0 + tid] : 0;
      int in_round;
      const int k = scan_before(__popc(word), warp_sums, in_round);
      for (uint32_t left = __ballot_sync(~0u, word != 0); left; left &= left - 1) {
        const int from = __ffs(left) - 1;
        const uint32_t x = __shfl_sync(~0u, word, from);
        const int k0 = __shfl_sync(~0u, k, from);
        if (x >> lane & 1) {
          const int page = (rank * set.words + w0 + warp * 32 + from) * 32 + lane;
          p.free_pages[at + k0 + __popc(x & ((1u << lane) - 1))] = page;
          p.shares[page] = 0;
        }
      }
      at += in_round;
    }
  }
  if ((fail || over || odd) && (odd || (rank == 0 && tid == 0))) atomicOr(p.err, (uint32_t)DEV_BAD_VALUE);
  if (rank == 0) {
    const bool none = fail || over;
    if (tid == 0) *a.free_used_out = none ? used : used - all;
    if (a.lens_out != p.lens)
      for (int b = tid; b < p.B; b += kThreads)
        if (none || !(seen[b >> 5] >> (b & 31) & 1)) a.lens_out[b] = p.lens[b];
    if (!none)
      for (int i = tid; i < a.N; i += kThreads) {
        const int row = a.rows[i];
        if (row >= 0) a.lens_out[row] = a.keep ? a.keep[i] : 0;
      }
  }
}

// ------------------------------------------------------------------- fork

// A child takes its parent's full pages, whose share counts rise, and a fresh page for the tokens of
// a last one that is not full: those are to be copied, and the list says so.  Children of one parent that
// take the same of it raise a page's count together, by one of them: scattered atomics go 32 cycles a
// warp (128 children of 512 pages: 65536 of them or 512, and 12 us, by the table entries).
__global__ void __launch_bounds__(kThreads, 1) pages_fork_kernel(const __grid_constant__ PagesForkArgs a) {
  extern __shared__ int fresh[];   // [N] free pages taken before the entry
  int* const lead = fresh + a.N;   // [B] first entry of a parent
  int* const count = lead + a.p.B; // [B] its entries
  __shared__ uint32_t seen[kMaxPagedBatch / 32];    // children
  __shared__ uint32_t mixed[kMaxPagedBatch / 32];   // parents whose children take different lengths
  __shared__ int warp_sums[32];
  const cg::cluster_group cluster = cg::this_cluster();
  const PagesPool& p = a.p;
  const int tid = threadIdx.x, rank = cluster.block_rank();
  const int P = 1 << p.page_shift;
  for (int i = tid; i < kMaxPagedBatch / 32; i += kThreads) seen[i] = mixed[i] = 0;
  for (int b = tid; b < p.B; b += kThreads) {
    lead[b] = a.N;
    count[b] = 0;
  }
  __syncthreads();
  const int used = *p.free_used;
  const long long most = (long long)p.max_pages << p.page_shift;
  const int per = (a.N + kThreads - 1) / kThreads;
  const int i0 = min(tid * per, a.N), i1 = min(i0 + per, a.N);
  auto length = [&](int i, int parent) { return a.fork_lens ? a.fork_lens[i] : p.lens[parent]; };

  bool bad = used < 0 || used > p.n_free;
  int need = 0;
  for (int i = i0; i < i1; ++i) {
    const int parent = a.parents[i], child = a.children[i];
    if (parent < 0) continue;
    if (parent >= p.B || child < 0 || child >= p.B || child == parent) { bad = true; continue; }
    bad |= (atomicOr(&seen[child >> 5], 1u << (child & 31)) >> (child & 31) & 1) != 0;
    const int held = p.lens[parent], n = length(i, parent);
    bad |= p.lens[child] != 0 || held < 0 || held > most || n < 0 || n > held;
    need += (n & (P - 1)) != 0;
    atomicMin(&lead[parent], i);
    atomicAdd(&count[parent], 1);
  }
  int all;
  int k = scan_before(need, warp_sums, all);
  for (int i = i0; i < i1; ++i) {   // (the scan's barriers: all children are in `seen`)
    const int parent = a.parents[i];
    if (parent < 0 || parent >= p.B) continue;
    bad |= (seen[parent >> 5] >> (parent & 31) & 1) != 0;
    const int first = lead[parent];
    if (a.fork_lens && first < a.N && a.fork_lens[i] != a.fork_lens[first])
      atomicOr(&mixed[parent >> 5], 1u << (parent & 31));
  }
  const bool fail = __syncthreads_or(bad || all > p.n_free - used);
  if (!fail)
    for (int i = i0; i < i1; ++i) {
      fresh[i] = k;
      const int parent = a.parents[i];
      if (parent >= 0) k += (length(i, parent) & (P - 1)) != 0;
    }
  __syncthreads();
  if (fail) {
    for (int i = rank * kThreads + tid; i < a.N * 3; i += kCtas * kThreads) a.copies[i] = i % 3 == 2 ? 0 : -1;
  } else {
    auto range = [&](int i, int& first, int& last) {
      const int parent = a.parents[i];
      first = 0;
      last = parent < 0 ? 0 : pages_of(length(i, parent), p.page_shift);
      last = max(last, 1);   // (one at least: it writes the entry's copy)
      return true;
    };
    auto entry = [&](int i, int j) {
      const int parent = a.parents[i];
      return parent < 0 || j >= p.max_pages ? -1 : p.block_table[(int64_t)parent * p.max_pages + j];
    };
    auto known = [&](int page) { return page >= 0 && page < p.n_pages; };
    over_entries(rank, a.N, range, entry, Nothing{}, [&](int i, int j, int page, int) {
      const int parent = a.parents[i];
      const int n = parent < 0 ? 0 : length(i, parent), full = n >> p.page_shift, part = n & (P - 1);
      int32_t* const copy = a.copies + (int64_t)i * 3;
      if (j == full && part) {
        const int to = p.free_pages[used + fresh[i]];
        const bool both = known(page) && known(to);
        a.table[(int64_t)a.children[i] * p.max_pages + j] = to;
        copy[0] = both ? page : -1;
        copy[1] = both ? to : -1;
        copy[2] = both ? part : 0;
        if (!both) atomicOr(p.err, (uint32_t)DEV_BAD_VALUE);
      } else if (j < full) {
        a.table[(int64_t)a.children[i] * p.max_pages + j] = page;
        if (!known(page))
          atomicOr(p.err, (uint32_t)DEV_BAD_VALUE);
        else if (mixed[parent >> 5] >> (parent & 31) & 1)
          atomicAdd(&p.shares[page], 1);
        else if (lead[parent] == i)
          atomicAdd(&p.shares[page], count[parent]);
      }
      if (j == 0 && !part) {
        copy[0] = copy[1] = -1;
        copy[2] = 0;
      }
    }, [] {});
  }
  cluster.sync();   // all lengths have been read
  if (rank == 0) {
    if (tid == 0) {
      *a.free_used_out = fail ? used : used + all;
      if (fail) atomicOr(p.err, (uint32_t)DEV_BAD_VALUE);
    }
    // (no parent is a child of the call: in place, its length is still there)
    if (a.lens_out != p.lens)
      for (int b = tid; b < p.B; b += kThreads)
        if (fail || !(seen[b >> 5] >> (b & 31) & 1)) a.lens_out[b] = p.lens[b];
    if (!fail)
      for (int i = i0; i < i1; ++i)
        if (a.parents[i] >= 0) a.lens_out[a.children[i]] = length(i, a.parents[i]);
  }
}

// ---------------------------------------------------------------- compact

// Held pages H (in a table, before its request's end) and free ones F.  With the j-th highest held
// page h_j and the j-th lowest free page f_j, page h_j moves to f_j for as long as f_j < h_j: after
// it the held pages are as low as they can be.  A page asks for itself: a held one with j held
// pages above it moves if more than j free ones are below it; a free one with j free pages below it
// is taken if more than j held ones are above it.  Both counts are sums over bits.  (128 requests of up to 256
// pages, 4096 moves: 9 us, five cluster barriers and the loads between them; their copy 165.)
__global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(const __grid_constant__ PagesCompactArgs a) {
  extern __shared__ uint32_t sm[];
  __shared__ int warp_sums[32];
  __shared__ int counts[4];   // held, free, free afterwards, something is wrong
  const cg::cluster_group cluster = cg::this_cluster();
  const PagesPool& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = cluster.block_rank();
  const int words = set_words(p.n_pages), g = rank * kThreads + tid;
  constexpr int grid = kCtas * kThreads;
  uint32_t *const held = sm, *const spare = sm + words;
  int *const held_before = (int*)(sm + 2 * words), *const spare_before = held_before + words;
  for (int i = tid; i < 2 * words; i += kThreads) sm[i] = 0;
  if (tid < 4) counts[tid] = 0;
  const int used = *p.free_used;
  const long long most_len = (long long)p.max_pages << p.page_shift;
  bool bad = used < 0 || used > p.n_free;
  for (int b = tid; b < p.B; b += kThreads) bad |= p.lens[b] < 0 || p.lens[b] > most_len;
  const bool wrong = __syncthreads_or(bad);   // the same in all CTAs
  for (int64_t i = g; i < (int64_t)a.max_moves * 3; i += grid) a.moves[i] = i % 3 == 2 ? 0 : -1;

  auto row = [&](int b, int& first, int& last) {
    first = 0;
    last = pages_of(p.lens[b], p.page_shift);
    return true;
  };
  auto entry = [&](int b, int j) { return p.block_table[(int64_t)b * p.max_pages + j]; };
  const PageSet in_use{cluster, held, words}, unused{cluster, spare, words};
  bad = false;
  over_entries(rank, wrong ? 0 : p.B, row, entry, Nothing{}, [&](int, int, int page, int) {
    if (page < 0 || page >= p.n_pages) bad = true;
    else in_use.put(page);
  }, [&] { cluster.sync(); });   // (the sets are empty)
  if (!wrong) {
    for (int64_t i = (int64_t)used + g; i < p.n_free; i += grid) {   // (lists may end at any int)
      const int page = p.free_pages[i];
      bad |= page < 0 || page >= p.n_pages || unused.put(page);   // (twice in the list)
    }
    if (bad) counts[3] = 1;
  }
  cluster.sync();
  // counts of the words before each of this CTA's
  const int per = (words + kThreads - 1) / kThreads, w0 = min(tid * per, words), w1 = min(w0 + per, words);
  auto sums = [&](const uint32_t* set, int* before) {
    int n = 0, total;
    for (int w = w0; w < w1; ++w) n += __popc(set[w]);
    int k = scan_before(n, warp_sums, total);
    for (int w = w0; w < w1; ++w) {
      before[w] = k;
      k += __popc(set[w]);
    }
    return total;
  };
  const int n_held = sums(held, held_before), n_spare = sums(spare, spare_before);
  bool both = false;
  for (int w = w0; w < w1; ++w) both |= (held[w] & spare[w]) != 0;   // free and in a table
  if (both) counts[3] = 1;
  if (tid == 0) { counts[0] = n_held; counts[1] = n_spare; }
  cluster.sync();
  int all_held = 0, below_held[kCtas], below_spare = 0;   // pages of the CTAs before each, before this one
  bool fail = wrong;
  for (int c = 0; c < kCtas; ++c) {
    const int* const x = cluster.map_shared_rank(counts, c);
    below_held[c] = all_held;
    all_held += x[0];
    if (c < rank) below_spare += x[1];
    fail |= x[3] != 0;
  }
  // held pages before `page`, anywhere
  auto held_below = [&](int page) {
    const int w = page >> 5, c = w / words, at = w - c * words;
    const uint32_t x = cluster.map_shared_rank(held, c)[at];
    return below_held[c] + cluster.map_shared_rank(held_before, c)[at] + __popc(x & ((1u << (page & 31)) - 1));
  };

  if (!fail) {
    // a warp a word, a lane a page
    for (int w = warp; w < words; w += kWarps) {
      const uint32_t h = held[w], f = spare[w], below = (1u << lane) - 1;
      const int page = (rank * words + w) * 32 + lane;
      const int hb = below_held[rank] + held_before[w] + __popc(h & below);
      const int fb = below_spare + spare_before[w] + __popc(f & below);
      const bool is_held = h >> lane & 1, is_free = f >> lane & 1;
      const int above = all_held - hb - (is_held ? 1 : 0);
      const bool goes = is_held && fb > above && above < a.max_moves;
      const bool taken = is_free && above > fb && fb < a.max_moves;
      if (goes) {
        a.moves[(int64_t)above * 3] = page;
        a.moves[(int64_t)above * 3 + 2] = 1 << p.page_shift;
      }
      if (taken) a.moves[(int64_t)fb * 3 + 1] = page;
      const uint32_t went = __ballot_sync(~0u, goes), took = __ballot_sync(~0u, taken);
      if (lane == 0) spare[w] = (f & ~took) | went;   // free afterwards
    }
    __syncthreads();
    const int after = sums(spare, spare_before);
    if (tid == 0) counts[2] = after;
  }
  if (!fail && a.shares_out != p.shares)
    for (int i = g; i < p.n_pages; i += grid) a.shares_out[i] = p.shares[i];
  cluster.sync();   // the moves are known, and the free pages after them
  if (fail) {
    if (g == 0) atomicOr(p.err, (uint32_t)DEV_BAD_VALUE);
    if (a.table_out != p.block_table)
      for (int64_t i = g; i < (int64_t)p.B * p.max_pages; i += grid) a.table_out[i] = p.block_table[i];
    if (a.shares_out != p.shares)
      for (int i = g; i < p.n_pages; i += grid) a.shares_out[i] = p.shares[i];
    if (a.free_out != p.free_pages)
      for (int64_t i = (int64_t)max(used, 0) + g; i < p.n_free; i += grid) a.free_out[i] = p.free_pages[i];
  } else {
    for (int64_t i = g; i < a.max_moves; i += grid) {
      const int src = __ldcg(a.moves + i * 3), dst = __ldcg(a.moves + i * 3 + 1);
      if (src < 0) continue;
      const int n = p.shares[src];   // (in place: no page is the source of one move and the end of another)
      a.shares_out[dst] = n;
      a.shares_out[src] = 0;
    }
    const bool in_place = a.table_out == p.block_table;
    auto whole = [&](int b, int& first, int& last) {
      row(b, first, last);
      if (!in_place) last = p.max_pages;   // what is behind a request's pages, too
      return true;
    };
    over_entries(rank, p.B, whole, entry, Nothing{}, [&](int b, int j, int page, int) {
      int to = page;
      if (j < pages_of(p.lens[b], p.page_shift)) {
        const int above = all_held - held_below(page) - 1;
        if (above < a.max_moves && __ldcg(a.moves + (int64_t)above * 3) == page)
          to = __ldcg(a.moves + (int64_t)above * 3 + 1);
      }
      if (!in_place || to != page) a.table_out[(int64_t)b * p.max_pages + j] = to;
    }, [] {});
    int at = used;
    for (int c = 0; c < rank; ++c) at += cluster.map_shared_rank(counts, c)[2];
    for (int w = warp; w < words; w += kWarps) {
      const uint32_t f = spare[w];
      if (f >> lane & 1)
        a.free_out[at + spare_before[w] + __popc(f & ((1u << lane) - 1))] = (rank * words + w) * 32 + lane;
    }
  }
  cluster.sync();   // nobody's shared memory goes before all have read it
}

// ------------------------------------------------------------------- copy

constexpr int kCopyThreads = 256, kCopyPer = 8;   // 16-byte units of a thread

// Part blockIdx.x % parts of move blockIdx.x / parts, in layer blockIdx.y / 2 of K or V.  Bound by
// memory; all loads of a thread are in flight before its first store.  4096 pages of 128 KB in all layers
// 165 us, 6.5 TB/s read and written; 128 copies of one page's 46 tokens 14 us, read from L2.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PagesCopyArgs a, int parts,
                                                                  int shift) {
  const int move = blockIdx.x / parts, part = blockIdx.x - move * parts;
  const int src = a.moves[(int64_t)move * 3], dst = a.moves[(int64_t)move * 3 + 1];
  const int tokens = a.moves[(int64_t)move * 3 + 2], P = 1 << a.lay.page_shift;
  if (src < 0 && dst < 0) return;   // no move
  if ((unsigned)src >= (unsigned)a.lay.n_pages || (unsigned)dst >= (unsigned)a.lay.n_pages ||
      (unsigned)tokens > (unsigned)P) {
    if (part == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
    return;
  }
  char* const cache = (char*)(blockIdx.y & 1 ? a.v_cache : a.k_cache) + (blockIdx.y >> 1) * a.layer;
  const char* const from = cache + src * a.lay.page;
  char* const to = cache + dst * a.lay.page;
  // units in the order of memory: dims, then tokens and heads, the nearer of the two first
  const bool heads_first = a.lay.token >= a.lay.head && a.K > 1;
  const uint32_t inner = heads_first ? a.K : tokens;
  const int64_t inner_step = heads_first ? a.lay.head : a.lay.token;
  const int64_t outer_step = heads_first ? a.lay.token : a.lay.head;
  const uint32_t all = ((uint32_t)tokens * a.K) << shift, upr = 1u << shift;   // units of the page
  const uint32_t i0 = part * (kCopyThreads * kCopyPer) + threadIdx.x;
  if (i0 >= all) return;
  uint4 x[kCopyPer];
  int64_t off[kCopyPer];
#pragma unroll
  for (int j = 0; j < kCopyPer; ++j) {
    const uint32_t i = i0 + j * kCopyThreads;
    if (i >= all) continue;
    const uint32_t r = i >> shift, o = r / inner;
    off[j] = o * outer_step + (r - o * inner) * inner_step + (i & (upr - 1)) * 16;
    x[j] = __ldcg(reinterpret_cast<const uint4*>(from + off[j]));
  }
#pragma unroll
  for (int j = 0; j < kCopyPer; ++j)
    if (i0 + j * kCopyThreads < all) *reinterpret_cast<uint4*>(to + off[j]) = x[j];
}

template <class Args>
cudaError_t launch_cluster(void (*kernel)(const Args), const Args& a, size_t smem, int most_smem, cudaStream_t st) {
  // (always to what the largest call needs: the limit is the function's, and another thread's launch
  // or an instantiated graph would meet a smaller one)
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = kCtas;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_pages_free(const PagesFreeArgs& a, cudaStream_t st) {
  return launch_cluster(pages_free_kernel, a, (size_t)set_words(a.p.n_pages) * 4, set_words(kMaxPoolPages) * 4, st);
}

cudaError_t launch_pages_fork(const PagesForkArgs& a, cudaStream_t st) {
  return launch_cluster(pages_fork_kernel, a, ((size_t)a.N + 2 * (size_t)a.p.B) * 4, kMaxPagedBatch * 12, st);
}

cudaError_t launch_pages_compact(const PagesCompactArgs& a, cudaStream_t st) {
  return launch_cluster(pages_compact_kernel, a, (size_t)set_words(a.p.n_pages) * 16, set_words(kMaxPoolPages) * 16,
                        st);
}

cudaError_t launch_pages_copy(const PagesCopyArgs& a, cudaStream_t st) {
  int shift = 0;
  while ((16 << shift) < a.row_bytes) ++shift;
  const int64_t units = ((int64_t)a.K << a.lay.page_shift) << shift;
  const int parts = (int)((units + kCopyThreads * kCopyPer - 1) / (kCopyThreads * kCopyPer));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.N * (int64_t)parts), 2 * a.layers);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, pages_copy_kernel, a, parts, shift);
}

}  // namespace fa
