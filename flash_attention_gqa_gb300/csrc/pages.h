// Internal interface of the page management (pages.cu): requests freed, cut and forked, pools
// compacted, pages copied.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "paged.h"

namespace fa {

constexpr int kMaxPoolPages = 1 << 21;   // of one pool: its bits and their counts stay in shared memory
constexpr int kMaxCopyLayers = 16384;    // twice as many are a grid's second dimension

// What the three operators on tables have in common.
struct PagesPool {
  const int32_t* lens;         // [B]
  const int32_t* block_table;  // [B, max_pages] (free, compact: read through it)
  int32_t* shares;             // [n_pages] requests beside the first that hold a page
  int32_t* free_pages;         // [n_free]
  const int32_t* free_used;    // [1]
  int B, max_pages, n_pages, n_free, page_shift;
  uint32_t* err;
};

struct PagesFreeArgs {
  PagesPool p;
  const int32_t* rows;         // [N], < 0: none
  const int32_t* keep;         // [N] or null: 0
  int32_t *lens_out, *free_used_out;   // may be the inputs
  int N;
};

struct PagesForkArgs {
  PagesPool p;
  const int32_t *parents, *children;   // [N], parent < 0: none
  const int32_t* fork_lens;            // [N] or null: the parents' lengths
  int32_t* table;                      // p.block_table, written
  int32_t *lens_out, *free_used_out;   // may be the inputs
  int32_t* copies;                     // [N, 3] source page, page, tokens
  int N;
};

struct PagesCompactArgs {
  PagesPool p;
  int32_t *table_out, *shares_out, *free_out;   // may be the inputs
  int32_t* moves;              // [max_moves, 3] source page, page, tokens
  int max_moves;
};

struct PagesCopyArgs {
  const int32_t* moves;        // [N, 3]
  void *k_cache, *v_cache;
  PagedLayout lay;
  int64_t layer;               // byte stride
  int N, layers, K, row_bytes; // bytes of a token's head
  uint32_t* err;
};

cudaError_t launch_pages_free(const PagesFreeArgs& a, cudaStream_t st);
cudaError_t launch_pages_fork(const PagesForkArgs& a, cudaStream_t st);
cudaError_t launch_pages_compact(const PagesCompactArgs& a, cudaStream_t st);
cudaError_t launch_pages_copy(const PagesCopyArgs& a, cudaStream_t st);

}  // namespace fa
