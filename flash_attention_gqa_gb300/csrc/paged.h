// Internal interface of the paged key-value cache operators (paged.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

constexpr int kMaxPagedBatch = 8192;       // requests of one call: their offsets stay in shared memory
constexpr int kMaxPagedGroups = 4096;      // groups that share a prefix, of one call
constexpr int kMaxPageSize = 65536;        // tokens per page, a power of two
constexpr int kMaxPagedLen = 1 << 30;      // keys of one request (max_pages * page_size)
constexpr int kMaxPagedRows = 128;         // query rows per kv head, G * T

// Where key (page, kv head, offset in the page) of a cache starts, in bytes
// from the cache's base: the strides are those of [pages, K, page_size, H].
struct PagedLayout {
  int64_t page, head, token;   // byte strides
  int n_pages;
  int page_shift;              // log2(page_size)
};

struct PagedTablesArgs {
  const int32_t* cached_lens;  // [B]
  const int32_t* new_lens;     // [B]
  const int32_t* free_pages;   // [n_free]
  const int32_t* free_used;    // [1]
  int32_t* block_table;        // [B, max_pages]
  int32_t* total_lens;         // [B], may be cached_lens
  int32_t* token_starts;       // [B + 1]
  int64_t* slots;              // [max_tokens]
  int32_t* positions;          // [max_tokens] or null
  int32_t* free_used_out;      // [1], may be free_used
  int B, n_free, n_pages, page_shift, max_pages, max_tokens;
  uint32_t* err;
};

struct PagedAppendArgs {
  const void *k, *v;                       // bf16 [N, K, H], through the strides below
  int64_t k_token, k_head, v_token, v_head;  // byte strides
  const int64_t* slots;                    // [N]
  void *k_cache, *v_cache;
  const float *k_scale, *v_scale;          // [K] or null
  PagedLayout lay;
  int N, K, H;
  bool e4m3;
  uint32_t* err;
};

// An item (b * K + k) whose tiles CTAs first .. last share; first < 0: none.  One
// entry per item where there are no more of them than CTAs, else one per CTA,
// for the item that begins in it.
struct PagedDecodeSplit {
  int item, first, last, pad;
};

// Attention of requests that share a prefix: its keys are attended to once for all rows of a group
// (HEAD: tiles of 128 rows of one group, "chunks", take the requests' place), every request's own keys
// behind it apart (TAIL), and both joined.
enum DecodeMode { DECODE_ALL, DECODE_TAIL, DECODE_HEAD };

// Rows [row, row + rows) of a group, counted over its members' G * T rows one member after the other.
struct PagedChunk {
  int len, leader;     // keys of the prefix, the request whose table row has their pages
  int member, row;     // the group's first entry in members; the chunk's first row
  int rows, base, pad0, pad1;   // base: rows, rounded up to 8 a chunk, of the chunks before
};
struct PagedSharedTables {
  int32_t* begins;     // [B] first key that is not in the request's prefix
  int32_t* places;     // [B] 128 * chunk + row of the request's first row, -1: no prefix
  int32_t* members;    // [n_members] requests, -1: none
  int32_t* n_chunks;
  PagedChunk* chunks;
  float* whole;        // partials of items that one CTA does: TAIL by item, HEAD by the chunks' bases
};

struct PagedDecodeArgs {
  const void* q;               // bf16 [B, K, G, T, H]
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;  // [K] or null
  PagedLayout lay;
  const int32_t* block_table;  // [B, max_pages]
  const int32_t* lens;         // [B]
  void* o;                     // bf16 [B, K, G, T, H]
  float* lse;                  // [B, K, G, T]
  int B, K, G, T, H, max_pages;
  int window;                  // 0: none
  float* partials;             // workspace: [CTAs][2][paged_partial_floats] of split items
  uint64_t wait_limit_ns;      // of the waits on barriers (the tcgen05 kernel)
  PagedDecodeSplit* splits;    // workspace: [CTAs]
  bool by_item;                // entries of splits are items
  bool unsplit;                // no item is shared: no splits, no partials (set by the launch)
  bool by_warps;               // many short items may go to single warps (DecodeCfg::SOLO)
  uint32_t* err;
  PagedSharedTables shared;    // TAIL and HEAD
};

// Workspace of a decode: the splits, then partials, on a GPU with sm_count SMs.
// CTAs an SM: two of 4 warps up to H = 128 and 32 query rows, else one: what rings
// and registers allow.
struct PagedDecodePlan {
  int ctas;
  size_t partials;   // offset
  size_t total;
};
// Rows of a partial: over 16 of them, whole groups of 8.
__host__ __device__ inline int paged_partial_rows(int R) { return R > 16 ? (R + 7) & ~7 : R; }
// Floats of one partial, with P rows: o [P, H] (the tcgen05 kernel: [H / 4, P, 4]), m [P],
// l [P], rounded up to 16 bytes.
__host__ __device__ inline int64_t paged_partial_floats(int R, int H) {
  return ((int64_t)paged_partial_rows(R) * (H + 2) + 3) & ~(int64_t)3;
}
inline PagedDecodePlan paged_decode_plan(int R, int H, int sm_count) {
  PagedDecodePlan p;
  p.ctas = sm_count * (H <= 128 && R <= 32 ? 2 : 1);
  p.partials = ((size_t)p.ctas * sizeof(PagedDecodeSplit) + 255) & ~(size_t)255;
  p.total = p.partials + (((size_t)p.ctas * 2 * paged_partial_floats(R, H) * 4 + 255) & ~(size_t)255);
  return p;
}

// ---- attention of requests that share prefixes
// The HEAD grid's: the decode's, with chunks as its requests, and maps of the caches with boxes of
// `rows` tokens of a page (64 dims of bf16, whole rows of e4m3); none where rows is 0.
struct PagedHeadArgs {
  CUtensorMap k_map, v_map;
  PagedDecodeArgs a;
  int rows;
};
// A map of a cache, for boxes of `rows` tokens; false where its strides cannot be mapped.
bool make_cache_map(CUtensorMap* m, const void* cache, const PagedLayout& lay, int K, int H, bool e4m3, int rows);

struct PagedSharedArgs {
  PagedDecodeArgs tail;        // the requests' own keys: splits by item, partials
  PagedDecodeSplit* head_splits;   // [chunks * K]
  float* head_partials;        // [CTAs][2][128 rows]
  float* head_whole;           // partials of whole items, by the chunks' bases
  const int32_t *members, *group_starts, *prefix_lens;   // the caller's
  int n_members, n_groups, max_chunks;
  int head_ctas, tail_ctas, tail_parts;   // (parts: that the requests' own keys are dealt to)
};

// Whether the requests' own keys go to single warps (DecodeCfg::SOLO; not where a CTA's warps share the
// queries' fragments): with two items for each CTA.  CTAs and warps, all of the call: 1024 items of up to
// 1024 keys 57.7 and 53.7 us, 4400 of up to 46 keys 67.8 and 51.7, 3968 of up to 390 keys 72.9 and 63.0;
// but 512 of up to 512 keys 48.2 and 49.5, since the join gets more parts of each item.
inline bool paged_tail_solo(int64_t items, int R, int H, int ctas) {
  return items >= 2 * ctas && (R <= 8 || (R <= 16 && H <= 128) || (R <= 32 && H == 64));
}

// Its workspace: the tables that the first kernel writes, splits, partials.
struct PagedSharedPlan {
  int max_chunks, head_ctas, tail_ctas, tail_parts;
  size_t begins, places, members, n_chunks, chunks, head_splits, tail_splits, head_partials, tail_partials,
      head_whole, tail_whole, total;
};
inline PagedSharedPlan paged_shared_plan(int B, int K, int R, int H, int n_groups, int n_members, int sm_count) {
  PagedSharedPlan p;
  const int64_t rows = (int64_t)n_members * R;
  p.max_chunks = (int)((rows + 127) / 128) + (n_groups < n_members ? n_groups : n_members);
  p.head_ctas = sm_count;
  p.tail_ctas = paged_decode_plan(R, H, sm_count).ctas;
  p.tail_parts = p.tail_ctas * (paged_tail_solo((int64_t)B * K, R, H, p.tail_ctas) ? 4 : 1);
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += ((size_t)bytes + 255) & ~(size_t)255;
    return here;
  };
  const int64_t split = sizeof(PagedDecodeSplit);
  p.begins = take((int64_t)B * 4);
  p.places = take((int64_t)B * 4);
  p.members = take((int64_t)n_members * 4);
  p.n_chunks = take(4);
  p.chunks = take((int64_t)p.max_chunks * sizeof(PagedChunk));
  p.head_splits = take((int64_t)p.max_chunks * K * split);
  p.tail_splits = take((int64_t)B * K * split);
  p.head_partials = take((int64_t)p.head_ctas * 2 * paged_partial_floats(128, H) * 4);
  p.tail_partials = take((int64_t)p.tail_parts * 2 * paged_partial_floats(R, H) * 4);
  p.head_whole = take((rows + 8 * (int64_t)p.max_chunks) * K * (H + 2) * 4);
  p.tail_whole = take((int64_t)B * K * paged_partial_floats(R, H) * 4);
  p.total = at;
  return p;
}

cudaError_t launch_paged_shared_setup(const PagedSharedArgs& a, cudaStream_t st);
cudaError_t launch_paged_shared_h64_bf16(const PagedSharedArgs& a, cudaStream_t st);
cudaError_t launch_paged_shared_h64_e4m3(const PagedSharedArgs& a, cudaStream_t st);
cudaError_t launch_paged_shared_h128_bf16(const PagedSharedArgs& a, cudaStream_t st);
cudaError_t launch_paged_shared_h128_e4m3(const PagedSharedArgs& a, cudaStream_t st);
cudaError_t launch_paged_shared_h256_bf16(const PagedSharedArgs& a, cudaStream_t st);
cudaError_t launch_paged_shared_h256_e4m3(const PagedSharedArgs& a, cudaStream_t st);

cudaError_t launch_paged_tables(const PagedTablesArgs& a, cudaStream_t st);
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st);
cudaError_t launch_paged_decode_h64_bf16(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h64_e4m3(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h128_bf16(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h128_e4m3(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h256_bf16(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h256_e4m3(const PagedDecodeArgs& a, int grid, cudaStream_t st);

}  // namespace fa
