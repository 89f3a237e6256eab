// Internal interface of the paged key-value cache operators (paged.cu).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

constexpr int kMaxPagedBatch = 8192;       // requests of one call: their offsets stay in shared memory
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
  uint32_t* err;
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

cudaError_t launch_paged_tables(const PagedTablesArgs& a, cudaStream_t st);
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st);
cudaError_t launch_paged_decode_h64_bf16(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h64_e4m3(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h128_bf16(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h128_e4m3(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h256_bf16(const PagedDecodeArgs& a, int grid, cudaStream_t st);
cudaError_t launch_paged_decode_h256_e4m3(const PagedDecodeArgs& a, int grid, cudaStream_t st);

}  // namespace fa
