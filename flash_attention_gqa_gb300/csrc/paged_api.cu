// C ABI of the paged key-value cache operators: argument checks and launches.
// Every check happens on the host before anything is enqueued; nothing here
// allocates device memory or synchronises.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/fa.h"
#include "kernels.h"
#include "paged.h"
#include "paged_checks.h"

using namespace fa;

namespace {

// Bytes of keys and values, each request's counted as far as its row of the table reaches (lengths are on the
// device), up to which a call with shared prefixes does not make use of them: the three grids that it takes more
// cost some 10 us, what several requests read comes from L2, and a tile of 128 rows takes its time however few of
// them there are.  Shared and not, in us: bf16 at H = 128, 16 requests of one prefix x 8 kv heads x 2112 keys
// (138 MB) 21 and 19, x 8256 (541 MB) 24 and 52; 64 x 8 x 576 (151 MB) 27 and 22; e4m3 64 x 8 x 2112 (277 MB) 29
// and 39, 48 in threes x 4 x 4112 (202 MB) 34 and 29, 48 in fours x 4 x 16400 (806 MB) 67 and 104.  In pairs, 48
// requests x 4 heads: bf16 at H = 64 x 4112 (202 MB) 36 and 26, at H = 128 (404 MB) 49 and 60; e4m3 at H = 64 x 16400
// (403 MB) 84 and 79, at H = 256 x 4112 (404 MB) 73 and 60, at H = 128 x 16400 (806 MB) 107 and 124.
// The rule looks at neither the head dim nor how many share beyond three: the threes above are on its wrong side, by
// 5 us of 29.  And where a table reaches far behind its requests it takes the grids for few keys: with a table for
// 32768 tokens, 4 requests x 2 heads x 552 keys at H = 256 17.8 us and 8.9, 64 x 8 x 576 27.0 and 22.6, 16 x 8 x 2112
// 24.3 and 19.6.
inline double shared_least(bool bf16, int n_groups, int n_members) {
  return n_members >= 3 * (int64_t)n_groups ? 200e6 : bf16 ? 400e6 : 800e6;
}

bool decode_shape_ok(int B, int K, int G, int T, int H) {
  return head_dim_ok(H) && (int64_t)G * T <= kMaxPagedRows && B <= kMaxPagedBatch &&
         (int64_t)B * K <= 65535;
}

}  // namespace

extern "C" {

int fa_paged_tables(const int32_t* cached_lens, const int32_t* new_lens, const int32_t* free_pages,
                    int n_free, const int32_t* free_used, int32_t* block_table, int max_pages,
                    int32_t* total_lens, int32_t* token_starts, int64_t* slots, int32_t* positions,
                    int max_tokens, int32_t* free_used_out, int B, int n_pages, int page_size,
                    void* stream) {
  if (B < 0 || n_free < 0 || max_pages < 0 || max_tokens < 0 || n_pages < 0 || page_size < 1)
    return FA_ERR_INVALID_ARG;
  const int shift = log2_exact(page_size);
  if (shift < 0 || page_size > fa::kMaxPageSize || B > fa::kMaxPagedBatch) return FA_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * page_size > fa::kMaxPagedLen || max_tokens > fa::kMaxPagedLen)
    return FA_ERR_UNSUPPORTED;
  if (!usable(token_starts, 4) || !usable(free_used, 4) || !usable(free_used_out, 4))
    return FA_ERR_INVALID_ARG;
  if (B > 0 && (!usable(cached_lens, 4) || !usable(new_lens, 4) || !usable(total_lens, 4)))
    return FA_ERR_INVALID_ARG;
  if (n_free > 0 && !usable(free_pages, 4)) return FA_ERR_INVALID_ARG;
  if (B > 0 && max_pages > 0 && !usable(block_table, 4)) return FA_ERR_INVALID_ARG;
  if (max_tokens > 0 && !usable(slots, 8)) return FA_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return FA_ERR_INVALID_ARG;
  fa::PagedTablesArgs a{};
  a.cached_lens = cached_lens;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.free_used = free_used;
  a.block_table = block_table;
  a.total_lens = total_lens;
  a.token_starts = token_starts;
  a.slots = slots;
  a.positions = positions;
  a.free_used_out = free_used_out;
  a.B = B; a.n_free = n_free; a.n_pages = n_pages;
  a.page_shift = shift; a.max_pages = max_pages; a.max_tokens = max_tokens;
  a.err = fa::device_error_word();
  if (!a.err) return FA_ERR_CUDA;
  return status(fa::launch_paged_tables(a, static_cast<cudaStream_t>(stream)));
}

int fa_paged_append(const void* k, const void* v, int64_t k_token_stride, int64_t k_head_stride,
                    int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                    void* k_cache, void* v_cache, int cache_type, const float* k_scale,
                    const float* v_scale, int64_t page_stride, int64_t head_stride,
                    int64_t token_stride, int N, int K, int H, int n_pages, int page_size,
                    void* stream) {
  if (N < 0 || K < 0 || H < 0) return FA_ERR_INVALID_ARG;
  fa::PagedAppendArgs a{};
  const int rc = make_layout(&a.lay, cache_type, page_stride, head_stride, token_stride, K, n_pages, page_size);
  if (rc != FA_OK) return rc;
  if (!head_dim_ok(H) || K > 65535) return FA_ERR_UNSUPPORTED;
  if (N <= 1) k_token_stride = v_token_stride = 0;
  if (K <= 1) k_head_stride = v_head_stride = 0;
  const int64_t most = int64_t{1} << 40;
  if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0 ||
      k_token_stride > most || k_head_stride > most || v_token_stride > most || v_head_stride > most ||
      ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7))
    return FA_ERR_INVALID_ARG;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return FA_ERR_INVALID_ARG;
  if (cache_type == FA_CACHE_BF16 && (k_scale || v_scale)) return FA_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return FA_OK;
  if (!usable(k, 16) || !usable(v, 16) || !usable(slots, 8)) return FA_ERR_INVALID_ARG;
  if (n_pages > 0 && (!usable(k_cache, 16) || !usable(v_cache, 16))) return FA_ERR_INVALID_ARG;
  a.k = k; a.v = v;
  a.k_token = k_token_stride * 2; a.k_head = k_head_stride * 2;
  a.v_token = v_token_stride * 2; a.v_head = v_head_stride * 2;
  a.slots = slots;
  a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.N = N; a.K = K; a.H = H;
  a.e4m3 = cache_type == FA_CACHE_E4M3;
  a.err = fa::device_error_word();
  if (!a.err) return FA_ERR_CUDA;
  return status(fa::launch_paged_append(a, static_cast<cudaStream_t>(stream)));
}

size_t fa_paged_decode_workspace_size(int B, int K, int G, int T, int H) {
  if (B <= 0 || K <= 0 || G <= 0 || T <= 0 || !decode_shape_ok(B, K, G, T, H)) return 0;
  return fa::paged_decode_plan(G * T, H, fa_device_sm_count()).total;
}

// `by_warps`: as in PagedDecodeArgs.  (fa_paged_decode leaves short items to CTAs, whose sums come in another
// order: its results stay what they were.)
static int decode(bool by_warps, const void* q, const void* k_cache, const void* v_cache, int cache_type,
                  const float* k_scale, const float* v_scale, int64_t page_stride, int64_t head_stride,
                  int64_t token_stride, const int32_t* block_table, const int32_t* lens, int window, void* o,
                  float* lse, void* workspace, size_t workspace_bytes, int B, int K, int G, int T, int H,
                  int n_pages, int page_size, int max_pages, void* stream) {
  if (B < 0 || K < 0 || G < 0 || T < 0 || H < 0 || max_pages < 0 || window < 0)
    return FA_ERR_INVALID_ARG;
  fa::PagedDecodeArgs a{};
  const int rc = make_layout(&a.lay, cache_type, page_stride, head_stride, token_stride, K, n_pages, page_size);
  if (rc != FA_OK) return rc;
  if (!decode_shape_ok(B, K, G, T, H) || (int64_t)max_pages * page_size > fa::kMaxPagedLen)
    return FA_ERR_UNSUPPORTED;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return FA_ERR_INVALID_ARG;
  if (cache_type == FA_CACHE_BF16 && (k_scale || v_scale)) return FA_ERR_INVALID_ARG;
  if ((int64_t)B * K * G * T == 0) return FA_OK;
  if (!usable(q, 16) || !usable(o, 16) || !usable(lse, 4) || !usable(lens, 4)) return FA_ERR_INVALID_ARG;
  if (max_pages > 0 && !usable(block_table, 4)) return FA_ERR_INVALID_ARG;
  if (n_pages > 0 && (!usable(k_cache, 16) || !usable(v_cache, 16))) return FA_ERR_INVALID_ARG;
  const fa::PagedDecodePlan plan = fa::paged_decode_plan(G * T, H, fa_device_sm_count());
  if (!usable(workspace, 256) || workspace_bytes < plan.total) return FA_ERR_INVALID_ARG;
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.block_table = block_table; a.lens = lens;
  a.o = o; a.lse = lse;
  a.B = B; a.K = K; a.G = G; a.T = T; a.H = H; a.max_pages = max_pages;
  // A window that reaches past the longest request is none.
  a.window = window >= max_pages * page_size ? 0 : window;
  a.splits = static_cast<fa::PagedDecodeSplit*>(workspace);
  a.by_item = B * K <= plan.ctas;
  a.by_warps = by_warps;
  a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.partials);
  a.wait_limit_ns = fa::device_wait_limit_ns();
  a.err = fa::device_error_word();
  if (!a.err || plan.ctas == 0) return FA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache_type == FA_CACHE_E4M3;
  switch (H) {
    case 64:
      return status(e4m3 ? fa::launch_paged_decode_h64_e4m3(a, plan.ctas, st)
                         : fa::launch_paged_decode_h64_bf16(a, plan.ctas, st));
    case 128:
      return status(e4m3 ? fa::launch_paged_decode_h128_e4m3(a, plan.ctas, st)
                         : fa::launch_paged_decode_h128_bf16(a, plan.ctas, st));
    default:
      return status(e4m3 ? fa::launch_paged_decode_h256_e4m3(a, plan.ctas, st)
                         : fa::launch_paged_decode_h256_bf16(a, plan.ctas, st));
  }
}

int fa_paged_decode(const void* q, const void* k_cache, const void* v_cache, int cache_type,
                    const float* k_scale, const float* v_scale, int64_t page_stride,
                    int64_t head_stride, int64_t token_stride, const int32_t* block_table,
                    const int32_t* lens, int window, void* o, float* lse, void* workspace,
                    size_t workspace_bytes, int B, int K, int G, int T, int H, int n_pages,
                    int page_size, int max_pages, void* stream) {
  return decode(false, q, k_cache, v_cache, cache_type, k_scale, v_scale, page_stride, head_stride, token_stride,
                block_table, lens, window, o, lse, workspace, workspace_bytes, B, K, G, T, H, n_pages, page_size,
                max_pages, stream);
}

size_t fa_paged_decode_shared_workspace_size(int B, int K, int G, int T, int H, int n_groups, int n_members) {
  if (B <= 0 || K <= 0 || G <= 0 || T <= 0 || !decode_shape_ok(B, K, G, T, H)) return 0;
  if (n_groups < 0 || n_members < 0 || n_groups > kMaxPagedGroups || n_members > B) return 0;
  const size_t shared = paged_shared_plan(B, K, G * T, H, n_groups, n_members, fa_device_sm_count()).total;
  return std::max(shared, fa_paged_decode_workspace_size(B, K, G, T, H));   // (small calls are decodes)
}

int fa_paged_decode_shared(const void* q, const void* k_cache, const void* v_cache, int cache_type,
                           const float* k_scale, const float* v_scale, int64_t page_stride, int64_t head_stride,
                           int64_t token_stride, const int32_t* block_table, const int32_t* lens,
                           const int32_t* members, int n_members, const int32_t* group_starts,
                           const int32_t* prefix_lens, int n_groups, void* o, float* lse, void* workspace,
                           size_t workspace_bytes, int B, int K, int G, int T, int H, int n_pages, int page_size,
                           int max_pages, void* stream) {
  if (B < 0 || K < 0 || G < 0 || T < 0 || H < 0 || max_pages < 0 || n_members < 0 || n_groups < 0)
    return FA_ERR_INVALID_ARG;
  PagedSharedArgs s{};
  PagedDecodeArgs& a = s.tail;
  const int rc = make_layout(&a.lay, cache_type, page_stride, head_stride, token_stride, K, n_pages, page_size);
  if (rc != FA_OK) return rc;
  if (!decode_shape_ok(B, K, G, T, H) || (int64_t)max_pages * page_size > kMaxPagedLen || n_groups > kMaxPagedGroups)
    return FA_ERR_UNSUPPORTED;
  if (n_members > B) return FA_ERR_INVALID_ARG;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return FA_ERR_INVALID_ARG;
  if (cache_type == FA_CACHE_BF16 && (k_scale || v_scale)) return FA_ERR_INVALID_ARG;
  if ((int64_t)B * K * G * T == 0) return FA_OK;
  if (!usable(q, 16) || !usable(o, 16) || !usable(lse, 4) || !usable(lens, 4)) return FA_ERR_INVALID_ARG;
  if (max_pages > 0 && !usable(block_table, 4)) return FA_ERR_INVALID_ARG;
  if (n_pages > 0 && (!usable(k_cache, 16) || !usable(v_cache, 16))) return FA_ERR_INVALID_ARG;
  if (n_members > 0 && !usable(members, 4)) return FA_ERR_INVALID_ARG;
  if (!usable(group_starts, 4) || (n_groups > 0 && !usable(prefix_lens, 4))) return FA_ERR_INVALID_ARG;
  const PagedSharedPlan plan = paged_shared_plan(B, K, G * T, H, n_groups, n_members, fa_device_sm_count());
  if (!usable(workspace, 256) || workspace_bytes < std::max(plan.total, paged_decode_plan(G * T, H, fa_device_sm_count()).total))
    return FA_ERR_INVALID_ARG;
  // (With a group for every member nothing is shared.)
  const double keys = (double)n_members * max_pages * page_size * K * H * (cache_type == FA_CACHE_BF16 ? 4 : 2);
  if (n_groups >= n_members || keys <= shared_least(cache_type == FA_CACHE_BF16, n_groups, n_members))
    return decode(true, q, k_cache, v_cache, cache_type, k_scale, v_scale, page_stride, head_stride, token_stride,
                  block_table, lens, 0, o, lse, workspace, workspace_bytes, B, K, G, T, H, n_pages, page_size,
                  max_pages, stream);
  char* const ws = static_cast<char*>(workspace);
  a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.block_table = block_table; a.lens = lens;
  a.o = o; a.lse = lse;
  a.B = B; a.K = K; a.G = G; a.T = T; a.H = H; a.max_pages = max_pages;
  a.by_item = true;
  a.splits = reinterpret_cast<PagedDecodeSplit*>(ws + plan.tail_splits);
  a.partials = reinterpret_cast<float*>(ws + plan.tail_partials);
  a.shared.begins = reinterpret_cast<int32_t*>(ws + plan.begins);
  a.shared.places = reinterpret_cast<int32_t*>(ws + plan.places);
  a.shared.members = reinterpret_cast<int32_t*>(ws + plan.members);
  a.shared.n_chunks = reinterpret_cast<int32_t*>(ws + plan.n_chunks);
  a.shared.chunks = reinterpret_cast<PagedChunk*>(ws + plan.chunks);
  a.shared.whole = reinterpret_cast<float*>(ws + plan.tail_whole);
  s.head_splits = reinterpret_cast<PagedDecodeSplit*>(ws + plan.head_splits);
  s.head_partials = reinterpret_cast<float*>(ws + plan.head_partials);
  s.head_whole = reinterpret_cast<float*>(ws + plan.head_whole);
  s.members = members; s.group_starts = group_starts; s.prefix_lens = prefix_lens;
  s.n_members = n_members; s.n_groups = n_groups; s.max_chunks = plan.max_chunks;
  s.head_ctas = plan.head_ctas; s.tail_ctas = plan.tail_ctas; s.tail_parts = plan.tail_parts;
  a.wait_limit_ns = device_wait_limit_ns();
  a.err = device_error_word();
  if (!a.err || plan.tail_ctas == 0) return FA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache_type == FA_CACHE_E4M3;
  switch (H) {
    case 64: return status(e4m3 ? launch_paged_shared_h64_e4m3(s, st) : launch_paged_shared_h64_bf16(s, st));
    case 128: return status(e4m3 ? launch_paged_shared_h128_e4m3(s, st) : launch_paged_shared_h128_bf16(s, st));
    default: return status(e4m3 ? launch_paged_shared_h256_e4m3(s, st) : launch_paged_shared_h256_bf16(s, st));
  }
}

int fa_paged_tables_packed(const int64_t* args) { return call_packed(fa_paged_tables, args); }
int fa_paged_append_packed(const int64_t* args) { return call_packed(fa_paged_append, args); }
int fa_paged_decode_packed(const int64_t* args) { return call_packed(fa_paged_decode, args); }
int fa_paged_decode_shared_packed(const int64_t* args) { return call_packed(fa_paged_decode_shared, args); }

}  // extern "C"
