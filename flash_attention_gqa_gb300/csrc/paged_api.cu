// C ABI of the paged key-value cache operators: argument checks and launches.
// Every check happens on the host before anything is enqueued; nothing here
// allocates device memory or synchronises.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/fa.h"
#include "kernels.h"
#include "paged.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A required pointer of `n`-byte aligned elements.
bool usable(const void* p, unsigned n) { return p != nullptr && aligned(p, n); }

int log2_exact(int n) {
  if (n < 1 || (n & (n - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

bool head_dim_ok(int H) { return H == 64 || H == 128 || H == 256; }

// Checks a cache's type, strides (in elements) and page geometry, and fills
// `lay` with them in bytes.  Rows start on 16-byte boundaries.  The stride of a
// dimension of one is never used, whatever it is.
int make_layout(fa::PagedLayout* lay, int cache_type, int64_t page_stride, int64_t head_stride,
                int64_t token_stride, int K, int n_pages, int page_size) {
  if (cache_type != FA_CACHE_BF16 && cache_type != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
  if (n_pages <= 1) page_stride = 0;
  if (K <= 1) head_stride = 0;
  if (page_size == 1) token_stride = 0;
  if (n_pages < 0 || page_size < 1 || page_stride < 0 || head_stride < 0 || token_stride < 0)
    return FA_ERR_INVALID_ARG;
  const int shift = log2_exact(page_size);
  if (shift < 0 || page_size > fa::kMaxPageSize) return FA_ERR_UNSUPPORTED;
  const int64_t es = cache_type == FA_CACHE_BF16 ? 2 : 1;
  const int64_t most = int64_t{1} << 40;
  if (page_stride > most || head_stride > most || token_stride > most) return FA_ERR_INVALID_ARG;
  if (((page_stride | head_stride | token_stride) * es) & 15) return FA_ERR_INVALID_ARG;
  *lay = fa::PagedLayout{page_stride * es, head_stride * es, token_stride * es, n_pages, shift};
  return FA_OK;
}

bool decode_shape_ok(int B, int K, int G, int T, int H) {
  return head_dim_ok(H) && (int64_t)G * T <= fa::kMaxPagedRows && B <= fa::kMaxPagedBatch &&
         (int64_t)B * K <= 65535;
}

// The status of a launch.  A failed one leaves nothing behind that a later call, of this library or
// of another user of the runtime, would take for its own.
int status(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  cudaGetLastError();
  return FA_ERR_CUDA;
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

int fa_paged_decode(const void* q, const void* k_cache, const void* v_cache, int cache_type,
                    const float* k_scale, const float* v_scale, int64_t page_stride,
                    int64_t head_stride, int64_t token_stride, const int32_t* block_table,
                    const int32_t* lens, int window, void* o, float* lse, void* workspace,
                    size_t workspace_bytes, int B, int K, int G, int T, int H, int n_pages,
                    int page_size, int max_pages, void* stream) {
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

}  // extern "C"

namespace {

// Reads a record of 8-byte arguments in order; `ok` falls where a size does not
// fit an int.
struct Record {
  const int64_t* at;
  bool ok = true;
  template <class T>
  T* ptr() { return reinterpret_cast<T*>(static_cast<uintptr_t>(*at++)); }
  int64_t wide() { return *at++; }
  int size() {
    const int64_t x = *at++;
    if (x < INT32_MIN || x > INT32_MAX) ok = false;
    return static_cast<int>(x);
  }
};

}  // namespace

extern "C" {

int fa_paged_tables_packed(const int64_t* args) {
  if (!args) return FA_ERR_INVALID_ARG;
  Record r{args};
  const auto* cached = r.ptr<const int32_t>();
  const auto* fresh = r.ptr<const int32_t>();
  const auto* free_pages = r.ptr<const int32_t>();
  const int n_free = r.size();
  const auto* used = r.ptr<const int32_t>();
  auto* table = r.ptr<int32_t>();
  const int max_pages = r.size();
  auto* total = r.ptr<int32_t>();
  auto* starts = r.ptr<int32_t>();
  auto* slots = r.ptr<int64_t>();
  auto* positions = r.ptr<int32_t>();
  const int max_tokens = r.size();
  auto* used_out = r.ptr<int32_t>();
  const int B = r.size(), n_pages = r.size(), page_size = r.size();
  void* stream = r.ptr<void>();
  if (!r.ok) return FA_ERR_INVALID_ARG;
  return fa_paged_tables(cached, fresh, free_pages, n_free, used, table, max_pages, total, starts, slots,
                         positions, max_tokens, used_out, B, n_pages, page_size, stream);
}

int fa_paged_append_packed(const int64_t* args) {
  if (!args) return FA_ERR_INVALID_ARG;
  Record r{args};
  const void* k = r.ptr<const void>();
  const void* v = r.ptr<const void>();
  const int64_t kt = r.wide(), kh = r.wide(), vt = r.wide(), vh = r.wide();
  const auto* slots = r.ptr<const int64_t>();
  void* kc = r.ptr<void>();
  void* vc = r.ptr<void>();
  const int type = r.size();
  const auto* ks = r.ptr<const float>();
  const auto* vs = r.ptr<const float>();
  const int64_t page = r.wide(), head = r.wide(), token = r.wide();
  const int N = r.size(), K = r.size(), H = r.size(), n_pages = r.size(), page_size = r.size();
  void* stream = r.ptr<void>();
  if (!r.ok) return FA_ERR_INVALID_ARG;
  return fa_paged_append(k, v, kt, kh, vt, vh, slots, kc, vc, type, ks, vs, page, head, token, N, K, H,
                         n_pages, page_size, stream);
}

int fa_paged_decode_packed(const int64_t* args) {
  if (!args) return FA_ERR_INVALID_ARG;
  Record r{args};
  const void* q = r.ptr<const void>();
  const void* kc = r.ptr<const void>();
  const void* vc = r.ptr<const void>();
  const int type = r.size();
  const auto* ks = r.ptr<const float>();
  const auto* vs = r.ptr<const float>();
  const int64_t page = r.wide(), head = r.wide(), token = r.wide();
  const auto* table = r.ptr<const int32_t>();
  const auto* lens = r.ptr<const int32_t>();
  const int window = r.size();
  void* o = r.ptr<void>();
  auto* lse = r.ptr<float>();
  void* workspace = r.ptr<void>();
  const size_t bytes = static_cast<size_t>(r.wide());
  const int B = r.size(), K = r.size(), G = r.size(), T = r.size(), H = r.size();
  const int n_pages = r.size(), page_size = r.size(), max_pages = r.size();
  void* stream = r.ptr<void>();
  if (!r.ok) return FA_ERR_INVALID_ARG;
  return fa_paged_decode(q, kc, vc, type, ks, vs, page, head, token, table, lens, window, o, lse, workspace,
                         bytes, B, K, G, T, H, n_pages, page_size, max_pages, stream);
}

}  // extern "C"
