// C ABI of the rotary positions and of the page management: argument checks and launches.
// Every check happens on the host before anything is enqueued; nothing here
// allocates device memory or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "kernels.h"
#include "pages.h"
#include "paged_checks.h"
#include "rotary.h"

using namespace fa;

namespace {

constexpr int64_t kMostStride = int64_t{1} << 40;

// A tensor [B, T, heads, H] of bf16: strides in elements, rows on 16-byte boundaries.  The stride of a
// dimension of one is never used, whatever it is.
bool make_rows(RotaryRows* r, const void* at, int64_t batch, int64_t token, int64_t head, int B, int T, int heads) {
  if (B <= 1) batch = 0;
  if (T <= 1) token = 0;
  if (heads <= 1) head = 0;
  if (batch < 0 || token < 0 || head < 0 || batch > kMostStride || token > kMostStride || head > kMostStride ||
      ((batch | token | head) & 7) != 0)
    return false;
  *r = RotaryRows{const_cast<void*>(at), batch * 2, token * 2, head * 2};
  return true;
}

bool same_rows(const RotaryRows& a, const RotaryRows& b) {
  return a.batch == b.batch && a.token == b.token && a.head == b.head;
}

// What both rotary calls check: sizes, frequencies, positions.
int check_turning(RotaryArgs* a, const int32_t* positions, int64_t axis, int64_t batch, int64_t token,
                  const float* inv_freq, const int32_t* axes, int n_pairs, int n_axes, int adjacent, float q_scale,
                  int B, int T, int q_heads, int k_heads, int H) {
  if (B < 0 || T < 0 || q_heads < 0 || k_heads < 0 || H < 0 || n_pairs < 0 || n_axes < 1) return FA_ERR_INVALID_ARG;
  if (adjacent != 0 && adjacent != 1) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(q_scale)) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(H) || (int64_t)B * T > kMaxRotaryTokens || (int64_t)q_heads + 2 * (int64_t)k_heads > 65535 ||
      n_axes > kMaxRotaryAxes || n_pairs % 8 != 0 || n_pairs < 8 || 2 * n_pairs > H)
    return FA_ERR_UNSUPPORTED;
  if (n_axes <= 1) axis = 0;
  if (B <= 1) batch = 0;
  if (T <= 1) token = 0;
  if (axis < 0 || batch < 0 || token < 0 || axis > kMostStride || batch > kMostStride || token > kMostStride)
    return FA_ERR_INVALID_ARG;
  if (!aligned(axes, 4)) return FA_ERR_INVALID_ARG;
  a->positions = positions;
  a->pos_axis = axis; a->pos_batch = batch; a->pos_token = token;
  a->inv_freq = inv_freq;
  a->axes = axes;
  a->pairs = n_pairs; a->n_axes = n_axes;
  a->adjacent = adjacent != 0;
  a->q_scale = q_scale;
  a->B = B; a->T = T; a->QH = q_heads; a->KH = k_heads; a->H = H;
  return FA_OK;
}

// What the calls on tables check of a pool.
int make_pool(PagesPool* p, const int32_t* lens, const int32_t* block_table, int max_pages, int32_t* shares,
              int32_t* free_pages, int n_free, const int32_t* free_used, int B, int n_pages, int page_size) {
  if (B < 0 || max_pages < 0 || n_free < 0 || n_pages < 0 || page_size < 1) return FA_ERR_INVALID_ARG;
  const int shift = log2_exact(page_size);
  if (shift < 0 || page_size > kMaxPageSize || B > kMaxPagedBatch || n_pages > kMaxPoolPages ||
      (int64_t)max_pages * page_size > kMaxPagedLen)
    return FA_ERR_UNSUPPORTED;
  if (!usable(free_used, 4)) return FA_ERR_INVALID_ARG;
  if (B > 0 && !usable(lens, 4)) return FA_ERR_INVALID_ARG;
  if (B > 0 && max_pages > 0 && !usable(block_table, 4)) return FA_ERR_INVALID_ARG;
  if (n_pages > 0 && !usable(shares, 4)) return FA_ERR_INVALID_ARG;
  if (n_free > 0 && !usable(free_pages, 4)) return FA_ERR_INVALID_ARG;
  *p = PagesPool{lens, block_table, shares, free_pages, free_used, B, max_pages, n_pages, n_free, shift,
                 nullptr};
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_rotary(const void* q, int64_t q_batch_stride, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
              int64_t q_out_batch_stride, int64_t q_out_token_stride, int64_t q_out_head_stride, const void* k,
              int64_t k_batch_stride, int64_t k_token_stride, int64_t k_head_stride, void* k_out,
              int64_t k_out_batch_stride, int64_t k_out_token_stride, int64_t k_out_head_stride,
              const int32_t* positions, int64_t pos_axis_stride, int64_t pos_batch_stride,
              int64_t pos_token_stride, const float* inv_freq, const int32_t* axes, int n_pairs, int n_axes,
              int adjacent, int inverse, float q_scale, int B, int T, int q_heads, int k_heads, int H,
              void* stream) {
  RotaryArgs a{};
  const int rc = check_turning(&a, positions, pos_axis_stride, pos_batch_stride, pos_token_stride, inv_freq, axes,
                               n_pairs, n_axes, adjacent, q_scale, B, T, q_heads, k_heads, H);
  if (rc != FA_OK) return rc;
  if (inverse != 0 && inverse != 1) return FA_ERR_INVALID_ARG;
  a.inverse = inverse != 0;
  if (!make_rows(&a.q, q, q_batch_stride, q_token_stride, q_head_stride, B, T, q_heads) ||
      !make_rows(&a.q_out, q_out, q_out_batch_stride, q_out_token_stride, q_out_head_stride, B, T, q_heads) ||
      !make_rows(&a.k, k, k_batch_stride, k_token_stride, k_head_stride, B, T, k_heads) ||
      !make_rows(&a.k_out, k_out, k_out_batch_stride, k_out_token_stride, k_out_head_stride, B, T, k_heads))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)B * T * (q_heads + k_heads) == 0) return FA_OK;
  if (q_heads > 0 && (!usable(q, 16) || !usable(q_out, 16))) return FA_ERR_INVALID_ARG;
  if (k_heads > 0 && (!usable(k, 16) || !usable(k_out, 16))) return FA_ERR_INVALID_ARG;
  if (!usable(positions, 4) || !usable(inv_freq, 4)) return FA_ERR_INVALID_ARG;
  // In place every value is read by the thread that writes it: only with the same strides.
  if ((q_heads > 0 && q == q_out && !same_rows(a.q, a.q_out)) ||
      (k_heads > 0 && k == k_out && !same_rows(a.k, a.k_out)))
    return FA_ERR_INVALID_ARG;
  a.err = device_error_word();
  const int sms = fa_device_sm_count();
  if (!a.err || sms == 0) return FA_ERR_CUDA;
  return status(launch_rotary(a, ROTARY_PLAIN, sms, static_cast<cudaStream_t>(stream)));
}

int fa_paged_rotary_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                           int64_t q_out_batch_stride, int64_t q_out_token_stride, int64_t q_out_head_stride,
                           const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                           int64_t v_token_stride, int64_t v_head_stride, const int32_t* positions,
                           int64_t pos_axis_stride, int64_t pos_token_stride, const float* inv_freq,
                           const int32_t* axes, int n_pairs, int n_axes, int adjacent, float q_scale,
                           const int64_t* slots, void* k_cache, void* v_cache, int cache_type,
                           const float* k_scale, const float* v_scale, int64_t page_stride, int64_t head_stride,
                           int64_t token_stride, int B, int T, int q_heads, int k_heads, int H, int n_pages,
                           int page_size, void* stream) {
  RotaryArgs a{};
  int rc = check_turning(&a, positions, pos_axis_stride, 0, pos_token_stride, inv_freq, axes, n_pairs, n_axes,
                         adjacent, q_scale, B, T, q_heads, k_heads, H);
  if (rc != FA_OK) return rc;
  rc = make_layout(&a.lay, cache_type, page_stride, head_stride, token_stride, k_heads, n_pages, page_size);
  if (rc != FA_OK) return rc;
  // Tokens are numbered b * T + t: a batch is T token strides on.
  const int64_t N = (int64_t)B * T;
  if (N <= 1) q_token_stride = k_token_stride = v_token_stride = pos_token_stride = 0;
  const int64_t most = (int64_t{1} << 60) / (T > 0 ? T : 1);   // a batch's stride fits
  if (pos_token_stride < 0 || pos_token_stride > most) return FA_ERR_INVALID_ARG;
  a.pos_token = pos_token_stride;
  a.pos_batch = pos_token_stride * T;
  auto flat = [&](RotaryRows* r, const void* at, int64_t token, int64_t head, int heads) {
    if (token > most / 2 || !make_rows(r, at, 0, token, head, 1, 2, heads)) return false;
    r->batch = r->token * T;
    return true;
  };
  if (!flat(&a.q, q, q_token_stride, q_head_stride, q_heads) || !flat(&a.k, k, k_token_stride, k_head_stride, k_heads) ||
      !flat(&a.v, v, v_token_stride, v_head_stride, k_heads) ||
      !make_rows(&a.q_out, q_out, q_out_batch_stride, q_out_token_stride, q_out_head_stride, B, T, q_heads))
    return FA_ERR_INVALID_ARG;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return FA_ERR_INVALID_ARG;
  if (cache_type == FA_CACHE_BF16 && (k_scale || v_scale)) return FA_ERR_INVALID_ARG;
  if (N * (q_heads + k_heads) == 0) return FA_OK;
  if (q_heads > 0 && (!usable(q, 16) || !usable(q_out, 16))) return FA_ERR_INVALID_ARG;
  if (k_heads > 0 && (!usable(k, 16) || !usable(v, 16))) return FA_ERR_INVALID_ARG;
  if (k_heads > 0 && n_pages > 0 && (!usable(k_cache, 16) || !usable(v_cache, 16))) return FA_ERR_INVALID_ARG;
  if (!usable(positions, 4) || !usable(inv_freq, 4) || !usable(slots, 8)) return FA_ERR_INVALID_ARG;
  if (q_heads > 0 && q == q_out && !same_rows(a.q, a.q_out)) return FA_ERR_INVALID_ARG;
  a.slots = slots;
  a.k_cache = k_cache; a.v_cache = v_cache;
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.err = device_error_word();
  const int sms = fa_device_sm_count();
  if (!a.err || sms == 0) return FA_ERR_CUDA;
  return status(launch_rotary(a, cache_type == FA_CACHE_E4M3 ? ROTARY_E4M3 : ROTARY_BF16, sms,
                              static_cast<cudaStream_t>(stream)));
}

int fa_paged_free(const int32_t* rows, const int32_t* keep, int N, const int32_t* lens, const int32_t* block_table,
                  int max_pages, int32_t* shares, int32_t* free_pages, int n_free, const int32_t* free_used,
                  int32_t* lens_out, int32_t* free_used_out, int B, int n_pages, int page_size, void* stream) {
  PagesFreeArgs a{};
  const int rc = make_pool(&a.p, lens, block_table, max_pages, shares, free_pages, n_free, free_used, B, n_pages,
                           page_size);
  if (rc != FA_OK) return rc;
  if (N < 0) return FA_ERR_INVALID_ARG;
  if (N > kMaxPagedBatch) return FA_ERR_UNSUPPORTED;
  if ((N > 0 && !usable(rows, 4)) || !aligned(keep, 4)) return FA_ERR_INVALID_ARG;
  if ((B > 0 && !usable(lens_out, 4)) || !usable(free_used_out, 4)) return FA_ERR_INVALID_ARG;
  a.rows = rows;
  a.keep = keep;
  a.lens_out = lens_out;
  a.free_used_out = free_used_out;
  a.N = N;
  a.p.err = device_error_word();
  if (!a.p.err) return FA_ERR_CUDA;
  return status(launch_pages_free(a, static_cast<cudaStream_t>(stream)));
}

int fa_paged_fork(const int32_t* parents, const int32_t* children, const int32_t* fork_lens, int N,
                  const int32_t* lens, int32_t* block_table, int max_pages, int32_t* shares,
                  const int32_t* free_pages, int n_free, const int32_t* free_used, int32_t* lens_out,
                  int32_t* copies, int32_t* free_used_out, int B, int n_pages, int page_size, void* stream) {
  PagesForkArgs a{};
  const int rc = make_pool(&a.p, lens, block_table, max_pages, shares, const_cast<int32_t*>(free_pages), n_free,
                           free_used, B, n_pages, page_size);
  if (rc != FA_OK) return rc;
  if (N < 0) return FA_ERR_INVALID_ARG;
  if (N > kMaxPagedBatch) return FA_ERR_UNSUPPORTED;
  if (N > 0 && (!usable(parents, 4) || !usable(children, 4) || !usable(copies, 4))) return FA_ERR_INVALID_ARG;
  if (!aligned(fork_lens, 4)) return FA_ERR_INVALID_ARG;
  if ((B > 0 && !usable(lens_out, 4)) || !usable(free_used_out, 4)) return FA_ERR_INVALID_ARG;
  a.parents = parents;
  a.children = children;
  a.fork_lens = fork_lens;
  a.table = block_table;
  a.lens_out = lens_out;
  a.free_used_out = free_used_out;
  a.copies = copies;
  a.N = N;
  a.p.err = device_error_word();
  if (!a.p.err) return FA_ERR_CUDA;
  return status(launch_pages_fork(a, static_cast<cudaStream_t>(stream)));
}

int fa_paged_compact(const int32_t* lens, const int32_t* block_table, int max_pages, const int32_t* shares,
                     const int32_t* free_pages, int n_free, const int32_t* free_used, int32_t* block_table_out,
                     int32_t* shares_out, int32_t* free_pages_out, int32_t* moves, int max_moves, int B, int n_pages,
                     int page_size, void* stream) {
  PagesCompactArgs a{};
  const int rc = make_pool(&a.p, lens, block_table, max_pages, const_cast<int32_t*>(shares),
                           const_cast<int32_t*>(free_pages), n_free, free_used, B, n_pages, page_size);
  if (rc != FA_OK) return rc;
  if (max_moves < 0) return FA_ERR_INVALID_ARG;
  if (B > 0 && max_pages > 0 && !usable(block_table_out, 4)) return FA_ERR_INVALID_ARG;
  if (n_pages > 0 && !usable(shares_out, 4)) return FA_ERR_INVALID_ARG;
  if (n_free > 0 && !usable(free_pages_out, 4)) return FA_ERR_INVALID_ARG;
  if (max_moves > 0 && !usable(moves, 4)) return FA_ERR_INVALID_ARG;
  a.table_out = block_table_out;
  a.shares_out = shares_out;
  a.free_out = free_pages_out;
  a.moves = moves;
  a.max_moves = max_moves;
  a.p.err = device_error_word();
  if (!a.p.err) return FA_ERR_CUDA;
  return status(launch_pages_compact(a, static_cast<cudaStream_t>(stream)));
}

int fa_paged_copy(const int32_t* moves, int N, void* k_cache, void* v_cache, int cache_type, int64_t layer_stride,
                  int64_t page_stride, int64_t head_stride, int64_t token_stride, int layers, int K, int H,
                  int n_pages, int page_size, void* stream) {
  if (N < 0 || layers < 0 || K < 0 || H < 0) return FA_ERR_INVALID_ARG;
  PagesCopyArgs a{};
  const int rc = make_layout(&a.lay, cache_type, page_stride, head_stride, token_stride, K, n_pages, page_size);
  if (rc != FA_OK) return rc;
  const int es = cache_type == FA_CACHE_BF16 ? 2 : 1;
  if (layers <= 1) layer_stride = 0;
  if (layer_stride < 0 || layer_stride > kMostStride || (layer_stride * es & 15) != 0) return FA_ERR_INVALID_ARG;
  if (!head_dim_ok(H) || layers > kMaxCopyLayers || K > 65535) return FA_ERR_UNSUPPORTED;
  // (units of a page are counted in 32 bits, parts of all moves in a grid)
  const int64_t units = (int64_t)K * page_size * (H * es / 16);
  if (units > INT32_MAX || ((units + 2047) / 2048) * N > INT32_MAX) return FA_ERR_UNSUPPORTED;
  if (N == 0 || layers == 0 || K == 0) return FA_OK;
  if (!usable(moves, 4)) return FA_ERR_INVALID_ARG;
  if (n_pages > 0 && (!usable(k_cache, 16) || !usable(v_cache, 16))) return FA_ERR_INVALID_ARG;
  a.moves = moves;
  a.k_cache = k_cache; a.v_cache = v_cache;
  a.layer = layer_stride * es;
  a.N = N; a.layers = layers; a.K = K; a.row_bytes = H * es;
  a.err = device_error_word();
  if (!a.err) return FA_ERR_CUDA;
  return status(launch_pages_copy(a, static_cast<cudaStream_t>(stream)));
}

int fa_rotary_packed(const int64_t* args) { return call_packed(fa_rotary, args); }
int fa_paged_rotary_append_packed(const int64_t* args) { return call_packed(fa_paged_rotary_append, args); }
int fa_paged_free_packed(const int64_t* args) { return call_packed(fa_paged_free, args); }
int fa_paged_fork_packed(const int64_t* args) { return call_packed(fa_paged_fork, args); }
int fa_paged_compact_packed(const int64_t* args) { return call_packed(fa_paged_compact, args); }
int fa_paged_copy_packed(const int64_t* args) { return call_packed(fa_paged_copy, args); }

}  // extern "C"
