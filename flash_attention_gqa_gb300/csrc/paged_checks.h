// Checks that the C entry points of the paged cache, its pages and the rotary positions share.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/fa.h"
#include "paged.h"

namespace fa {

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A required pointer of `n`-byte aligned elements.
inline bool usable(const void* p, unsigned n) { return p != nullptr && aligned(p, n); }

inline int log2_exact(int n) {
  if (n < 1 || (n & (n - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

inline bool head_dim_ok(int H) { return H == 64 || H == 128 || H == 256; }

// Checks a cache's type, strides (in elements) and page geometry, and fills
// `lay` with them in bytes.  Rows start on 16-byte boundaries.  The stride of a
// dimension of one is never used, whatever it is.
inline int make_layout(PagedLayout* lay, int cache_type, int64_t page_stride, int64_t head_stride,
                       int64_t token_stride, int K, int n_pages, int page_size) {
  if (cache_type != FA_CACHE_BF16 && cache_type != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
  if (n_pages <= 1) page_stride = 0;
  if (K <= 1) head_stride = 0;
  if (page_size == 1) token_stride = 0;
  if (n_pages < 0 || page_size < 1 || page_stride < 0 || head_stride < 0 || token_stride < 0)
    return FA_ERR_INVALID_ARG;
  const int shift = log2_exact(page_size);
  if (shift < 0 || page_size > kMaxPageSize) return FA_ERR_UNSUPPORTED;
  const int64_t es = cache_type == FA_CACHE_BF16 ? 2 : 1;
  const int64_t most = int64_t{1} << 40;
  if (page_stride > most || head_stride > most || token_stride > most) return FA_ERR_INVALID_ARG;
  if (((page_stride | head_stride | token_stride) * es) & 15) return FA_ERR_INVALID_ARG;
  *lay = PagedLayout{page_stride * es, head_stride * es, token_stride * es, n_pages, shift};
  return FA_OK;
}

// The status of a launch.  A failed one leaves nothing behind that a later call, of this library or
// of another user of the runtime, would take for its own.
inline int status(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  cudaGetLastError();
  return FA_ERR_CUDA;
}

// A call with its arguments in one record of 8-byte values, in order: addresses as integers, sizes
// as signed integers that have to fit their type, a float as its bits.
struct Record {
  const int64_t* at;
  bool ok = true;
  template <class T>
  T next() {
    const int64_t x = *at++;
    if constexpr (std::is_pointer_v<T>) {
      return reinterpret_cast<T>(static_cast<uintptr_t>(x));
    } else if constexpr (std::is_same_v<T, float>) {
      const uint32_t bits = static_cast<uint32_t>(x);
      float f;
      __builtin_memcpy(&f, &bits, 4);
      return f;
    } else {
      if (sizeof(T) < 8 && (x < INT32_MIN || x > INT32_MAX)) ok = false;
      return static_cast<T>(x);
    }
  }
};
template <class... A>
int call_packed(int (*call)(A...), const int64_t* args) {
  if (!args) return FA_ERR_INVALID_ARG;
  Record r{args};
  // (braces: the arguments are read in their order)
  struct Call {
    int rc;
    Call(int (*call)(A...), const bool& ok, A... a) : rc(ok ? call(a...) : (int)FA_ERR_INVALID_ARG) {}
  };
  return Call{call, r.ok, r.next<A>()...}.rc;
}

}  // namespace fa
