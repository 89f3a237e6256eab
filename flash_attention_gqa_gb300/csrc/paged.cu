// Paged key-value cache: block tables and slot maps from request lengths, and new
// keys and values written into pages.
#include <cstdint>
#include <cuda_runtime.h>

#include "paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

// ----------------------------------------------------------------- tables

constexpr int kTablesThreads = 1024;

// Request b holds ceil(c_b / P) pages and needs ceil((c_b + n_b) / P): two
// exclusive sums over the requests (tokens, opened pages) place every token
// and every page.  A call that cannot be met changes nothing.
//
// Every CTA forms the sums for itself (8 bytes a request) and then fills its
// share of the tokens; nothing is exchanged.  Latency bounds it: lengths, sums,
// a search per token, its table entry, its slot (64 requests of one token 3.4 us,
// 128 with 94000 tokens 4.6 us).
// Where the outputs replace the inputs, all lengths have to be read before
// anything is written: the CTAs are then one cluster, with its barrier between.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kTablesThreads) paged_tables_kernel(const __grid_constant__ PagedTablesArgs a) {
  extern __shared__ int sm[];
  int* starts = sm;               // [B + 1] first token of each request
  int* cached = sm + a.B + 1;     // [B]
  int* taken = cached + a.B;      // [B] free pages taken before the request
  __shared__ long long warp_tok[32], warp_pg[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << a.page_shift;
  const int per = (a.B + kTablesThreads - 1) / kTablesThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  const long long most = (long long)a.max_pages << a.page_shift;

  auto pages = [&](long long n) { return (n + P - 1) >> a.page_shift; };
  bool bad = false;
  long long tok = 0, pg = 0;
  for (int b = b0; b < b1; ++b) {
    const long long c = a.cached_lens[b], n = a.new_lens[b];
    bad |= c < 0 || n < 0 || c + n > most;
    tok += n;
    pg += pages(c + n) - pages(c);
  }
  long long it = tok, ip = pg;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long t = __shfl_up_sync(~0u, it, d), p = __shfl_up_sync(~0u, ip, d);
    if (lane >= d) { it += t; ip += p; }
  }
  if (lane == 31) { warp_tok[warp] = it; warp_pg[warp] = ip; }
  __syncthreads();
  if (warp == 0) {
    long long t = warp_tok[lane], p = warp_pg[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(~0u, t, d), y = __shfl_up_sync(~0u, p, d);
      if (lane >= d) { t += x; p += y; }
    }
    warp_tok[lane] = t;
    warp_pg[lane] = p;
  }
  __syncthreads();
  const long long all_tok = warp_tok[31], all_pg = warp_pg[31];
  const int used = *a.free_used;
  bad |= all_tok > a.max_tokens || used < 0 || used + all_pg > a.n_free;
  const bool fail = __syncthreads_or(bad);
  if (!fail) {
    long long t = it - tok + (warp ? warp_tok[warp - 1] : 0);
    long long p = ip - pg + (warp ? warp_pg[warp - 1] : 0);
    for (int b = b0; b < b1; ++b) {
      const long long c = a.cached_lens[b], n = a.new_lens[b];
      starts[b] = (int)t;
      cached[b] = (int)c;
      taken[b] = (int)p;
      t += n;
      p += pages(c + n) - pages(c);
    }
    if (tid == 0) starts[a.B] = (int)all_tok;
  }
  if (IN_PLACE)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
  if (blockIdx.x != 0) {
  } else if (fail) {
    for (int b = tid; b < a.B; b += kTablesThreads) a.total_lens[b] = a.cached_lens[b];
    for (int b = tid; b <= a.B; b += kTablesThreads) a.token_starts[b] = 0;
    if (tid == 0) {
      *a.free_used_out = used;
      atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
    }
  } else {
    for (int b = tid; b < a.B; b += kTablesThreads) a.total_lens[b] = cached[b] + starts[b + 1] - starts[b];
    for (int b = tid; b <= a.B; b += kTablesThreads) a.token_starts[b] = starts[b];
    if (tid == 0) *a.free_used_out = used + (int)all_pg;
  }
  const int tokens = fail ? 0 : (int)all_tok;
#pragma unroll 2
  for (int i = blockIdx.x * kTablesThreads + tid; i < a.max_tokens; i += gridDim.x * kTablesThreads) {
    if (i >= tokens) {
      a.slots[i] = -1;
      if (a.positions) a.positions[i] = -1;
      continue;
    }
    int lo = 0, hi = a.B;   // the request with starts[b] <= i < starts[b + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= i) lo = mid; else hi = mid;
    }
    const int b = lo;
    const int pos = cached[b] + i - starts[b];
    const int col = pos >> a.page_shift, held = (int)pages(cached[b]);
    int32_t* entry = a.block_table + (int64_t)b * a.max_pages + col;
    int page;
    if (col >= held) {
      page = a.free_pages[used + taken[b] + col - held];
      if ((pos & (P - 1)) == 0) *entry = page;
    } else {
      page = *entry;
    }
    int64_t slot = ((int64_t)page << a.page_shift) + (pos & (P - 1));
    if (page < 0 || page >= a.n_pages) {
      atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
      slot = -1;
    }
    a.slots[i] = slot;
    if (a.positions) a.positions[i] = pos;
  }
}

// ----------------------------------------------------------------- append

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;   // round to nearest even, saturating at +-448; NaN stays NaN
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// A thread takes 8 head dims of a key and of the value beside it, `PER` of them
// with all loads in flight before the first store; a CTA takes `tokens` tokens.
// Bound by memory: 16000 tokens x 8 heads x 128 dims 21.6 us, 6.1 TB/s read and
// written; 64 tokens 1.5 us, a launch.
template <bool E4M3, int PER>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ PagedAppendArgs a,
                                                                      int tokens) {
  const uint32_t vecs = a.H / 8, units = a.K * vecs;      // 16-byte units of a token
  const int shift = a.H == 64 ? 3 : a.H == 128 ? 4 : 5;   // log2(vecs)
  const int64_t n0 = (int64_t)blockIdx.x * tokens;
  const uint32_t all = (uint32_t)min((int64_t)tokens, a.N - n0) * units;
  for (uint32_t i0 = threadIdx.x; i0 < all; i0 += PER * kAppendThreads) {
    uint4 xk[PER], xv[PER];
    int64_t slot[PER];
    uint32_t k[PER], u[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint32_t i = i0 + j * kAppendThreads;
      slot[j] = -1;
      if (i >= all) continue;
      const uint32_t t = i / units, rest = i - t * units;
      const int64_t n = n0 + t;
      k[j] = rest >> shift;
      u[j] = rest & (vecs - 1);
      slot[j] = a.slots[n];
      xk[j] = __ldg(reinterpret_cast<const uint4*>((const char*)a.k + n * a.k_token + k[j] * a.k_head + u[j] * 16));
      xv[j] = __ldg(reinterpret_cast<const uint4*>((const char*)a.v + n * a.v_token + k[j] * a.v_head + u[j] * 16));
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (slot[j] < 0) continue;   // padding
      const int64_t page = slot[j] >> a.lay.page_shift, in = slot[j] & ((1 << a.lay.page_shift) - 1);
      if (page >= a.lay.n_pages) {
        atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
        continue;
      }
      const int64_t dst = page * a.lay.page + k[j] * a.lay.head + in * a.lay.token;
      if (!E4M3) {
        *reinterpret_cast<uint4*>((char*)a.k_cache + dst + u[j] * 16) = xk[j];
        *reinterpret_cast<uint4*>((char*)a.v_cache + dst + u[j] * 16) = xv[j];
      } else {
        auto squeeze = [](uint4 x, float s) {
          const float2 p = unpack_bf16x2(x.x), q = unpack_bf16x2(x.y);
          const float2 r = unpack_bf16x2(x.z), t = unpack_bf16x2(x.w);
          return make_uint2(pack_e4m3x4(p.x / s, p.y / s, q.x / s, q.y / s),
                            pack_e4m3x4(r.x / s, r.y / s, t.x / s, t.y / s));
        };
        const float sk = a.k_scale ? a.k_scale[k[j]] : 1.0f, sv = a.v_scale ? a.v_scale[k[j]] : 1.0f;
        *reinterpret_cast<uint2*>((char*)a.k_cache + dst + u[j] * 8) = squeeze(xk[j], sk);
        *reinterpret_cast<uint2*>((char*)a.v_cache + dst + u[j] * 8) = squeeze(xv[j], sv);
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_tables(const PagedTablesArgs& a, cudaStream_t st) {
  const bool in_place = a.total_lens == a.cached_lens || a.free_used_out == a.free_used;
  auto* const kernel = in_place ? paged_tables_kernel<true> : paged_tables_kernel<false>;
  const size_t smem = (3 * (size_t)a.B + 1) * sizeof(int);
  // (needed from 48 KB of dynamic and static memory together on; half a KB is static.
  // Always to what the largest call needs: the limit is the function's, and a smaller one
  // would be met by the launch of another thread, or by an instantiated graph.)
  if (smem > 47 * 1024) {
    constexpr int most = (3 * kMaxPagedBatch + 1) * sizeof(int);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  // Two tokens a thread: the searches and look-ups of a token are a chain of
  // latencies (94000 tokens: 76 us in one CTA).  A cluster has at most 8 CTAs.
  int ctas = 1;
  while (ctas < (in_place ? 8 : 128) && ctas * 2 * kTablesThreads < a.max_tokens) ctas *= 2;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = in_place ? ctas : 1;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTablesThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st) {
  const int64_t units = (int64_t)a.K * (a.H / 8), all = a.N * units;
  // Four 16-byte pairs a thread once that fills the GPU (8 CTAs on each of its
  // SMs), one below.
  const bool four = all >= (int64_t)4 * kAppendThreads * 1216;
  int64_t tokens = (four ? 4 : 1) * kAppendThreads / units;
  if (tokens < 1) tokens = 1;
  const unsigned blocks = (unsigned)((a.N + tokens - 1) / tokens);
  // (cudaLaunchKernelEx: its status is this launch's, whatever error an earlier call has left)
  auto* const kernel = a.e4m3 ? (four ? paged_append_kernel<true, 4> : paged_append_kernel<true, 1>)
                              : (four ? paged_append_kernel<false, 4> : paged_append_kernel<false, 1>);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, a, (int)tokens);
}

}  // namespace fa
