// Attention of requests that share prefixes, its first kernel: who shares what.
//
// Checks the caller's groups and writes what the others go by (paged.h): the first key that each
// request has for itself, where its rows are among its group's, and the groups' rows in chunks of
// 128.  Whatever does not hold together is not shared, and reported: every request's keys are then
// its own, and its result is the same.  A group of one shares nothing either.  Latency bounds it (one
// CTA; the grids behind it are launched while it runs): 3.5 us of a call for 64 members, two trips to memory and
// six barriers; 1.2 more with 1024 threads, whose barriers take longer.
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "paged.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 1024;

// Entry of a sorted list of n + 1 with list[e] <= x < list[e + 1].
__device__ __forceinline__ int entry_of(const int* list, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (list[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads, 1) paged_shared_setup_kernel(const __grid_constant__ PagedSharedArgs a) {
  extern __shared__ int sm[];
  const int n = a.n_groups, N = a.n_members, B = a.tail.B, T = a.tail.T, R = a.tail.G * T, tid = threadIdx.x;
  const int threads = blockDim.x;
  int* const starts = sm;              // [n + 1]
  int* const prefix = starts + n + 1;  // [n] the caller's, then what is shared
  int* const least = prefix + n;       // [n] longest prefix that all members' queries see
  int* const lead = least + n;         // [n] lowest entry with a request, then that request
  int* const live = lead + n;          // [n] entries with one
  int* const first = live + n;         // [n + 1] chunks before the group
  int* const base = first + n + 1;     // [n] padded rows before it
  int* const claim = base + n;         // [B] lowest entry that names the request
  __shared__ int sums[2][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const PagedSharedTables& out = a.tail.shared;
  const int most = a.tail.max_pages << a.tail.lay.page_shift;
  // Two trips to memory, where the members are no more than the threads: members and groups, lengths.
  int member = -1, len = 0;   // of entry tid
  if (tid < N) member = a.members[tid];
  int lo = a.group_starts[0], hi = a.group_starts[n];
  for (int g = tid; g <= n; g += threads) starts[g] = a.group_starts[g];
  for (int g = tid; g < n; g += threads) {
    prefix[g] = a.prefix_lens[g];
    least[g] = lead[g] = INT_MAX;
    live[g] = 0;
  }
  for (int b = tid; b < B; b += threads) claim[b] = INT_MAX;
  if ((unsigned)member < (unsigned)B) len = a.tail.lens[member];
  auto member_of = [&](int i) { return i == tid ? member : a.members[i]; };
  auto length_of = [&](int i, int r) { return min(max(i == tid ? len : a.tail.lens[r], 0), most); };
  __syncthreads();
  bool bad = false;
  for (int g = tid; g < n; g += threads) bad |= starts[g] < 0 || starts[g + 1] < starts[g] || starts[g + 1] > N;
  const bool none = __syncthreads_or(bad) || n == 0;   // no groups to go by
  if (none) lo = hi = 0;
  for (int i = tid; i < hi; i += threads) {
    if (i < lo) continue;
    const int r = member_of(i);
    if ((unsigned)r < (unsigned)B) atomicMin(&claim[r], i);
    else bad = true;
  }
  __syncthreads();
  // the entry's request, -1: none, or named before
  auto request_of = [&](int i) {
    if (i < lo || i >= hi) return -1;
    const int r = member_of(i);
    return (unsigned)r < (unsigned)B && claim[r] == i ? r : -1;
  };
  for (int i = tid; i < hi; i += threads) {
    if (i < lo) continue;
    const int r = request_of(i);
    if (r < 0) { bad = true; continue; }
    const int g = entry_of(starts, n, i);
    atomicMin(&least[g], max(0, length_of(i, r) - T + 1));
    atomicMin(&lead[g], i);
    atomicAdd(&live[g], 1);
  }
  __syncthreads();

  // chunks and padded rows of the groups before each
  const int per = (n + threads - 1) / threads, g0 = min(tid * per, n), g1 = min(g0 + per, n);
  auto rows_of = [&](int g) { return live[g] > 1 && prefix[g] > 0 ? (starts[g + 1] - starts[g]) * R : 0; };
  int chunks = 0, padded = 0;
  if (!none)
    for (int g = g0; g < g1; ++g) {
      const int want = prefix[g];
      if (live[g] > 0) {
        bad |= want < 0 || want > least[g];
        prefix[g] = min(max(want, 0), least[g]);
        lead[g] = a.members[lead[g]];
      }
      chunks += (rows_of(g) + 127) >> 7;
      padded += (rows_of(g) + 7) & ~7;
    }
  const int lane = tid & 31, warp = tid >> 5;
  int ic = chunks, ip = padded;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(~0u, ic, d), y = __shfl_up_sync(~0u, ip, d);
    if (lane >= d) { ic += x; ip += y; }
  }
  if (lane == 31) { sums[0][warp] = ic; sums[1][warp] = ip; }
  __syncthreads();
  int before = ic - chunks, base_at = ip - padded, all = 0;
#pragma unroll 4
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) { before += sums[0][w]; base_at += sums[1][w]; }
    all += sums[0][w];
  }
  if (!none)
    for (int g = g0; g < g1; ++g) {
      first[g] = before;
      base[g] = base_at;
      before += (rows_of(g) + 127) >> 7;
      base_at += (rows_of(g) + 7) & ~7;
    }
  if (tid == 0) {
    first[n] = all;
    *out.n_chunks = all;
  }
  __syncthreads();
  for (int i = tid; i < N; i += threads) {
    const int r = request_of(i);
    out.members[i] = r;
    if (r < 0) continue;
    const int g = entry_of(starts, n, i);
    const bool shares = rows_of(g) > 0;
    out.begins[r] = shares ? prefix[g] : 0;
    out.places[r] = shares ? first[g] * 128 + (i - starts[g]) * R : -1;
  }
  for (int b = tid; b < B; b += threads)
    if (claim[b] == INT_MAX) {
      out.begins[b] = 0;
      out.places[b] = -1;
    }
  for (int c = tid; c < all; c += threads) {
    const int g = entry_of(first, n, c), row = (c - first[g]) * 128;
    int4* const at = reinterpret_cast<int4*>(out.chunks + c);
    at[0] = make_int4(prefix[g], lead[g], starts[g], row);
    at[1] = make_int4(min(128, rows_of(g) - row), base[g] + row, 0, 0);
  }
  if (bad) atomicOr(a.tail.err, (uint32_t)DEV_BAD_VALUE);
}

}  // namespace

cudaError_t launch_paged_shared_setup(const PagedSharedArgs& a, cudaStream_t st) {
  const size_t smem = ((size_t)7 * a.n_groups + 2 + a.tail.B) * sizeof(int);
  // (always to what the largest call needs, as for the tables)
  if (smem > 47 * 1024) {
    constexpr int most = (7 * kMaxPagedGroups + 2 + kMaxPagedBatch) * sizeof(int);
    const cudaError_t e =
        cudaFuncSetAttribute(paged_shared_setup_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  // (a thread a member, where that goes: few warps meet sooner)
  const int most = a.n_members > a.n_groups ? a.n_members : a.n_groups + 1;
  cfg.blockDim = dim3(most <= 128 ? 128 : most < kThreads ? (most + 31) & ~31 : kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, paged_shared_setup_kernel, a);
}

}  // namespace fa
