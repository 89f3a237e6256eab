// Launches of the paged decode: the kernel for a call's rows, and the join.
#pragma once
#include "paged_decode.cuh"
#include "paged_decode_tc.cuh"

namespace fa {

// The most tiles that a request can have.
template <class C>
int64_t decode_most_tiles(const PagedDecodeArgs& a) {
  int64_t keys = (int64_t)a.max_pages << a.lay.page_shift;
  const int64_t seen = (int64_t)a.window + a.T - 1 + C::CK - 1;   // from a multiple of CK on
  if (a.window > 0 && seen < keys) keys = seen;
  return (keys + C::TK - 1) / C::TK;
}
// Requests of few tiles are not split, which saves the second launch: up to 4
// tiles (64 requests x 8 kv heads x 256 keys: 20.0 us split, 17.5 whole; 8 x 8:
// 8.2 and 7.8; 1 x 2 at H = 256: 8.1 and 8.9, and 2 us of the host), with items
// for every CTA up to 512 keys (64 x 8 x 512 keys: 29.7 split and 27.7 us whole; 40 rows
// at H = 256, 64 x 4 x 500 keys: 38.0 and 33.8).  With more keys it depends on how full the
// last round of CTAs is, which the rule does not look at: 64 rows, 40 x 4 x 900 28.5 split and
// 35.4 whole; at H = 64 40 x 8 x 700 17.6 and 19.4, but 64 x 8 x 1000 28.0 and 26.4.
template <class C>
int64_t decode_whole_tiles(int64_t items, int ctas) { return items >= ctas ? 512 / C::TK : 4; }

template <int H, bool TC>
cudaError_t launch_join(const PagedDecodeArgs& a, int grid, cudaStream_t st) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  // Partials of an item: about grid / items, two more at most.  Up to 4: all in
  // flight in one thread; up to 16: two shares of 8; more (one kv head of 131072
  // keys: 304): 16 shares, 8 in flight each.
  const int items = a.B * a.K, elements = (TC ? paged_partial_rows(a.G * a.T) : a.G * a.T) * (H / 4), partials = grid / items + 2;
  const int shares = partials <= 4 ? 1 : partials <= 16 ? 2 : 16;
  int per = shares == 16 ? 32 : 256 / shares;
  while (per > 32 && per / 2 >= elements) per /= 2;
  cfg.gridDim = dim3(a.by_item ? items : grid, (elements + per - 1) / per);
  cfg.blockDim = dim3(shares * per);
  switch (shares) {
    case 1: return cudaLaunchKernelEx(&cfg, paged_join_kernel<H, TC, 4, 256>, a, grid, per);
    case 2: return cudaLaunchKernelEx(&cfg, paged_join_kernel<H, TC, 8, 256>, a, grid, per);
    default: return cudaLaunchKernelEx(&cfg, paged_join_kernel<H, TC, 8, 512>, a, grid, per);
  }
}

// The first grid: KERNEL of a configuration C, then the join unless no item is split.
template <class C, void (*KERNEL)(const PagedDecodeArgs)>
cudaError_t launch_decode(PagedDecodeArgs a, int grid, cudaStream_t st) {
  static bool ready[64] = {};   // per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  a.unsplit = decode_most_tiles<C>(a) <= decode_whole_tiles<C>((int64_t)a.B * a.K, grid);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  e = cudaLaunchKernelEx(&cfg, KERNEL, a);   // this launch's status, whatever an earlier call has left
  if (e != cudaSuccess || a.unsplit) return e;
  return launch_join<C::H, C::TC>(a, grid, st);
}
template <class C>
cudaError_t launch_decode(const PagedDecodeArgs& a, int grid, cudaStream_t st) {
  return launch_decode<C, paged_decode_kernel<C>>(a, grid, st);
}

// Up to 8, 16 and 32 rows: mma.sync, warps on their own (teams of two for 8-bit
// caches' 32 rows at H = 256: registers).  More, and over 16 rows of bf16 at H =
// 256: tcgen05.  Both sides at 16 requests x 4 kv heads x 8192 keys, mma.sync and
// tcgen05: bf16 at H = 64 32 rows take 35 and 46 us; at H = 128 17 rows 53 and 56,
// 32 rows 56 and 56, 64 rows 102 and 57; at H = 256 16 rows 89 and 89, 32 rows 99
// and 93, 64 rows 202 and 97.  8-bit at H = 128 32 rows 44 and 50, 64 rows 79 and
// 52, 128 rows 139 and 54; at H = 256 32 rows 77 and 87.
template <int H, bool E4M3>
cudaError_t launch_decode_rows(const PagedDecodeArgs& a, int grid, cudaStream_t st) {
  const int R = a.G * a.T;
  if (R <= 8) return launch_decode<DecodeCfg<H, E4M3, 1, 1>>(a, grid, st);
  if (R <= 16) return launch_decode<DecodeCfg<H, E4M3, 2, 1>>(a, grid, st);
  if constexpr (H <= 128 || E4M3) {
    constexpr int NT = H == 256 ? 2 : 4;
    if (R <= 32) return launch_decode<DecodeCfg<H, E4M3, NT, 4 / NT>>(a, grid, st);
  }
  using Tc = DecodeTcCfg<H, E4M3>;
  return launch_decode<Tc, paged_decode_tc_kernel<Tc>>(a, grid, st);
}

}  // namespace fa
