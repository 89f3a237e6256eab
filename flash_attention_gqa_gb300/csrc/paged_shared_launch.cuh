// Attention of requests that share prefixes: the grids behind the first kernel (paged_shared.cu).
//
//   x = q . k over the prefix's keys, once for all rows of a group (HEAD), and over the request's own
//   keys (TAIL); each leaves sums o, weights' sum l and base m, and the join adds them up:
//   o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
//
// HEAD is paged_shared_head.cuh, TAIL the decode kernels over keys from a request's first own one on; both
// leave partials of whole items, too.  The four grids are launched early, one behind the other: TAIL's CTAs start as
// HEAD's end.  HEAD waits for the tables before it lets TAIL start, TAIL ends only after HEAD has, and
// the join waits for TAIL.
#pragma once
#include "paged_decode.cuh"
#include "paged_decode_tc.cuh"
#include "paged_shared_head.cuh"

namespace fa {

// A thread per 4 dims of a row of item (b, k), a warp up to 8 rows (2^rows_shift) side by side; `per` such
// a CTA, times shares of the partials, summed in order behind it.  U partials of a thread in flight.
// Bound by three dependent loads (512 items of 8 rows, H = 128: 5 us of a call), two of them from L2; its
// first is done while the grid before it runs.
template <int H, bool TC, int U, int THREADS>
__global__ void __launch_bounds__(THREADS)
paged_shared_join_kernel(const __grid_constant__ PagedSharedArgs s, int per, int rows_shift) {
  __shared__ float4 sx[THREADS];
  __shared__ float2 sml[THREADS];
  const PagedDecodeArgs& a = s.tail;
  const int item = blockIdx.x, b = item / a.K, k = item - b * a.K, R = a.G * a.T, P = paged_partial_rows(R);
  const int shares = blockDim.x / per, share = threadIdx.x / per, at = threadIdx.x % per;
  const int i = blockIdx.y * per + at, tile = i / 32, side = 1 << rows_shift, groups = (R + side - 1) >> rows_shift;
  const int d = tile / groups * (32 >> rows_shift) + (i % 32 >> rows_shift);   // of 4
  const int r = d < H / 4 ? tile % groups * side + (i & (side - 1)) : R;
  // (written by the grids before, maybe while this one was already there: L2 loads.  The first kernel's
  // tables have been there since before HEAD let the next grid start.)
  const int place = r < R ? __ldcg(a.shared.places + b) : -1;
  int4 c = make_int4(0, 0, 0, 0);
  if (place >= 0) c = __ldcg(reinterpret_cast<const int4*>(a.shared.chunks + ((place + r) >> 7)) + 1);
  grid_before();
  const int4 tail = __ldcg(reinterpret_cast<const int4*>(a.splits) + item);
  // (an entry may hold anything where a wait ran out before it was written)
  const bool tail_split = tail.y >= 0 && tail.z >= tail.y && tail.z < s.tail_parts;
  const int n_tail = tail_split ? tail.z - tail.y + 1 : 1;
  const int64_t part = paged_partial_floats(R, H), part_head = paged_partial_floats(128, H);
  const float* const tail_at = tail_split ? a.partials + (int64_t)tail.y * 2 * part : a.shared.whole + item * part;
  int n_head = 0, P_head = 128, r_head = 0;
  const float* head_at = nullptr;
  bool head_split = false;
  if (place >= 0) {
    const int row = place + r, chunk = row >> 7;
    r_head = row & 127;
    const int4 head = __ldcg(reinterpret_cast<const int4*>(s.head_splits) + (int64_t)chunk * a.K + k);
    head_split = head.y >= 0 && head.z >= head.y && head.z < s.head_ctas;
    n_head = head_split ? head.z - head.y + 1 : 1;
    if (!head_split) P_head = (c.x + 7) & ~7;
    head_at = head_split ? s.head_partials + (int64_t)head.y * 2 * part_head
                         : s.head_whole + ((int64_t)c.y * a.K + (int64_t)k * P_head) * (H + 2);
  }
  JoinSum sum;
  if (r < R) {
    const int n = n_head + n_tail;
    for (int p0 = share; p0 < n; p0 += U * shares) {
      float4 y[U];
      float m[U], l[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = p0 + u * shares;
        m[u] = -INFINITY;
        if (p < n) {
          // partial 0 of a split item is in slot 1 of its CTA, the others in slot 0 of theirs
          const bool h = p < n_head;
          const int q = h ? p : p - n_head;
          const float* const src = h ? head_at + (head_split ? (q ? q * 2 : 1) * part_head : 0)
                                     : tail_at + (tail_split ? (q ? q * 2 : 1) * part : 0);
          const int rows = h ? P_head : P, row = h ? r_head : r;
          const int64_t at4 = h || TC ? ((int64_t)d * rows + row) * 4 : (int64_t)row * H + d * 4;
          y[u] = __ldcg(reinterpret_cast<const float4*>(src + at4));
          m[u] = __ldcg(src + (int64_t)rows * H + row);
          l[u] = __ldcg(src + (int64_t)rows * (H + 1) + row);
        }
      }
      sum.add(y, m, l, [&](int u) { return p0 + u * shares < n; });
    }
  }
  if (shares > 1) sum.meet(sx, sml, share, shares, at, per);
  if (share == 0 && r < R)
    put_result((char*)a.o + (int64_t)item * R * H * 2, a.lse + (int64_t)item * R, H, r, d * 4, sum.x,
               sum.M, sum.L, a.v_scale ? a.v_scale[k] : 1.0f);
}

// A grid that may start while the one before it in the stream still runs.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class C, class Args, void (*KERNEL)(const Args)>
cudaError_t launch_shared_part(const Args& a, int grid, cudaStream_t st) {
  static bool ready[64] = {};   // per device; setting it twice is harmless
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  return launch_early(KERNEL, dim3(grid), C::THREADS, C::SMEM, st, a);
}

template <int H, bool TC>
cudaError_t launch_shared_join(const PagedSharedArgs& s, cudaStream_t st) {
  const int R = s.tail.G * s.tail.T, items = s.tail.B * s.tail.K;
  int rows_shift = H == 64 ? 1 : 0;   // (a warp's dims are no more than a row's)
  while (rows_shift < 3 && (1 << rows_shift) < R) ++rows_shift;
  const int side = 1 << rows_shift, elements = (R + side - 1) / side * side * (H / 4);
  // Partials of a row: about CTAs / items, two more at most, of its own keys and of the prefix's, whose
  // items are at least the rows in chunks times the heads.  Several shares of them where they are many,
  // as far as all threads are there at once (156 items of 20 partials: 25 us with 16 shares, 1248 CTAs of 512).
  const int chunks = max(1, max(min(s.n_groups, s.n_members / 2), (int)((int64_t)s.n_members * R / 128)));
  const int partials = s.tail_parts / items + 2 + s.head_ctas / (chunks * s.tail.K) + 2;
  const int64_t room = (int64_t)s.head_ctas * 1024 / ((int64_t)items * elements);
  const int shares = partials <= 8 || room < 2 ? 1 : partials <= 16 || room < 4 ? 2 : room < 16 ? 4 : 16;
  int per = shares == 16 ? 32 : shares == 4 ? 64 : 256 / shares;
  while (per > 32 && per / 2 >= elements) per /= 2;
  const dim3 grid(items, (elements + per - 1) / per);
  switch (shares) {
    case 1: return launch_early(paged_shared_join_kernel<H, TC, 4, 256>, grid, per, 0, st, s, per, rows_shift);
    case 2:
    case 4: return launch_early(paged_shared_join_kernel<H, TC, 8, 256>, grid, shares * per, 0, st, s, per, rows_shift);
    default: return launch_early(paged_shared_join_kernel<H, TC, 8, 512>, grid, 16 * per, 0, st, s, per, rows_shift);
  }
}

template <int H, class C, void (*TAIL)(const PagedDecodeArgs)>
cudaError_t launch_shared_grids(const PagedSharedArgs& s, const PagedHeadArgs& head, cudaStream_t st,
                                cudaError_t (*launch_head)(const PagedHeadArgs&, int, cudaStream_t)) {
  cudaError_t e = launch_paged_shared_setup(s, st);
  if (e != cudaSuccess) return e;
  e = launch_head(head, s.head_ctas, st);
  if (e != cudaSuccess) return e;
  e = launch_shared_part<C, PagedDecodeArgs, TAIL>(s.tail, s.tail_ctas, st);
  if (e != cudaSuccess) return e;
  return launch_shared_join<H, C::TC>(s, st);
}

// Up to NT * 8 rows.
template <int H, bool E4M3, int NT>
cudaError_t launch_shared_rows(const PagedSharedArgs& s, const PagedHeadArgs& head, cudaStream_t st,
                               cudaError_t (*launch_head)(const PagedHeadArgs&, int, cudaStream_t)) {
  constexpr int tiles = H == 256 && NT == 4 ? 2 : NT;
  if constexpr (H * NT <= 256) {
    if (s.tail_parts > s.tail_ctas) {
      using C = DecodeCfg<H, E4M3, NT, 1, DECODE_TAIL, true>;
      static_assert(C::WARPS == 4, "as in paged_shared_plan");
      return launch_shared_grids<H, C, paged_decode_kernel<C>>(s, head, st, launch_head);
    }
  }
  using C = DecodeCfg<H, E4M3, tiles, NT / tiles, DECODE_TAIL>;
  return launch_shared_grids<H, C, paged_decode_kernel<C>>(s, head, st, launch_head);
}

// The kernel for a request's own keys goes by its rows, as in launch_decode_rows.
template <int H, bool E4M3>
cudaError_t launch_shared(const PagedSharedArgs& s, cudaStream_t st) {
  const int R = s.tail.G * s.tail.T;
  using Head = HeadCfg<H, E4M3>;
  PagedHeadArgs head;
  head.a = s.tail;
  head.a.splits = s.head_splits;
  head.a.partials = s.head_partials;
  head.a.shared.whole = s.head_whole;
  // (boxes of less than 8 rows: more of them than lanes, and not on the swizzle's boundaries)
  const int page = 1 << s.tail.lay.page_shift;
  head.rows = page < 8 ? 0 : page < Head::TN ? page : Head::TN;
  if (head.rows && !(make_cache_map(&head.k_map, s.tail.k_cache, s.tail.lay, s.tail.K, H, E4M3, head.rows) &&
                     make_cache_map(&head.v_map, s.tail.v_cache, s.tail.lay, s.tail.K, H, E4M3, head.rows)))
    head.rows = 0;
  auto* const launch_head = launch_shared_part<Head, PagedHeadArgs, paged_head_kernel<Head>>;
  if (R <= 8) return launch_shared_rows<H, E4M3, 1>(s, head, st, launch_head);
  if (R <= 16) return launch_shared_rows<H, E4M3, 2>(s, head, st, launch_head);
  if constexpr (H <= 128 || E4M3) {
    if (R <= 32) return launch_shared_rows<H, E4M3, 4>(s, head, st, launch_head);
  }
  using C = DecodeTcCfg<H, E4M3, DECODE_TAIL>;
  return launch_shared_grids<H, C, paged_decode_tc_kernel<C>>(s, head, st, launch_head);
}

}  // namespace fa
