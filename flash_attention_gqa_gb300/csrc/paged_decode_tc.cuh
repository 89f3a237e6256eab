// Paged decode for many query rows per kv head (up to 128): tcgen05 products on
// tiles of 128 rows x 128 keys (64 at H = 256).
//
// The split over CTAs, the partials and the join are those of paged_decode.cuh;
// only the work on a tile differs.  The query rows fill the 128-row operand here,
// and with mma.sync the products and the instructions around them bound the kernel.
// A tile of 128 keys takes 8 + 16 instructions of 64 cycles each at H = 128 (bf16:
// the weights enter as two terms), 1536 of the 3000 cycles in which an SM's share
// of the memory rate delivers its 64 KB.
//
// Measured, 16 requests x 4 kv heads x 8192 keys: bf16, H = 128, 64 rows 57 us
// (memory 40, and the fixed 10 of paged_decode.cuh): a tile every 2980 cycles, of
// which the softmax warps work 2100 and the products take 1800; 128 rows 60 us.  H =
// 256: 64 rows 97 us (memory 80).  H = 64: 46 us (memory 20): the softmax, 2300 cycles
// a tile, is the bound, as it does not shrink with H.  8-bit caches: 52 us (H = 128,
// 64 rows; memory 20), a tile every 2650 cycles, for the same reason.
//
// Roles (one CTA an SM):
//   warps 0-7   softmax and results: warps w and w + 4 share 32 rows (a thread
//               per row, a lane of tensor memory), each half of the keys of a
//               tile and half of the head dims of o
//   warps 8, 9  copies: each half of the keys of a tile, by cp.async (pages may end
//               anywhere, and keys past the request have to arrive as zeros); 8-bit
//               caches: warps 8 and 9 for K, 10 and 11 for V, which they also convert
//   last warp   products, tensor memory
// Tensor memory: S of tiles n and n + 1, o, and the weights, A operands of o += P V:
// one term over its S (in each half of it), the other of bf16's two beside o.
// Shared memory: the queries and rings of K and V tiles, in chunks of [rows x 128 B]
// with the 128-byte swizzle of the operand descriptors.
#pragma once
#include "paged_decode.cuh"

namespace fa {

template <int H_, bool E4M3_>
struct DecodeTcCfg {
  static constexpr int H = H_, HC = H / 64;
  static constexpr bool TC = true, E4M3 = E4M3_;
  static constexpr int TN = H == 256 ? 64 : 128;        // keys of a tile
  static constexpr int CK = TN, TEAMS = 1, TK = TN;
  // An item's fixed cost in tiles.  64 requests of 1 to 8192 keys, 64 rows: 46.4 us with 1,
  // 38.6 with 2, 39.6 with 3; 8-bit 42.7, 37.1 and 38.1; at H = 256, 32 rows, to 4096 keys
  // 38.4, 36.5 and 37.7; at H = 64, 40 rows 32.3, 30.9 and 33.1.
  static constexpr int ITEM_UNITS = 2;
  static constexpr int CW = E4M3 ? 4 : 2;               // copying warps, two for a tile
  static constexpr int WARPS = 9 + CW, THREADS = WARPS * 32;
  static constexpr int KPW = TN / 2;                    // keys of a tile a copying warp
  static constexpr int QCHUNK = 128 * 128;              // 128 query rows of 64 dims
  static constexpr int QBYTES = HC * QCHUNK;
  static constexpr int CHUNK = TN * 128;                // TN keys of 64 dims
  static constexpr int SLOT = HC * CHUNK;               // a tile of K or of V
  // bf16: 192, 192 and 160 KB.  8-bit: 96, 128 and 96 KB of f16 tiles, and 80, 64 and
  // 64 KB of bytes that wait for their conversion.
  static constexpr int STAGES = E4M3 ? (H == 64 ? 6 : H == 128 ? 4 : 3) : H == 64 ? 12 : H == 128 ? 6 : 5;
  static constexpr int KS = STAGES / 2, VS = STAGES - KS;   // for K and for V
  static constexpr int RAW = E4M3 ? TN * H : 0, RAW_STAGES = H == 64 ? 5 : 2;   // of K, and of V
  static constexpr int FLIGHT = RAW_STAGES - 1;         // 8-bit tiles in flight behind the newest
  static constexpr int RING = STAGES * SLOT;
  static constexpr int SMEM = QBYTES + RING + 2 * RAW_STAGES * RAW;
  // Tensor memory: S at 0 and TN, o at 256, the weights' second terms at REST_COL
  // and TN / 2 behind it.
  static constexpr uint32_t O_COL = 256, REST_COL = H == 256 ? 128 : 384;
  static constexpr int UPR = (E4M3 ? 1 : 2) * H / 16;   // 16-byte units of a key
};

// The bounded waits of this kernel's barriers, each by whole warps.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, const Abort& ab) {
  return __all_sync(~0u, mbar_wait(bar, parity, ab));
}

// One arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

// True in one lane of the warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// 32 lanes x 1 column.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return __uint_as_float(r);
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) paged_decode_tc_kernel(const __grid_constant__ PagedDecodeArgs a) {
  constexpr int H = C::H, HC = C::HC, S = C::STAGES, TN = C::TN;
  constexpr bool E4M3 = C::E4M3;
  constexpr uint32_t O_COL = C::O_COL, REST_COL = C::REST_COL;
  constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ DecodeShared<C> sh;
  __shared__ __align__(8) uint64_t bars[2 * S + 13];
  __shared__ uint32_t sh_tmem;
  __shared__ int sh_abort, sh_keep;    // sh_keep: o holds something before an item's first product
  __shared__ uint32_t sh_bad[2][8];    // keys of a tile (by its parity) whose value is not finite
  __shared__ float sh_top[2][2][128];  // [parity][half] largest scores of the rows; sums at the end

  const uint32_t q_u = smem_u32(sm), ring_u = q_u + C::QBYTES;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.G * a.T, P = paged_partial_rows(R);
  const DecodeShape<C> shape{a};
  const Abort ab{&sh_abort, a.wait_limit_ns, a.err};
  // Slots: K(n) takes turn n / KS of slot n % KS, V(n) the same behind them.
  auto slot_of = [](int n, int kv) { return kv ? C::KS + n % C::VS : n % C::KS; };
  auto turn_of = [](int n, int kv) { return kv ? n / C::VS : n / C::KS; };
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + S + s); };
  auto s_full = [&](int n) { return smem_u32(bars + 2 * S + (n & 1)); };
  auto p_full = [&](int n) { return smem_u32(bars + 2 * S + 2 + (n & 1)); };
  auto pv_done = [&](int n) { return smem_u32(bars + 2 * S + 4 + (n & 1)); };
  const uint32_t q_full = smem_u32(bars + 2 * S + 6), rows_met = smem_u32(bars + 2 * S + 7);
  const uint32_t teardown = smem_u32(bars + 2 * S + 8);
  auto pair_met = [&](int w) { return smem_u32(bars + 2 * S + 9 + (w & 3)); };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  DecodeWalk walk;
  if (!decode_units<C>(a, sh, walk)) return;
  if (tid == 0) {
    sh_abort = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 64);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 256);
      mbar_init(pv_done(i), 1);
    }
    mbar_init(q_full, 256);
    mbar_init(rows_met, 256);
    for (int w = 0; w < 4; ++w) mbar_init(pair_met(w), 64);
    mbar_init(teardown, 1);
    fence_barrier_init();
  }
  if (warp == C::WARPS - 1) {
    tmem_alloc(smem_u32(&sh_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh_tmem;

  if (warp == C::WARPS - 1) {
    // -------------------------------------------------------------- products
    // The warp runs this as one, and one lane issues: what an instruction names is the
    // same in all lanes, and said to be so (a shuffle).
    const bool lead = elect_one();
    constexpr auto idesc = E4M3 ? idesc_f16 : idesc_bf16;
    constexpr uint32_t id_s = idesc(128, TN, false, false);   // S = Q K^T
    constexpr uint32_t id_o = idesc(128, H, false, true);      // o += P V
    const uint64_t dq = sdesc_sw128(q_u, 16, 1024), dk = sdesc_sw128(ring_u, 16, 1024);
    const uint64_t dv = sdesc_sw128(ring_u, C::CHUNK, 1024);
    auto same = [](uint32_t x) { return __shfl_sync(~0u, x, 0); };
    const uint32_t tm = same(tmem);
    bool ok = true;
    int n = 0;   // tiles so far
    auto issue_pv = [&](int n, bool first) -> bool {
      if (!tc_wait(full(slot_of(n, 1)), turn_of(n, 1) & 1, ab) || !tc_wait(p_full(n), (n >> 1) & 1, ab)) return false;
      if (!E4M3) fence_proxy_async_smem();   // the copies were the generic proxy's
      tc_fence_after();
      const uint32_t odd = same(n & 1), slot = same(slot_of(n, 1)), p = tm + TN * odd, rest = tm + REST_COL + TN / 2 * odd;
      const uint64_t v = sdesc_add(dv, slot * C::SLOT);
      const uint32_t keep = same(!first || *reinterpret_cast<volatile int*>(&sh_keep));
      if (lead) {
#pragma unroll
        for (int kk = 0; kk < TN / 16; ++kk)
          mma_ts(tm + O_COL, p + kk / (TN / 32) * (TN / 2) + kk % (TN / 32) * 8, sdesc_add(v, kk * 2048), id_o,
                 kk > 0 ? 1u : keep);
#pragma unroll
        for (int kk = 0; !E4M3 && kk < TN / 16; ++kk)
          mma_ts(tm + O_COL, rest + kk * 8, sdesc_add(v, kk * 2048), id_o, 1u);
        mma_commit(empty(slot));
        mma_commit(pv_done(odd));
      }
      __syncwarp();
      return true;
    };
    for (int item = 0; ok; ++item) {
      ok = tc_wait(q_full, item & 1, ab);
      for (; ok && walk.tile < walk.end; ++walk.tile, ++n) {
        if (!(ok = tc_wait(full(slot_of(n, 0)), turn_of(n, 0) & 1, ab))) break;
        if (!E4M3) fence_proxy_async_smem();   // the copies were the generic proxy's
        tc_fence_after();
        const uint32_t odd = same(n & 1), slot = same(slot_of(n, 0)), s = tm + TN * odd;
        const uint64_t k = sdesc_add(dk, slot * C::SLOT);
        if (lead) {
#pragma unroll
          for (int c = 0; c < HC; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(s, sdesc_add(dq, c * C::QCHUNK + kk * 32), sdesc_add(k, c * C::CHUNK + kk * 32), id_s,
                     c > 0 || kk > 0 ? 1u : 0u);
          mma_commit(empty(slot));
          mma_commit(s_full(odd));
        }
        __syncwarp();
        // o += P V of the tile before, while this one's softmax runs
        if (walk.tile > walk.begun) ok = issue_pv(n - 1, walk.tile - 1 == walk.begun);
      }
      if (ok) ok = issue_pv(n - 1, walk.end - 1 == walk.begun);
      if (!shape.next_item(walk, sh.ends[1])) break;
    }
    // Until the products issued are over, whichever wait may have run out: the softmax warps'
    // wait for the last one may, after this warp has done all that it had to.  Tensor memory is
    // freed below and shared memory is given back.  They take microseconds.
    if (lead) mma_commit(teardown);
    mbar_wait_teardown(teardown, 0, max(a.wait_limit_ns, (uint64_t)1000000000));
    __syncwarp();
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- copies
    // bf16: two warps, each half of the keys of K(n) and then of V(n).  8-bit: two for K
    // and two for V, which then wait for slots of their own kind only.
    const int w = (warp - 8) & 1, kind = E4M3 ? (warp - 8) >> 1 : 0;
    constexpr int RPJ = 32 / C::UPR, NJ = C::KPW / RPJ, D = C::FLIGHT;   // rows a copy of the warp; copies
    const int64_t lane_src = (lane / C::UPR) * a.lay.token + (lane % C::UPR) * 16;
    const int64_t row_step = a.lay.token * RPJ;
    const int u = lane % C::UPR, lr = lane / C::UPR;   // unit and first row of this lane
    // 8-bit: this thread's units of a tile wait in places of its own, and are two units each as f16
    const int u16 = E4M3 ? 2 * u : u;
    const uint32_t lane_dst = (u16 >> 3) * C::CHUNK + (w * C::KPW + lr) * 128 + (((u16 & 7) ^ lr) << 4);
    const uint32_t raw_u = ring_u + C::RING + (kind * C::RAW_STAGES * 2 + w) * (C::RAW / 2) + lane * 16;
    auto row_place = [&](int slot, int j) {   // of copy j
      return ring_u + slot * C::SLOT + (lane_dst ^ (((j * RPJ) & 7) << 4)) + j * RPJ * 128;
    };
    auto place = [&](int n, int kv, int j) -> uint32_t {
      return E4M3 ? raw_u + n % C::RAW_STAGES * C::RAW + j * 512 : row_place(slot_of(n, kv), j);
    };
    auto free_slot = [&](int n, int kv) -> bool {
      return turn_of(n, kv) == 0 || tc_wait(empty(slot_of(n, kv)), (turn_of(n, kv) - 1) & 1, ab);
    };
    // 8-bit tile n has landed: to f16 (exact).
    auto hand_over = [&](int n) -> bool {
      if (!free_slot(n, kind)) return false;
      const int slot = slot_of(n, kind);
      const uint32_t turn = (u >> 2 & 1) << 4;   // four lanes write the odd unit first: other banks
#pragma unroll
      for (int j0 = 0; j0 < NJ; j0 += 8) {   // eight reads in flight
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = lds16(place(n, kind, j0 + j));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint4 y[2];
          e4m3x4_to_f16(x[j].x, y[0].x, y[0].y);
          e4m3x4_to_f16(x[j].y, y[0].z, y[0].w);
          e4m3x4_to_f16(x[j].z, y[1].x, y[1].y);
          e4m3x4_to_f16(x[j].w, y[1].z, y[1].w);
          const uint32_t dst = row_place(slot, j0 + j);
          sts16(dst ^ turn, turn ? y[1] : y[0]);
          sts16(dst ^ turn ^ 16, turn ? y[0] : y[1]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(full(slot));
      return true;
    };
    bool more = true, ok = true;
    int n = 0;
    // This lane's keys of the next tile: looked up a tile early.
    constexpr int NK = C::KPW < 32 ? 1 : C::KPW / 32;
    bool live[NK];
    int page[NK], in[NK], head = 0, next_lo = 0, next_hi = 0;   // rows [lo, hi) are keys
    auto look_up = [&]() {
      head = walk.k;
      const int row0 = walk.first + walk.tile * TN + w * C::KPW;
      next_lo = shape.low(walk.len) - row0;
      next_hi = walk.len - row0;
#pragma unroll
      for (int h = 0; h < NK; ++h) {
        const int row = h * 32 + lane, s = row0 + row;
        live[h] = more && row >= next_lo && row < next_hi;
        in[h] = s & ((1 << a.lay.page_shift) - 1);
        page[h] = -1;
        if (live[h])
          page[h] = __ldg(a.block_table + (int64_t)walk.b * a.max_pages + (s >> a.lay.page_shift));
      }
    };
    look_up();
    for (; more && ok; ++n) {
      int64_t off[NK];
      const int lo = next_lo, hi = next_hi;
      bool all = true;
#pragma unroll
      for (int h = 0; h < NK; ++h) {
        off[h] = -1;
        if (live[h]) {
          if (page[h] >= 0 && page[h] < a.lay.n_pages)
            off[h] = page[h] * a.lay.page + head * a.lay.head + in[h] * a.lay.token;
          else
            atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
        }
        all &= off[h] >= 0;
      }
      const bool steps = a.lay.page_shift >= 3 && __all_sync(~0u, all);
      if (++walk.tile == walk.end) more = shape.next_item(walk, sh.ends[1]);
      look_up();
#pragma unroll 1
      for (int kv = kind; kv < (E4M3 ? kind + 1 : 2); ++kv) {
        const char* const base = (const char*)(kv ? a.v_cache : a.k_cache);
        if (!E4M3 && !(ok = free_slot(n, kv))) break;
        if (steps) {   // 8 keys or more a page: one offset per 8 keys, and steps
#pragma unroll
          for (int k8 = 0; k8 < C::KPW; k8 += 8) {
            const char* src = base + __shfl_sync(~0u, off[k8 / 32], k8 % 32) + lane_src;
#pragma unroll
            for (int j = k8 / RPJ; j < (k8 + 8) / RPJ; ++j) {
              cp_async16(place(n, kv, j), src);
              src += row_step;
            }
          }
        } else if (a.lay.page_shift >= 3) {   // the same, where some rows are no keys
#pragma unroll 1
          for (int k8 = 0; k8 < C::KPW; k8 += 8) {
            const int last = min(k8 + 8, hi) - 1;   // the last key of the 8
            const int64_t at = __shfl_sync(~0u, k8 < 32 ? off[0] : off[NK - 1], last & 31);
            const bool some = last >= max(k8, lo) && at >= 0;
            const char* src = base + at - (last - k8) * a.lay.token + lane_src;
            const int j = k8 / RPJ;
#pragma unroll
            for (int i = 0; i < 8 / RPJ; ++i) {
              const int row = (j + i) * RPJ + lr;
              if (some && row >= lo && row < hi)
                cp_async16(place(n, kv, j + i), src + i * row_step);
              else
                cp_zeros16(place(n, kv, j + i), a.q);
            }
          }
        } else {
#pragma unroll 1
          for (int j = 0; j < NJ; ++j) {
            const int row = j * RPJ + lr;
            const int64_t at0 = __shfl_sync(~0u, off[0], row & 31), at1 = __shfl_sync(~0u, off[NK - 1], row & 31);
            const int64_t at = row < 32 ? at0 : at1;
            if (at >= 0)
              cp_async16(place(n, kv, j), base + at + u * 16);
            else
              cp_zeros16(place(n, kv, j), a.q);
          }
        }
        if constexpr (!E4M3) {
          cp_async_arrive(full(slot_of(n, kv)));
        } else {
          cp_async_commit();
          if (n >= D) {
            cp_async_wait<D>();
            if (!(ok = hand_over(n - D))) break;
          }
        }
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    for (int i = max(0, n - D); E4M3 && ok && i < n; ++i) ok = hand_over(i);
  } else {
    // --------------------------------------------------------------- softmax
    const int r = tid & 127, half = tid >> 7, t = r % a.T;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) * 32 << 16);
    constexpr int HD = H / 2;        // dims of o of a half
    const int d0 = half * HD;
    bool ok = true;
    int n = 0, meetings = 0, pairs = 0;
    // all eight warps have got here (a barrier with a limit)
    auto meet = [&]() -> bool {
      mbar_arrive(rows_met);
      return tc_wait(rows_met, meetings++ & 1, ab);
    };
    // For the search of V: this thread's key of a tile and its part of the key's
    // 16-byte units, and the place in its chunk of a unit (turned by the key,
    // against bank conflicts, within the part).
    constexpr int PARTS = 256 / TN, UPP = HC * 8 / PARTS;
    const int v_key = tid % TN, v_unit = tid / TN * UPP;
    auto v_place = [&](int u) { return (u >> 3) * C::CHUNK + (UPP == 4 ? (u & 4) | ((u + v_key) & 3) : (u + v_key) & 7) * 16; };
    // This thread's half of its query row; rows past the last are zeros.
    auto load_q = [&](const DecodeWalk& w) {
      const char* const src = (const char*)a.q + (((int64_t)w.b * a.K + w.k) * R + r) * (H * 2);
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        const int u = half * (HD / 8) + i;
        const uint32_t dst = q_u + (u >> 3) * C::QCHUNK + sw128_offset(r, u & 7);
        if (r < R)
          cp_async16(dst, src + u * 16);
        else
          cp_zeros16(dst, a.q);
      }
      cp_async_commit();
    };
    // What turns a product of the row into log2 units.  8-bit caches: queries as f16, their
    // rows scaled to [2^10, 2^11) as in paged_decode.cuh (`met`: a place of sh_top that is free).
    float sl2 = LOG2E, sl2_next = LOG2E;
    auto q_loaded = [&](const DecodeWalk& w, float (&met)[2][128]) -> bool {
      cp_async_wait<0>();
      if constexpr (E4M3) {
        auto place = [&](int i) { return q_u + ((half * (HD / 8) + i) >> 3) * C::QCHUNK + sw128_offset(r, (half * (HD / 8) + i) & 7); };
        float big = 0.0f;
#pragma unroll 4
        for (int i = 0; i < HD / 8; ++i) {
          const uint4 x = lds16(place(i));
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack_bf16x2(y[j]);
            big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        met[half][r] = big;
        mbar_arrive(pair_met(warp));
        if (!tc_wait(pair_met(warp), pairs++ & 1, ab)) return false;
        float up, down;
        e4m3_query_scale(fmaxf(big, met[half ^ 1][r]), up, down);
#pragma unroll 4
        for (int i = 0; i < HD / 8; ++i) {
          const uint4 x = lds16(place(i));
          uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack_bf16x2(y[j]);
            y[j] = pack_f16x2(f.x * up, f.y * up);
          }
          sts16(place(i), make_uint4(y[0], y[1], y[2], y[3]));
        }
        sl2_next = e4m3_score_scale(down, a.k_scale ? __ldg(a.k_scale + w.k) : 1.0f);
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
      return true;
    };
    load_q(walk);
    ok = q_loaded(walk, sh_top[1]);
    while (ok) {
      const int64_t item = (int64_t)walk.b * a.K + walk.k;
      sl2 = sl2_next;
      DecodeWalk then = walk;
      const bool go_on = shape.next_item(then, sh.ends[1]);
      const int hi = walk.len - a.T + t + 1, lo = a.window > 0 ? hi - a.window : 0;   // keys of this row
      const int full_hi = walk.len - a.T + 1;                              // keys of every row
      const int full_lo = a.window > 0 ? max(0, walk.len - a.window) : 0;
      float m = -INFINITY, l = 0.0f;   // base of the exponents (log2 units), sum of the weights
      for (; walk.tile < walk.end; ++walk.tile, ++n) {
        if (!(ok = tc_wait(s_full(n), (n >> 1) & 1, ab))) break;
        tc_fence_after();
        // With the last scores computed, the queries' place is free for the next item's.
        const bool last = walk.tile + 1 == walk.end;
        if (last && go_on) load_q(then);
        const uint32_t s_col = lanes + TN * (n & 1);
        const bool first = walk.tile == walk.begun;
        const int key0 = walk.first + walk.tile * TN;
        const bool masked = key0 < full_lo || key0 + TN > full_hi;
        // 32 scores at a time, twice: for the maximum and for the weights; TN / 2 a half
        auto load_s = [&](int i, uint32_t (&sv)[32]) {
          tmem_ld32(s_col + 32 * i, sv);
          tmem_wait_ld();
          if (masked) {
            const uint32_t keep = range_bits(lo - key0 - 32 * i, hi - key0 - 32 * i);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((keep >> j) & 1u)) sv[j] = __float_as_uint(-INFINITY);
          }
        };
        float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < TN / 64; ++i) {
          uint32_t sv[32];
          load_s(TN / 64 * half + i, sv);
#pragma unroll
          for (int j = 0; j < 32; ++j) pm[j & 3] = fmaxf(pm[j & 3], __uint_as_float(sv[j]));
        }
        float top = sl2 * fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
        sh_top[n & 1][half][r] = top;
        mbar_arrive(pair_met(warp));
        if (!(ok = tc_wait(pair_met(warp), pairs++ & 1, ab))) break;
        top = fmaxf(top, sh_top[n & 1][half ^ 1][r]);
        // The base is raised only where a score passes it by far, as in paged_decode.cuh.
        float alpha = 1.0f;
        if (top > m + kRaise<E4M3> || (first && top > m)) {
          const float to = top - kBelow<E4M3>;
          alpha = fast_exp2(m - to);   // 0 where there was none (top is no -inf here)
          m = to;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        if (!first && __any_sync(~0u, alpha != 1.0f)) {
          if (!(ok = tc_wait(pv_done(n - 1), ((n - 1) >> 1) & 1, ab))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = d0; c < d0 + HD; c += 32) {
            uint32_t ov[32];
            tmem_ld32(lanes + O_COL + c, ov);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(lanes + O_COL + c, ov);
          }
        }
        l *= alpha;

        if (first && tid == 0) sh_keep = 0;
        if (masked && a.T > 1) {
          // Values that are not finite, of keys that some row does not keep: 0 x inf
          // would reach it.  Their products are done here, row by row, and they are
          // zeros to the tensor cores.
          if (!(ok = tc_wait(full(slot_of(n, 1)), turn_of(n, 1) & 1, ab))) break;
          constexpr uint32_t INF = E4M3 ? 0x7c00u : 0x7f80u;
          uint8_t* const v_tile = sm + C::QBYTES + slot_of(n, 1) * C::SLOT;
          bool bad = false;
#pragma unroll
          for (int i = 0; i < UPP; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(v_tile + v_key * 128 + v_place(v_unit + i));
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              bad |= (y[j] & INF) == INF || (y[j] & INF << 16) == INF << 16;
          }
          const uint32_t ballot = __ballot_sync(~0u, bad);
          const uint32_t* const met = sh_bad[n & 1];
          if (lane == 0) sh_bad[n & 1][warp] = ballot;
          if (!(ok = meet())) break;
          // keys 32 i .. 32 i + 31
          auto bad_keys = [&](int i) {
            uint32_t x = 0;
#pragma unroll
            for (int p = 0; p < PARTS; ++p) x |= met[p * (TN / 32) + i];
            return x;
          };
          uint32_t any = 0;
#pragma unroll
          for (int i = 0; i < TN / 32; ++i) any |= bad_keys(i);
          if (any) {
            if (first) {
              uint32_t zero[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) zero[i] = 0;
#pragma unroll 1
              for (int c = d0; c < d0 + HD; c += 32) tmem_st32(lanes + O_COL + c, zero);
              if (tid == 0) sh_keep = 1;
            } else {
              if (!(ok = tc_wait(pv_done(n - 1), ((n - 1) >> 1) & 1, ab))) break;
              tc_fence_after();
            }
            tmem_wait_st();
#pragma unroll 1
            for (int key = 0; key < TN; ++key) {
              if (!((bad_keys(key >> 5) >> (key & 31)) & 1u)) continue;
              const bool kept = key0 + key >= lo && key0 + key < hi;
              const float x = tmem_ld1(s_col + key);
              tmem_wait_ld();
              const float p = fast_exp2(fmaf(x, sl2, -base));
#pragma unroll 1
              for (int c = d0; c < d0 + HD; c += 32) {
                uint32_t ov[32];
                tmem_ld32(lanes + O_COL + c, ov);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint4 x8 = *reinterpret_cast<const uint4*>(v_tile + (c >> 6) * C::CHUNK +
                                                                   sw128_offset(key, (c & 63) / 8 + i));
                  const uint32_t y[4] = {x8.x, x8.y, x8.z, x8.w};
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const float2 f = E4M3 ? unpack_f16x2(y[j]) : unpack_bf16x2(y[j]);
                    const int d = 8 * i + 2 * j;
                    if (kept) {
                      ov[d] = __float_as_uint(__uint_as_float(ov[d]) + p * f.x);
                      ov[d + 1] = __float_as_uint(__uint_as_float(ov[d + 1]) + p * f.y);
                    }
                  }
                }
                tmem_st32(lanes + O_COL + c, ov);
                tmem_wait_st();
              }
            }
            if (!(ok = meet())) break;   // all rows have read them
            if ((bad_keys(v_key >> 5) >> lane) & 1u) {
#pragma unroll
              for (int i = 0; i < UPP; ++i)
                *reinterpret_cast<uint4*>(v_tile + v_key * 128 + v_place(v_unit + i)) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
            fence_proxy_async_smem();
          }
        }

        // Weights as two bf16 terms (paged_decode.cuh): the cut over the scores that
        // this half has read, the rest beside o.  8-bit caches: one f16 term.
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < TN / 64; ++h) {
          const int i = TN / 64 * half + h;
          uint32_t sv[32], cut[16], rest[16];
          load_s(i, sv);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float x = fast_exp2(fmaf(__uint_as_float(sv[2 * j]), sl2, -base));
            const float y = fast_exp2(fmaf(__uint_as_float(sv[2 * j + 1]), sl2, -base));
            sum[j & 3] += x + y;
            if (E4M3) {
              cut[j] = pack_f16x2(x, y);
              continue;
            }
            const float hx = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
            const float hy = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
            cut[j] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
            rest[j] = pack_bf16x2(fmaf(x, 1 + 0x1p-20f, -hx), fmaf(y, 1 + 0x1p-20f, -hy));
          }
          tmem_st16(s_col + TN / 2 * half + 16 * h, cut);
          if (!E4M3) tmem_st16(lanes + REST_COL + TN / 2 * (n & 1) + 16 * i, rest);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(n));
        if (last && go_on && !(ok = q_loaded(then, sh_top[(n + 1) & 1]))) break;
      }
      // ---- end of the CTA's part of the item: o from tensor memory
      if (!ok || !(ok = tc_wait(pv_done(n - 1), ((n - 1) >> 1) & 1, ab))) break;
      tc_fence_after();
      // the last tile's place, which all have read; the next tile's may be written before it is read
      float(&sums)[2][128] = sh_top[(n - 1) & 1];
      sums[half][r] = l;
      mbar_arrive(pair_met(warp));
      if (!(ok = tc_wait(pair_met(warp), pairs++ & 1, ab))) break;
      l += sums[half ^ 1][r];
      const bool whole = walk.begun == 0 && walk.end == walk.tiles;
      const float f = l == 0.0f ? 0.0f : (a.v_scale ? __ldg(a.v_scale + walk.k) : 1.0f) / l;
      float* const mine =
          a.partials + ((int64_t)blockIdx.x * 2 + (walk.begun == 0 ? 1 : 0)) * paged_partial_floats(R, H);
#pragma unroll 1
      for (int c = d0; c < d0 + HD; c += 32) {
        uint32_t ov[32];
        tmem_ld32(lanes + O_COL + c, ov);
        tmem_wait_ld();
        if (r < R && whole) {
          uint4* const dst = reinterpret_cast<uint4*>((char*)a.o + ((item * R + r) * H + c) * 2);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              y[j] = pack_bf16x2(__uint_as_float(ov[8 * i + 2 * j]) * f, __uint_as_float(ov[8 * i + 2 * j + 1]) * f);
            dst[i] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else if (r < R) {
          // lanes side by side: rows as they are would take eight times the store cycles
          uint4* const dst = reinterpret_cast<uint4*>(mine) + (int64_t)(c / 4) * P + r;
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i * P] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
        }
        __syncwarp();
      }
      if (r < R && half == 0) {
        if (whole) {
          a.lse[item * R + r] = (m + log2f(l)) * LN2;   // -inf with no key
        } else {
          mine[(int64_t)P * H + r] = m;
          mine[(int64_t)P * (H + 1) + r] = l;
        }
      }
      if (whole && a.by_item && !a.unsplit && tid == 0) a.splits[item] = PagedDecodeSplit{(int)item, -1, 0, 0};
      tc_fence_before();
      if (!go_on) break;
      walk = then;
    }
    if (!ok) {   // a wait has run out: until what is in flight has landed
      cp_async_wait<0>();
      tmem_wait_st();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::WARPS - 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
