// Attention over shared prefixes, HEAD: chunks of up to 128 rows of a group against the group's prefix,
// tcgen05 products on tiles of 128 rows x 128 keys (64 at H = 256).
//
// The split over CTAs and the partials are those of the paged decode (paged_decode.cuh,
// paged_decode_tc.cuh), with chunks in the requests' place.  What differs is what bounds it: with many
// chunks the prefix comes from L2 and the work on a tile is all there is.  A tile takes 1536 cycles of
// products at H = 128 in bf16 (the weights enter as two terms), and a softmax of some 2800 cycles of
// latencies, in which one warp's row needs its scores, their maximum, the exponentials and their way
// back to tensor memory.  So two tiles are in work at once: each four softmax warps (a thread per row)
// take every other tile, whole, and hand on the base of the exponents as soon as their tile's maximum
// is known; and scores are computed three tiles ahead, so that none waits for a product.
// A tile takes 1850 cycles then (2400 of 8-bit caches, by their way to f16; 1950 of 64 keys at H = 256, 1792
// of them products).  512 rows x 8 heads x 8192 keys in bf16 28 us, 13 of them tiles; 1024 rows x 2 heads x 32768 keys
// at H = 256 71 us, 55 of them tiles; the rest is the way to a CTA's first product and the ends of its parts.
//
// Roles (one CTA an SM):
//   warps 0-3, 4-7  softmax of even and of odd tiles; results, half of the head dims each
//   warps 8 ..      copies, of K and of V (head_copies)
//   last two warps  products, S and o; tensor memory
// Tensor memory: three S buffers and o.  The weights take their scores' place, 32 keys at a time: their
// first terms in 16 columns, the others of bf16's two in the next 16.
#pragma once
#include "paged_decode_tc.cuh"

namespace fa {

template <int H_, bool E4M3_>
struct HeadCfg : DecodeTcCfg<H_, E4M3_, DECODE_HEAD> {
  using Base = DecodeTcCfg<H_, E4M3_, DECODE_HEAD>;
  static constexpr int H = H_, TN = Base::TN, STAGES = Base::STAGES;
  static constexpr int NS = 3;   // S buffers
  static constexpr uint32_t O_COL = H_ == 256 ? 256 : 384;
  static_assert(NS * TN <= (int)O_COL && O_COL + H_ <= 512, "");
  // Copying warps: one each for K and V; 8-bit caches: two more each, that make f16 of the bytes.
  static constexpr int CONVERT = E4M3_ ? 4 : 0, KPW = TN / 2;   // keys of a tile a converting warp
  static constexpr int WARPS = 12 + CONVERT, THREADS = WARPS * 32;
  // Slots: scores are computed ahead of the weights, so K needs more of them.
  static constexpr int VS = STAGES / 2, KS = STAGES - VS;
  __device__ static __forceinline__ int slot_of(int n, int kv) { return kv ? KS + n % VS : n % KS; }
  __device__ static __forceinline__ int turn_of(int n, int kv) { return kv ? n / VS : n / KS; }
  static constexpr int RAW_STAGES = Base::RAW_STAGES, RAW_BARS = E4M3_ ? 4 * RAW_STAGES : 0;   // full, empty, of K and V
};

// a * b + c and a + b of two floats at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A copying warp's work: every tile of K or of V (`kind`), into its place as that becomes free.  By TMA,
// a lane a box of one page's rows, in one instruction: cp.async by 16 bytes a lane keeps the load and store
// pipe busy for 2600 cycles a tile, more than all the rest of it takes.  Rows past the prefix have to be
// zeros, which a box can give for whole pages only (out of the map's range): a tile that ends inside a page
// goes by cp.async, as does everything where there is no map.  `place(n, ..)` waits until tile n's is free
// and gives its address and barrier, `landed(n)` until the tiles before n that may be on their way have come.
template <class C, class Place, class Landed>
__device__ __forceinline__ void head_copies(const PagedHeadArgs& s, const DecodeShape<C>& shape, DecodeWalk walk,
                                            const DecodeEnd& last, int kind, const Abort& ab, Place place,
                                            Landed landed) {
  constexpr int TN = C::TN, UPR = C::UPR;
  constexpr bool E4M3 = C::E4M3;
  constexpr int CHUNKS = E4M3 ? 1 : C::HC;   // boxes of a page's rows
  const PagedDecodeArgs& a = s.a;
  const int lane = threadIdx.x & 31;
  const int shift = a.lay.page_shift, rows = s.rows;
  const int boxes = rows ? TN / rows * CHUNKS : 0;   // (<= 32: pages of 8 tokens at least)
  const int box_row = rows ? lane / CHUNKS * rows : 0, box_chunk = lane % CHUNKS;
  // A row past the prefix: -1.
  auto page_of = [&](int key, int len, int table_row) -> int {
    return key < len ? __ldg(a.block_table + (int64_t)table_row * a.max_pages + (key >> shift)) : -1;
  };
  auto known = [&](int page) { return page >= 0 && page < a.lay.n_pages; };
  bool more = true, ok = true;
  int n = 0;
  // the page of this lane's box in the next tile, looked up a tile early
  int page = page_of(walk.tile * TN + box_row, walk.len, shape.table_row(walk));
  for (; more && ok; ++n) {
    const int row0 = walk.tile * TN, len = walk.len, head = walk.k, table_row = shape.table_row(walk);
    const int left = len - row0, mine = page;
    if (++walk.tile == walk.end) more = shape.next_item(walk, last);
    if (more) page = page_of(walk.tile * TN + box_row, walk.len, shape.table_row(walk));
    uint32_t dst, bar;
    if (!(ok = place(n, dst, bar))) break;
    if (rows && (left >= TN || (left & ((1 << shift) - 1)) == 0)) {
      if (lane == 0) mbar_arrive_expect_tx(bar, TN * CHUNKS * (E4M3 ? C::H : 128));
      __syncwarp();
      if (lane < boxes) {
        const bool key = box_row < left;
        if (key && !known(mine)) atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
        tma_load_4d(dst + (E4M3 ? box_row * C::H : box_chunk * C::CHUNK + box_row * 128),
                    kind ? &s.v_map : &s.k_map, bar, E4M3 ? 0 : box_chunk * 64,
                    (row0 + box_row) & ((1 << shift) - 1), head, key && known(mine) ? mine : a.lay.n_pages);
      }
      if (lane != 0) mbar_arrive(bar);
    } else {
      const char* const base = (const char*)(kind ? a.v_cache : a.k_cache);
#pragma unroll 1
      for (int r0 = 0; r0 < TN; r0 += 32) {   // a lane a row's page, then all lanes 16-byte units
        const int key = row0 + r0 + lane, at_page = page_of(key, len, table_row);
        int64_t off = -1;
        if (known(at_page))
          off = at_page * a.lay.page + head * a.lay.head + (key & ((1 << shift) - 1)) * a.lay.token;
        else if (key < len)
          atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
#pragma unroll 1
        for (int i = lane; i < 32 * UPR; i += 32) {
          const int row = i / UPR, u = i % UPR;
          const int64_t at = __shfl_sync(~0u, off, row);
          const uint32_t to =
              dst + (E4M3 ? (r0 + row) * C::H + u * 16 : (u >> 3) * C::CHUNK + sw128_offset(r0 + row, u & 7));
          if (at >= 0)
            cp_async16(to, base + at + u * 16);
          else
            cp_zeros16(to, a.q);
        }
      }
      cp_async_arrive(bar);
    }
  }
  // What is in flight lands before the CTA ends, whichever wait may run out, here or elsewhere, now or later.
  cp_async_wait<0>();
  landed(n);
}

// A converting warp's work, 8-bit caches: rows [w * KPW, (w + 1) * KPW) of every tile of K or of V from bytes
// to f16 (exact), from raw_u into the slots.
template <class C, class Full, class Empty, class RawFull, class RawEmpty>
__device__ __forceinline__ void head_converts(const DecodeShape<C>& shape, DecodeWalk walk, const DecodeEnd& last,
                                              uint32_t ring_u, uint32_t raw_u, int w, int kind, const Abort& ab,
                                              Full full, Empty empty, RawFull raw_full, RawEmpty raw_empty) {
  constexpr int UPR = C::UPR, RPJ = 32 / UPR, NJ = C::KPW / RPJ, RS = C::RAW_STAGES;
  const int lane = threadIdx.x & 31, u = lane % UPR, lr = lane / UPR;
  const uint32_t odd = (u >> 2 & 1) << 4;   // four lanes write the odd unit first: other banks
  bool more = true;
  for (int n = 0; more; ++n) {
    if (++walk.tile == walk.end) more = shape.next_item(walk, last);
    const int slot = C::slot_of(n, kind);
    if (!tc_wait(raw_full(n, kind), n / RS & 1, ab)) return;
    if (C::turn_of(n, kind) != 0 && !tc_wait(empty(slot), (C::turn_of(n, kind) - 1) & 1, ab)) return;
    const uint32_t from = raw_u + (kind * RS + n % RS) * C::RAW + w * (C::RAW / 2) + lane * 16;
    const uint32_t to = ring_u + slot * C::SLOT + (2 * u >> 3) * C::CHUNK + (w * C::KPW + lr) * 128;
#pragma unroll 1
    for (int j0 = 0; j0 < NJ; j0 += 8) {   // eight reads in flight
      uint4 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = lds16(from + (j0 + j) * 512);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint4 y[2];
        e4m3x4_to_f16(x[j].x, y[0].x, y[0].y);
        e4m3x4_to_f16(x[j].y, y[0].z, y[0].w);
        e4m3x4_to_f16(x[j].z, y[1].x, y[1].y);
        e4m3x4_to_f16(x[j].w, y[1].z, y[1].w);
        const int row = (j0 + j) * RPJ;
        const uint32_t dst = to + row * 128 + (((2 * u & 7) ^ ((lr + row) & 7)) << 4);
        sts16(dst ^ odd, odd ? y[1] : y[0]);
        sts16(dst ^ odd ^ 16, odd ? y[0] : y[1]);
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(full(slot));
    mbar_arrive(raw_empty(n, kind));
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) paged_head_kernel(const __grid_constant__ PagedHeadArgs args) {
  const PagedDecodeArgs& a = args.a;
  constexpr int H = C::H, HC = C::HC, S = C::STAGES, TN = C::TN, NS = C::NS;
  constexpr bool E4M3 = C::E4M3;
  constexpr uint32_t O_COL = C::O_COL;
  constexpr float LOG2E = 1.4426950408889634f;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ DecodeShared<C> sh;
  __shared__ __align__(8) uint64_t bars[2 * S + 3 * NS + 15 + C::RAW_BARS];
  __shared__ uint32_t sh_tmem;
  __shared__ int sh_abort;
  __shared__ float sh_base[128];        // base of the rows' exponents after the newest tile
  __shared__ float sh_sums[2][128];     // [item's parity] sums of the weights of odd tiles
  __shared__ float sh_big[2][128];      // largest values of the halves of a query row

  const uint32_t q_u = smem_u32(sm), ring_u = q_u + C::QBYTES;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int GT = a.G * a.T;
  const DecodeShape<C> shape{a};
  const Abort ab{&sh_abort, a.wait_limit_ns, a.err};
  // A barrier of NS comes round every NS tiles; a tile's scores are computed only after the products of the
  // tile NS before it, so nobody who has seen them can take that turn for this one.
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + S + s); };
  auto s_full = [&](int n) { return smem_u32(bars + 2 * S + n % NS); };
  auto p_full = [&](int n) { return smem_u32(bars + 2 * S + NS + n % NS); };
  auto pv_done = [&](int n) { return smem_u32(bars + 2 * S + 2 * NS + n % NS); };
  auto turn = [](int n) { return (uint32_t)(n / NS & 1); };
  const uint32_t q_full = smem_u32(bars + 2 * S + 3 * NS), o_free = q_full + 8, teardown = q_full + 16;
  auto base_known = [&](int odd, int w) { return smem_u32(bars + 2 * S + 3 * NS + 3 + odd * 4 + (w & 3)); };
  auto pair_met = [&](int w) { return smem_u32(bars + 2 * S + 3 * NS + 11 + (w & 3)); };

  auto raw_full = [&](int n, int kind) { return smem_u32(bars + 2 * S + 3 * NS + 15 + kind * C::RAW_STAGES + n % C::RAW_STAGES); };
  auto raw_empty = [&](int n, int kind) { return raw_full(n, kind) + 16 * C::RAW_STAGES; };

  // The tables are written; what comes after this grid reads them, too, and starts knowing that.
  grid_before();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  DecodeWalk walk;
  if (!decode_units<C>(a, sh, walk)) return;
  if (tid == 0) {
    sh_abort = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), E4M3 ? 64 : 32);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 128);
      mbar_init(pv_done(i), 1);
    }
    mbar_init(q_full, 256);
    mbar_init(o_free, 256);
    mbar_init(teardown, 2);
    for (int i = 0; i < C::RAW_BARS / 4; ++i)
      for (int kind = 0; kind < 2; ++kind) {
        mbar_init(raw_full(i, kind), 32);
        mbar_init(raw_empty(i, kind), 64);
      }
    for (int w = 0; w < 4; ++w) {
      mbar_init(base_known(0, w), 32);
      mbar_init(base_known(1, w), 32);
      mbar_init(pair_met(w), 64);
    }
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

  if (warp >= C::WARPS - 2) {
    // -------------------------------------------------------------- products
    // A warp issues S = Q K^T, the other o += P V: with one for both, what it waits for and says around
    // each of them (1000 cycles a tile) is time in which the tensor cores run dry.  Either runs as one, and
    // one lane issues (paged_decode_tc.cuh).
    const bool lead = elect_one();
    constexpr auto idesc = E4M3 ? idesc_f16 : idesc_bf16;
    constexpr uint32_t id_s = idesc(128, TN, false, false);   // S = Q K^T
    constexpr uint32_t id_o = idesc(128, H, false, true);      // o += P V
    auto same = [](uint32_t x) { return __shfl_sync(~0u, x, 0); };
    const uint32_t tm = same(tmem);
    bool ok = true;
    int n = 0;
    if (warp == C::WARPS - 2) {
      const uint64_t dq = sdesc_sw128(q_u, 16, 1024), dk = sdesc_sw128(ring_u, 16, 1024);
      for (int item = 0; ok; ++item) {
        ok = tc_wait(q_full, item & 1, ab);
        for (; ok && walk.tile < walk.end; ++walk.tile, ++n) {
          // the weights that were here have been taken
          if (!(ok = tc_wait(full(C::slot_of(n, 0)), C::turn_of(n, 0) & 1, ab) &&
                     (n < NS || tc_wait(pv_done(n - NS), turn(n - NS), ab))))
            break;
          if (!E4M3) fence_proxy_async_smem();   // the copies were the generic proxy's
          tc_fence_after();
          const uint32_t slot = same(C::slot_of(n, 0)), s = tm + TN * same(n % NS), bar = same(s_full(n));
          const uint64_t k = sdesc_add(dk, slot * C::SLOT);
          if (lead) {
#pragma unroll
            for (int c = 0; c < HC; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ss(s, sdesc_add(dq, c * C::QCHUNK + kk * 32), sdesc_add(k, c * C::CHUNK + kk * 32), id_s,
                       c > 0 || kk > 0 ? 1u : 0u);
            mma_commit(empty(slot));
            mma_commit(bar);
          }
          __syncwarp();
        }
        if (!shape.next_item(walk, sh.ends[1])) break;
      }
    } else {
      const uint64_t dv = sdesc_sw128(ring_u, C::CHUNK, 1024);
      for (int item = 0; ok; ++item) {
        // o of the item before has been read
        if (item > 0) ok = tc_wait(o_free, (item - 1) & 1, ab);
        for (; ok && walk.tile < walk.end; ++walk.tile, ++n) {
          if (!(ok = tc_wait(full(C::slot_of(n, 1)), C::turn_of(n, 1) & 1, ab) && tc_wait(p_full(n), turn(n), ab)))
            break;
          if (!E4M3) fence_proxy_async_smem();
          tc_fence_after();
          const uint32_t slot = same(C::slot_of(n, 1)), p = tm + TN * same(n % NS), bar = same(pv_done(n));
          const uint64_t v = sdesc_add(dv, slot * C::SLOT);
          const uint32_t add = same(walk.tile > walk.begun ? 1u : 0u);
          if (lead) {
#pragma unroll
            for (int kk = 0; kk < TN / 16; ++kk)
              mma_ts(tm + O_COL, p + kk / 2 * 32 + kk % 2 * 8, sdesc_add(v, kk * 2048), id_o, kk > 0 ? 1u : add);
#pragma unroll
            for (int kk = 0; !E4M3 && kk < TN / 16; ++kk)
              mma_ts(tm + O_COL, p + kk / 2 * 32 + 16 + kk % 2 * 8, sdesc_add(v, kk * 2048), id_o, 1u);
            mma_commit(empty(slot));
            mma_commit(bar);
          }
          __syncwarp();
        }
        if (!shape.next_item(walk, sh.ends[1])) break;
      }
    }
    // Until the products issued are over (paged_decode_tc.cuh).
    if (lead) mma_commit(teardown);
    mbar_wait_teardown(teardown, 0, max(a.wait_limit_ns, (uint64_t)1000000000));
    __syncwarp();
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- copies
    constexpr int RS = C::RAW_STAGES;
    const uint64_t limit = max(a.wait_limit_ns, (uint64_t)1000000000);
    if constexpr (E4M3) {
      if (warp < 8 + C::CONVERT) {
        head_converts<C>(shape, walk, sh.ends[1], ring_u, ring_u + C::RING, (warp - 8) & 1, (warp - 8) >> 1, ab, full,
                         empty, raw_full, raw_empty);
      } else {
        const int mine = warp - 8 - C::CONVERT;
        head_copies<C>(
            args, shape, walk, sh.ends[1], mine, ab,
            [&](int n, uint32_t& dst, uint32_t& bar) {
              dst = ring_u + C::RING + (mine * RS + n % RS) * C::RAW;
              bar = raw_full(n, mine);
              return n < RS || tc_wait(raw_empty(n, mine), (n / RS - 1) & 1, ab);
            },
            [&](int n) {
              for (int i = max(0, n - RS); i < n; ++i) mbar_wait_teardown(raw_full(i, mine), i / RS & 1, limit);
            });
      }
    } else {
      const int mine = warp - 8;
      head_copies<C>(
          args, shape, walk, sh.ends[1], mine, ab,
          [&](int n, uint32_t& dst, uint32_t& bar) {
            const int slot = C::slot_of(n, mine), turns = C::turn_of(n, mine);
            dst = ring_u + slot * C::SLOT;
            bar = full(slot);
            return turns == 0 || tc_wait(empty(slot), (turns - 1) & 1, ab);
          },
          [&](int n) {
            for (int i = max(0, n - (mine ? C::VS : C::KS)); i < n; ++i)
              mbar_wait_teardown(full(C::slot_of(i, mine)), C::turn_of(i, mine) & 1, limit);
          });
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int r = tid & 127, odd = tid >> 7;   // row; which tiles, and which half of queries and results
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) * 32 << 16);
    constexpr int HD = H / 2;
    const int d0 = odd * HD;
    bool ok = true;
    int n = 0, pairs = 0, rows_next = 0;
    // This thread's half of its query row; rows without a member are zeros.
    auto load_q = [&](const DecodeWalk& w) {
      const int4 c = __ldcg(reinterpret_cast<const int4*>(a.shared.chunks + w.b));
      rows_next = __ldcg(&a.shared.chunks[w.b].rows);
      const int at = c.w + r, m = at / GT;
      const int member = r < rows_next ? __ldcg(a.shared.members + c.z + m) : -1;
      const char* const src = (const char*)a.q + (((int64_t)max(member, 0) * a.K + w.k) * GT + at - m * GT) * (H * 2);
#pragma unroll 4
      for (int i = 0; i < HD / 8; ++i) {
        const int u = odd * (HD / 8) + i;
        const uint32_t dst = q_u + (u >> 3) * C::QCHUNK + sw128_offset(r, u & 7);
        if (member >= 0)
          cp_async16(dst, src + u * 16);
        else
          cp_zeros16(dst, a.q);
      }
      cp_async_commit();
    };
    // What turns a product of the row into log2 units.  8-bit caches: queries as f16, their
    // rows scaled to [2^10, 2^11) as in paged_decode.cuh.
    float sl2 = LOG2E, sl2_next = LOG2E;
    auto q_loaded = [&](const DecodeWalk& w) -> bool {
      cp_async_wait<0>();
      if constexpr (E4M3) {
        auto place = [&](int i) { return q_u + ((odd * (HD / 8) + i) >> 3) * C::QCHUNK + sw128_offset(r, (odd * (HD / 8) + i) & 7); };
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
        sh_big[odd][r] = big;
        mbar_arrive(pair_met(warp));
        if (!tc_wait(pair_met(warp), pairs++ & 1, ab)) return false;
        float up, down;
        e4m3_query_scale(fmaxf(big, sh_big[odd ^ 1][r]), up, down);
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
    ok = q_loaded(walk);
    for (int item = 0; ok; ++item) {
      sl2 = sl2_next;
      const int rows = rows_next;
      const bool idle = (warp & 3) * 32 >= rows;
      DecodeWalk then = walk;
      const bool go_on = shape.next_item(then, sh.ends[1]);
      float m = -INFINITY, l = 0.0f;   // base of the exponents (log2 units), sum of these tiles' weights
      for (; walk.tile < walk.end; ++walk.tile, ++n) {
        if ((n & 1) != odd) continue;
        if (!(ok = tc_wait(s_full(n), turn(n), ab))) break;
        tc_fence_after();
        // With the last scores computed, the queries' place is free for the next item's.
        const bool first = walk.tile == walk.begun, last = walk.tile + 1 == walk.end;
        if (last && go_on) load_q(then);
        // (Rows of a warp past the chunk's: whatever their weights are, nobody reads their results.)
        if (idle) {
          if (n > 0 && !(ok = tc_wait(base_known(odd ^ 1, warp), (n - 1) >> 1 & 1, ab))) break;
          mbar_arrive(base_known(odd, warp));
          mbar_arrive(p_full(n));
          if (last && go_on && !(ok = q_loaded(then))) break;
          continue;
        }
        const uint32_t s_col = lanes + TN * (n % NS);
        const int left = walk.len - walk.first - walk.tile * TN;   // keys from the tile's first on
        const bool masked = left < TN;
        // 32 scores at a time, twice: for the maximum and for the weights
        auto mask = [&](int i, uint32_t (&sv)[32]) {
          if (masked) {
            const uint32_t keep = range_bits(0, left - 32 * i);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((keep >> j) & 1u)) sv[j] = __float_as_uint(-INFINITY);
          }
        };
        float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int i = 0; i < TN / 32; i += 2) {   // (not unrolled: the first pass over the code costs its reading)
          uint32_t lo[32], hi[32];
          tmem_ld32(s_col + 32 * i, lo);
          tmem_ld32(s_col + 32 * i + 32, hi);
          tmem_wait_ld();
          mask(i, lo);
          mask(i + 1, hi);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            pm[j & 3] = fmaxf(pm[j & 3], fmaxf(__uint_as_float(lo[j]), __uint_as_float(hi[j])));
        }
        const float top = sl2 * fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
        // The base that the tile before has left, by the other warps; raised only where a score passes
        // it by far (paged_decode.cuh), and handed on.
        if (n > 0 && !(ok = tc_wait(base_known(odd ^ 1, warp), (n - 1) >> 1 & 1, ab))) break;
        const float before = first ? -INFINITY : sh_base[r];
        float to = before, alpha = 1.0f;
        if (top > before + kRaise<E4M3> || (first && top > before)) {
          to = top - kBelow<E4M3>;
          alpha = fast_exp2(before - to);
        }
        sh_base[r] = to;
        mbar_arrive(base_known(odd, warp));
        const float base = to == -INFINITY ? 0.0f : to;
        l *= fast_exp2(m - base);
        m = to;
        if (!first && __any_sync(~0u, alpha != 1.0f)) {
          if (!(ok = tc_wait(pv_done(n - 1), turn(n - 1), ab))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < H; c += 32) {
            uint32_t ov[32];
            tmem_ld32(lanes + O_COL + c, ov);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(lanes + O_COL + c, ov);
          }
        }
        // Weights as two bf16 terms, cut and rest (paged_decode.cuh); 8-bit caches: one f16 term.
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const float2 scale = make_float2(sl2, sl2), shift = make_float2(-base, -base);
        const float2 more = make_float2(1 + 0x1p-20f, 1 + 0x1p-20f);
#pragma unroll 1
        for (int i = 0; i < TN / 32; ++i) {
          uint32_t sv[32], cut[16], rest[16];
          tmem_ld32(s_col + 32 * i, sv);
          tmem_wait_ld();
          mask(i, sv);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 x = fma2(make_float2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), scale, shift);
            x = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            sum[j & 1] = add2(sum[j & 1], x);
            if (E4M3) {
              cut[j] = pack_f16x2(x.x, x.y);
              continue;
            }
            const float2 less = make_float2(-__uint_as_float(__float_as_uint(x.x) & 0xffff0000u),
                                            -__uint_as_float(__float_as_uint(x.y) & 0xffff0000u));
            cut[j] = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
            const float2 y = fma2(x, more, less);
            rest[j] = pack_bf16x2(y.x, y.y);
          }
          tmem_st16(s_col + 32 * i, cut);
          if (!E4M3) tmem_st16(s_col + 32 * i + 16, rest);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(n));
        if (last && go_on && !(ok = q_loaded(then))) break;
      }
      if (!ok) break;
      // ---- end of the CTA's part of the item: o from tensor memory
      if (((n - 1) & 1) != odd) {   // the last tile was the other warps'
        if (!(ok = tc_wait(s_full(n - 1), turn(n - 1), ab))) break;
        if (go_on) {
          load_q(then);
          if (!(ok = q_loaded(then))) break;
        }
        if (!(ok = tc_wait(base_known(odd ^ 1, warp), (n - 1) >> 1 & 1, ab))) break;
        const float to = sh_base[r];
        l *= fast_exp2(m - (to == -INFINITY ? 0.0f : to));
        m = to;
      }
      if (!(ok = tc_wait(pv_done(n - 1), turn(n - 1), ab))) break;
      tc_fence_after();
      if (odd) sh_sums[item & 1][r] = l;
      mbar_arrive(pair_met(warp));
      if (!(ok = tc_wait(pair_met(warp), pairs++ & 1, ab))) break;
      const bool whole = walk.begun == 0 && walk.end == walk.tiles;
      // a whole item's place is by its chunk's rows, a part's by its CTA
      const int P = whole ? (rows + 7) & ~7 : 128;
      float* const mine =
          whole ? a.shared.whole + ((int64_t)__ldcg(&a.shared.chunks[walk.b].base) * a.K + (int64_t)walk.k * P) * (H + 2)
                : a.partials + ((int64_t)blockIdx.x * 2 + (walk.begun == 0 ? 1 : 0)) * paged_partial_floats(128, H);
#pragma unroll 1
      for (int c = d0; c < d0 + HD && !idle; c += 32) {
        uint32_t ov[32];
        tmem_ld32(lanes + O_COL + c, ov);
        tmem_wait_ld();
        if (r < rows) {   // lanes side by side, as in paged_decode_tc.cuh
          uint4* const dst = reinterpret_cast<uint4*>(mine) + (int64_t)(c / 4) * P + r;
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i * P] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();
      mbar_arrive(o_free);
      if (r < rows && odd == 0) {
        mine[(int64_t)P * H + r] = m;
        mine[(int64_t)P * (H + 1) + r] = l + sh_sums[item & 1][r];
      }
      if (whole && tid == 0) {
        const int item_at = walk.b * a.K + walk.k;
        a.splits[item_at] = PagedDecodeSplit{item_at, -1, 0, 0};
      }
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
