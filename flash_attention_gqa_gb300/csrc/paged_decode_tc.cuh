// Paged decode for 33 to 128 query rows per kv head, bf16 caches, H = 64 and 128:
// tcgen05 products on tiles of 128 rows x 128 keys.
//
// The split over CTAs, the partials and the join are those of paged_decode.cuh;
// only the work on a tile differs.  The query rows fill the 128-row operand
// here, and with mma.sync the products and the instructions around them bound
// the kernel from 64 rows on.  A tile of 128 keys takes 8 + 16 instructions of
// 64 cycles each at H = 128 (the weights enter as two bf16 terms), half of the
// 3000 cycles in which an SM's share of the memory rate delivers its 64 KB, so
// memory is the bound again.
//
// Roles (288 threads, one CTA an SM):
//   warps 0-3  softmax and results: thread r owns row r, a lane of tensor memory
//   warps 4-7  copies: each 32 keys of a tile, by cp.async (pages may end
//              anywhere, and keys past the request have to arrive as zeros)
//   warp  8    products (lane 0), tensor memory
// Tensor memory: S of tiles n and n + 1 at columns 0 and 128, o at 256.  The
// weights' two bf16 terms, 64 columns each, are the A operands of o += P V: one
// over its S, one at 384 or 448.
// Shared memory: the queries and a ring of K, V pairs, in chunks of [rows x
// 128 B] with the 128-byte swizzle of the operand descriptors.
#pragma once
#include "paged_decode.cuh"

namespace fa {

template <int H_>
struct DecodeTcCfg {
  static constexpr int H = H_, HC = H / 64;
  static constexpr int CK = 128, TEAMS = 1, TK = 128;   // a tile is 128 keys
  static constexpr int ITEM_UNITS = 2;
  static constexpr int WARPS = 9, THREADS = WARPS * 32;
  static constexpr int CHUNK = 128 * 128;               // 128 rows of 64 dims
  static constexpr int HALF = HC * CHUNK;               // a slot holds K, then V
  static constexpr int SLOT = 2 * HALF;
  static constexpr int STAGES = H == 64 ? 6 : 3;        // 192 KB
  static constexpr int RING = STAGES * SLOT;
  static constexpr int SMEM = HALF + RING + 1024;       // queries, ring, alignment
  static constexpr int UPR = H / 8;                     // 16-byte units of a key
};

// The bounded waits of this kernel's barriers, each by whole warps.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, const Abort& ab) {
  return __all_sync(~0u, mbar_wait(bar, parity, ab));
}

// 32 lanes x 1 column.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return __uint_as_float(r);
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) paged_decode_tc_kernel(const __grid_constant__ PagedDecodeArgs a) {
  constexpr int H = C::H, HC = C::HC, S = C::STAGES;
  constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
  extern __shared__ uint8_t smem_raw[];
  __shared__ DecodeShared<C> sh;
  __shared__ __align__(8) uint64_t bars[2 * S + 9];
  __shared__ uint32_t sh_tmem;
  __shared__ int sh_abort, sh_keep;    // sh_keep: o holds something before an item's first product
  __shared__ uint32_t sh_bad[2][4];    // keys of a tile (by its parity) whose value is not finite

  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* const sm = smem_raw + (((raw + 1023) & ~1023u) - raw);
  const uint32_t q_u = smem_u32(sm), ring_u = q_u + C::HALF;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.G * a.T;
  const DecodeShape<C> shape{a};
  const Abort ab{&sh_abort, a.wait_limit_ns, a.err};
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + S + s); };
  auto s_full = [&](int n) { return smem_u32(bars + 2 * S + (n & 1)); };
  auto p_full = [&](int n) { return smem_u32(bars + 2 * S + 2 + (n & 1)); };
  auto pv_done = [&](int n) { return smem_u32(bars + 2 * S + 4 + (n & 1)); };
  const uint32_t q_full = smem_u32(bars + 2 * S + 6), rows_met = smem_u32(bars + 2 * S + 7);
  const uint32_t teardown = smem_u32(bars + 2 * S + 8);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  DecodeWalk walk;
  if (!decode_units<C>(a, sh, walk)) return;
  if (tid == 0) {
    sh_abort = 0;
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 128);
      mbar_init(empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 128);
      mbar_init(pv_done(i), 1);
    }
    mbar_init(q_full, 128);
    mbar_init(rows_met, 128);
    mbar_init(teardown, 1);
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&sh_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh_tmem;
  constexpr uint32_t O_COL = 256, REST_COL = 384;

  if (warp == 8) {
    // -------------------------------------------------------------- products
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16(128, 128, false, false);   // S = Q K^T
      constexpr uint32_t id_o = idesc_bf16(128, H, false, true);      // o += P V
      const uint64_t dq = sdesc_sw128(q_u, 16, 1024), dk = sdesc_sw128(ring_u, 16, 1024);
      const uint64_t dv = sdesc_sw128(ring_u + C::HALF, C::CHUNK, 1024);
      bool ok = true;
      int n = 0;   // tiles so far
      auto issue_pv = [&](int n, bool first) -> bool {
        if (!mbar_wait(p_full(n), (n >> 1) & 1, ab)) return false;
        tc_fence_after();
        const uint32_t p = tmem + 128 * (n & 1);
        const uint64_t v = sdesc_add(dv, (n % S) * C::SLOT);
        const bool keep = !first || *reinterpret_cast<volatile int*>(&sh_keep);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + O_COL, p + kk * 8, sdesc_add(v, kk * 2048), id_o, keep || kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + O_COL, tmem + REST_COL + 64 * (n & 1) + kk * 8, sdesc_add(v, kk * 2048), id_o, 1u);
        mma_commit(empty(n % S));
        mma_commit(pv_done(n));
        return true;
      };
      for (int item = 0; ok; ++item) {
        ok = mbar_wait(q_full, item & 1, ab);
        for (; ok && walk.tile < walk.end; ++walk.tile, ++n) {
          if (!(ok = mbar_wait(full(n % S), (n / S) & 1, ab))) break;
          tc_fence_after();
          const uint64_t k = sdesc_add(dk, (n % S) * C::SLOT);
#pragma unroll
          for (int c = 0; c < HC; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(tmem + 128 * (n & 1), sdesc_add(dq, c * C::CHUNK + kk * 32),
                     sdesc_add(k, c * C::CHUNK + kk * 32), id_s, c > 0 || kk > 0 ? 1u : 0u);
          mma_commit(s_full(n));
          // o += P V of the tile before, while this one's softmax runs
          if (walk.tile > walk.begun) ok = issue_pv(n - 1, walk.tile - 1 == walk.begun);
        }
        if (ok) ok = issue_pv(n - 1, walk.end - 1 == walk.begun);
        if (!shape.next_item(walk, sh.ends[1])) break;
      }
      if (!ok) {   // until the products issued are over (bounded): tensor memory is freed below
        mma_commit(teardown);
        mbar_wait_teardown(teardown, 0, a.wait_limit_ns);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- copies
    const int w = warp - 4;
    constexpr int RPJ = 32 / C::UPR;   // rows a copy of the warp
    const int64_t lane_src = (lane / C::UPR) * a.lay.token + (lane % C::UPR) * 16;
    const int64_t row_step = a.lay.token * RPJ;
    const int u = lane % C::UPR, lr = lane / C::UPR;   // unit and first row of this lane
    const uint32_t lane_dst = (u >> 3) * C::CHUNK + (w * 32 + lr) * 128 + (((u & 7) ^ lr) << 4);
    bool more = true, ok = true;
    int n = 0;
    while (more && ok) {
      const int s = walk.first + walk.tile * C::TK + w * 32 + lane;   // this lane's key
      const bool live = s >= shape.low(walk.len) && s < walk.len;
      int64_t off = -1;
      if (live) {
        const int page = __ldg(a.block_table + (int64_t)walk.b * a.max_pages + (s >> a.lay.page_shift));
        if (page >= 0 && page < a.lay.n_pages)
          off = page * a.lay.page + walk.k * a.lay.head + (s & ((1 << a.lay.page_shift) - 1)) * a.lay.token;
        else
          atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
      }
      if (n >= S && !(ok = tc_wait(empty(n % S), (n / S - 1) & 1, ab))) break;
      const uint32_t dst = ring_u + (n % S) * C::SLOT + lane_dst;
      if (a.lay.page_shift >= 4 && __all_sync(~0u, off >= 0)) {
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {   // 16 keys or more a page: one offset per 16 keys, and steps
          const int64_t at = __shfl_sync(~0u, off, kt * 16) + lane_src;
          const char *pk = (const char*)a.k_cache + at, *pv = (const char*)a.v_cache + at;
#pragma unroll
          for (int j = kt * 16 / RPJ; j < (kt + 1) * 16 / RPJ; ++j) {
            const uint32_t d = (dst ^ (((j * RPJ) & 7) << 4)) + j * RPJ * 128;
            cp_async16(d, pk, 16);
            cp_async16(d + C::HALF, pv, 16);
            pk += row_step;
            pv += row_step;
          }
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < 32 / RPJ; ++j) {
          const int64_t at = __shfl_sync(~0u, off, j * RPJ + lr);
          const uint32_t bytes = at >= 0 ? 16 : 0, d = (dst ^ (((j * RPJ) & 7) << 4)) + j * RPJ * 128;
          // nothing is read, and zeros are written, where bytes = 0 (q: an address that exists)
          cp_async16(d, at >= 0 ? (const char*)a.k_cache + at + u * 16 : (const char*)a.q, bytes);
          cp_async16(d + C::HALF, at >= 0 ? (const char*)a.v_cache + at + u * 16 : (const char*)a.q, bytes);
        }
      }
      cp_async_commit();
      if (n > 0) {   // the tile before has landed: for the tensor cores to read
        cp_async_wait<1>();
        fence_proxy_async_smem();
        mbar_arrive(full((n - 1) % S));
      }
      ++n;
      if (++walk.tile == walk.end) more = shape.next_item(walk, sh.ends[1]);
    }
    cp_async_wait<0>();
    if (ok) {
      fence_proxy_async_smem();
      mbar_arrive(full((n - 1) % S));
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int r = tid, t = r % a.T;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    bool ok = true;
    int n = 0, meetings = 0;
    // all four warps have got here (a barrier with a limit)
    auto meet = [&]() -> bool {
      mbar_arrive(rows_met);
      return tc_wait(rows_met, meetings++ & 1, ab);
    };
    while (true) {
      const int64_t item = (int64_t)walk.b * a.K + walk.k;
      const char* const src = (const char*)a.q + (item * R + r) * (H * 2);
#pragma unroll
      for (int u = 0; u < H / 8; ++u) {
        const uint4 x = r < R ? __ldg(reinterpret_cast<const uint4*>(src) + u) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(sm + (u >> 3) * C::CHUNK + sw128_offset(r, u & 7)) = x;
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
      const int hi = walk.len - a.T + t + 1, lo = a.window > 0 ? hi - a.window : 0;   // keys of this row
      const int full_hi = walk.len - a.T + 1;                              // keys of every row
      const int full_lo = a.window > 0 ? max(0, walk.len - a.window) : 0;
      float m = -INFINITY, l = 0.0f;   // base of the exponents (log2 units), sum of the weights
      for (; walk.tile < walk.end; ++walk.tile, ++n) {
        if (!(ok = tc_wait(s_full(n), (n >> 1) & 1, ab))) break;
        tc_fence_after();
        const uint32_t s_col = lanes + 128 * (n & 1);
        const bool first = walk.tile == walk.begun;
        const int key0 = walk.first + walk.tile * C::TK;
        const bool masked = key0 < full_lo || key0 + C::TK > full_hi;
        // 32 scores at a time, twice: for the maximum and for the weights
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
        for (int i = 0; i < 4; ++i) {
          uint32_t sv[32];
          load_s(i, sv);
#pragma unroll
          for (int j = 0; j < 32; ++j) pm[j & 3] = fmaxf(pm[j & 3], __uint_as_float(sv[j]));
        }
        const float top = LOG2E * fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
        // The base is raised only where a score passes it by 8, as in paged_decode.cuh.
        float alpha = 1.0f;
        if (top > m + 8.0f || (first && top > m)) {
          alpha = fast_exp2(m - top);   // 0 where there was none (top is no -inf here)
          m = top;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        if (!first && __any_sync(~0u, alpha != 1.0f)) {
          if (!(ok = tc_wait(pv_done(n - 1), ((n - 1) >> 1) & 1, ab))) break;
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
        l *= alpha;

        if (first && tid == 0) sh_keep = 0;
        if (masked && a.T > 1) {
          // Values that are not finite, of keys that some row does not keep: 0 x inf
          // would reach it.  Their products are done here, row by row, and they are
          // zeros to the tensor cores.
          if (!(ok = tc_wait(full(n % S), (n / S) & 1, ab))) break;
          uint8_t* const v_row = sm + C::HALF + (n % S) * C::SLOT + C::HALF + tid * 128;
          bool bad = false;   // key `tid` of the tile
#pragma unroll
          for (int c = 0; c < HC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 x = *reinterpret_cast<const uint4*>(v_row + c * C::CHUNK + i * 16);
              const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                bad |= (y[j] & 0x7f80u) == 0x7f80u || (y[j] & 0x7f800000u) == 0x7f800000u;
            }
          const uint32_t ballot = __ballot_sync(~0u, bad);
          const uint32_t* const met = sh_bad[n & 1];
          if (lane == 0) sh_bad[n & 1][warp] = ballot;
          if (!(ok = meet())) break;
          if (met[0] | met[1] | met[2] | met[3]) {
            if (first) {
              uint32_t zero[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) zero[i] = 0;
#pragma unroll 1
              for (int c = 0; c < H; c += 32) tmem_st32(lanes + O_COL + c, zero);
              if (tid == 0) sh_keep = 1;
            } else {
              if (!(ok = tc_wait(pv_done(n - 1), ((n - 1) >> 1) & 1, ab))) break;
              tc_fence_after();
            }
            tmem_wait_st();
#pragma unroll 1
            for (int key = 0; key < 128; ++key) {
              if (!((met[key >> 5] >> (key & 31)) & 1u)) continue;
              const bool kept = key0 + key >= lo && key0 + key < hi;
              const float x = tmem_ld1(s_col + key);
              tmem_wait_ld();
              const float p = fast_exp2(fmaf(x, LOG2E, -base));
              const uint8_t* const v = sm + C::HALF + (n % S) * C::SLOT + C::HALF;
#pragma unroll 1
              for (int c = 0; c < H; c += 32) {
                uint32_t ov[32];
                tmem_ld32(lanes + O_COL + c, ov);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint4 x8 = *reinterpret_cast<const uint4*>(v + (c >> 6) * C::CHUNK +
                                                                   sw128_offset(key, (c & 63) / 8 + i));
                  const uint32_t y[4] = {x8.x, x8.y, x8.z, x8.w};
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const float2 f = unpack_bf16x2(y[j]);
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
            if (bad) {
#pragma unroll
              for (int c = 0; c < HC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  *reinterpret_cast<uint4*>(v_row + c * C::CHUNK + i * 16) = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
            fence_proxy_async_smem();
          }
        }

        // Weights as two bf16 terms (paged_decode.cuh): the cut over scores already
        // read, the rest beside o.
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t sv[32], cut[16], rest[16];
          load_s(i, sv);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float x = fast_exp2(fmaf(__uint_as_float(sv[2 * j]), LOG2E, -base));
            const float y = fast_exp2(fmaf(__uint_as_float(sv[2 * j + 1]), LOG2E, -base));
            sum[j & 3] += x + y;
            const float hx = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
            const float hy = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
            cut[j] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
            rest[j] = pack_bf16x2(fmaf(x, 0x1p-20f, x - hx), fmaf(y, 0x1p-20f, y - hy));
          }
          tmem_st16(s_col + 16 * i, cut);
          tmem_st16(lanes + REST_COL + 64 * (n & 1) + 16 * i, rest);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(n));
      }
      // ---- end of the CTA's part of the item: o from tensor memory
      if (!ok || !(ok = tc_wait(pv_done(n - 1), ((n - 1) >> 1) & 1, ab))) break;
      tc_fence_after();
      const bool whole = walk.begun == 0 && walk.end == walk.tiles;
      const float f = l == 0.0f ? 0.0f : (a.v_scale ? __ldg(a.v_scale + walk.k) : 1.0f) / l;
      float* const mine =
          a.partials + ((int64_t)blockIdx.x * 2 + (walk.begun == 0 ? 1 : 0)) * paged_partial_floats(R, H);
#pragma unroll 1
      for (int c = 0; c < H; c += 32) {
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
          uint4* const dst = reinterpret_cast<uint4*>(mine + (int64_t)r * H + c);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
        }
        __syncwarp();
      }
      if (r < R) {
        if (whole) {
          a.lse[item * R + r] = (m + log2f(l)) * LN2;   // -inf with no key
        } else {
          mine[(int64_t)R * H + r] = m;
          mine[(int64_t)R * (H + 1) + r] = l;
        }
      }
      if (whole && a.by_item && !a.unsplit && tid == 0) a.splits[item] = PagedDecodeSplit{(int)item, -1, 0, 0};
      tc_fence_before();
      if (!shape.next_item(walk, sh.ends[1])) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
