// Attention of each request's T newest tokens over its pages.
//
//   x[r, s] = q[r] . k[s],  w = softmax over the keys that row r keeps,  o[r] = sum_s w[r, s] v[s]
//
// for the R = G * T query rows of a kv head, which share its keys.  Every key
// and value byte is needed once and meets R rows, R FLOP per byte in bf16: the
// bound is memory, and the kernel is built around keeping copies in flight.
// Measured (device time): 8 requests x 8 kv heads x 32768 keys, R = 8, H = 128:
// 161 us, 6.65 TB/s; from there on 7.1 TB/s for every further byte, over a fixed
// 9.5 us (3 us until the first copies are out, 1 us of latency, 2 us in which
// CTAs end at different times, 3 us of joining).
//
// Split.  The (request, kv head) items are cut into tiles of keys; all tiles of
// all items, in order, are dealt evenly to about one wave of CTAs, so ragged
// lengths and single long requests load the GPU alike (two or three waves of
// smaller parts cost more in starts than they gain in balance: 64 ragged
// requests 74 us in one, 78 and 80 us in two and three).  The lengths stay on
// the device: every CTA sums the tile counts for itself.  An item that ends up
// in several CTAs leaves one partial (o, m, l) in each, and a second kernel,
// launched early and waiting for the first to end, joins them in key order
// (a join by the last CTA to arrive took 4 to 20 us: it has one SM's loads).
// Nothing depends on timing.
//
// Products.  mma.sync with the keys as the 16-row operand: S^T = K Q^T and
// O^T += V^T P^T waste nothing at R = 8, where tcgen05's 128-row tile would be
// mostly padding and its operands would pass through tensor memory and
// barriers.  The issue slots are 21% used at R = 8 in bf16 and 36% with 8-bit
// caches, 29% at R = 32.  mma.sync runs at one m16n8k16 per 8 cycles and
// sub-core here (640 TFLOP/s), so it and the instructions around it are the bound
// from some 32 rows on (8 rows 47 us, 32 rows 56, 64 rows 102: 16 requests x 4 kv
// heads x 8192 keys): paged_decode_tc.cuh takes more than 32 rows, and at H = 256 more
// than 16 of bf16 caches.  The S^T
// accumulator becomes the P^T operand by one 8x8 transpose (movmatrix), and maxima
// and sums live in the lanes that own the columns.
//
// Streams.  Each warp is on its own: it copies its keys (16-byte cp.async,
// swizzled so that ldmatrix is conflict-free) into its own ring, and waits for
// nobody until its CTA's part of the item ends; the ring runs ahead across items.
// 17 to 32 rows of 8-bit caches at H = 256: teams of two warps share a ring and hold 16
// rows each.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "paged.h"
#include "ptx.cuh"

namespace fa {

// ------------------------------------------------------------- primitives
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Zeros; nothing is read (`src`: an address that exists).  With the size in a register
// every copy would cost several times as much.
__device__ __forceinline__ void cp_zeros16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, 0;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Not to be hoisted out of the loop that it stands in: that would take registers.
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr));
  return x;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 x) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// d += a b, a 16 x 16 (row), b 16 x 8 (column): bf16 or f16 in, f32 out.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
                 " {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
                 " {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four e4m3 bytes to two f16 pairs (exact): bytes 0, 1 and bytes 2, 3.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(x));
}

__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) { return __half22float2(*reinterpret_cast<__half2*>(&x)); }

// For 8-bit caches a query row, `big` its largest value, is scaled to [2^10, 2^11)
// (1 for rows of zeros or infinities) and rounded to f16: exact for bf16 values down
// to 2^-27 of the largest.
__device__ __forceinline__ void e4m3_query_scale(float big, float& up, float& down) {
  const int e = big > 0.0f && big < INFINITY ? min(10 - ((int)(__float_as_uint(big) >> 23) - 127), 126) : 0;
  up = __uint_as_float((uint32_t)(e + 127) << 23);
  down = __uint_as_float((uint32_t)(127 - e) << 23);
}
// What turns a product of such a row into log2 units.  Kept between the ends of fp32: masked
// scores (-inf) times zero, and scores of zero times infinity, would be no numbers.
__device__ __forceinline__ float e4m3_score_scale(float down, float kscale) {
  const float x = down * kscale * 1.4426950408889634f, least = 0x1p-126f, most = 0x1.fffffep127f;
  return x < least ? least : x > most ? most : x;   // (NaN stays)
}

// The base of a column that has met no score: finite, so that masked scores
// (-inf) have no weight against it.
constexpr float kNoScore = -3e38f;

// The base m of the exponents, per query row, in log2 units: it is raised only where a score x
// passes it by kRaise, and then to kBelow under the largest; weights are 2^(x - m), and m
// cancels in o / l.  bf16 terms reach as far down as fp32, so any base would do.  f16 ends
// at 2^16, is coarser below 2^-14 and zero below 2^-25: with the base 11 under the largest score
// (up to 15 under a later one), all weights down to 2^-25 of the largest keep f16's 2^-11, and
// smaller ones are off by up to 2^-36 of it.  (With the largest weight near 1, a first token of
// no value that stands 16 nats above the others would cost the result 6%.)
template <bool F16>
constexpr float kRaise = F16 ? 15.0f : 8.0f;
template <bool F16>
constexpr float kBelow = F16 ? 11.0f : 0.0f;

// ------------------------------------------------------------ configuration
// NT: n-tiles of 8 query rows per warp.  WR: warps of a team, which share a ring
// and the keys in it, NT * 8 rows each.
template <int H_, bool E4M3_, int NT_, int WR_>
struct DecodeCfg {
  static constexpr int H = H_, NT = NT_, WR = WR_;
  static constexpr bool TC = false, E4M3 = E4M3_, TEAM = WR > 1;
  static constexpr int ROWB = E4M3 ? H : 2 * H;        // bytes of a key
  static constexpr int UPR = ROWB / 16;                // 16-byte units of a key
  static constexpr int CK = E4M3 || H == 64 ? 32 : 16; // keys of a ring slot
  static constexpr int HALF = CK * ROWB;               // a slot holds K, then V
  static constexpr int SLOT = 2 * HALF;
  static constexpr int WARPS = TEAM ? 8 : 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int TEAMS = WARPS / WR;
  static constexpr int TK = TEAMS * CK;                // keys of a tile
  static constexpr int ITEM_UNITS = 8 / TEAMS;         // an item's fixed cost, in tiles (below)
  static constexpr bool QSMEM = TEAM || H * NT > 256;  // query fragments in shared memory
  static constexpr int QTILES = WR * NT;
  static constexpr int QBYTES = QSMEM ? H / 16 * QTILES * 32 * 8 : 0;
  // Streams of one warp: 24 KB of ring a warp up to H = 128 (two CTAs an SM,
  // up to 128 KB of copies in flight on it), 48 KB at H = 256 (one CTA).  Teams:
  // what the queries leave of 212 KB.
  static constexpr int STAGES = TEAM ? (212 * 1024 - QBYTES) / (TEAMS * SLOT) : (H == 256 ? 48 : 24) * 1024 / SLOT;
  static constexpr int RING = TEAMS * STAGES * SLOT;
  static constexpr int SMEM = RING + QBYTES;
  static constexpr int MIN_CTAS = !TEAM && H <= 128 ? 2 : 1;
  static_assert(TEAM || (NT < 2 ? NT : 2) * 8 * H * 4 <= SLOT, "16 rows of a warp's O^T fit in a ring slot");
  static_assert(!TEAM || 2 * 32 * H <= SLOT, "8 rows of two warps' O^T fit in a ring slot");
  static_assert(STAGES >= 3, "");
};

// Byte offset of 16-byte unit `u` of row `r`: any 8 consecutive rows have one
// unit in 8 different bank groups.
// A lane's address of unit u0 in its row, xor (u << 4), is that of unit u0 ^ u: slots
// are aligned to whole rows.
template <int UPR>
__device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t u) {
  return UPR >= 8 ? r * (UPR * 16) + ((u ^ (r & 7)) << 4) : r * 64 + ((u ^ ((r >> 1) & 3)) << 4);
}

// ------------------------------------------------------------------ the walk
// a / b for a, b >= 0: mostly in 32 bits, which takes a fraction of the time.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The list that is dealt to the CTAs: per item (b, k) ITEM_UNITS units that
// stand for its start and end (about the time of two tiles of four warps), then
// one unit per tile.  64 requests of 1 to 16384 tokens: 108 us without those
// units, 75.0, 74.4, 75.3 and 76.8 us with 1, 2, 3 and 6.

// A place in the list: unit `rem` of item (b, k).
struct DecodePlace {
  int b, k, rem;
};

// Unit t of request b's.
struct DecodeEnd {
  int b, len;
  long long t;
};

// The part of an item that a CTA does: tiles [begun, end) of its `tiles`.
struct DecodeWalk {
  int b, k, len, first, tiles;   // first: key of tile 0, a multiple of CK
  int tile, begun, end;
  int todo;                      // items that follow
};

template <class C>
struct DecodeShape {
  const PagedDecodeArgs& a;
  __device__ __forceinline__ int length(int b) const {
    const int n = a.lens[b];
    return min(max(n, 0), a.max_pages << a.lay.page_shift);
  }
  // First key any of the T queries keeps.
  __device__ __forceinline__ int low(int len) const {
    return a.window > 0 ? max(0, len - a.T + 1 - a.window) : 0;
  }
  __device__ __forceinline__ int first(int len) const { return low(len) & ~(C::CK - 1); }
  __device__ __forceinline__ int tiles(int len) const {
    return max(1, (len - first(len) + C::TK - 1) / C::TK);   // an empty item writes its zeros
  }
  __device__ __forceinline__ DecodePlace place(const DecodeEnd& e) const {
    const int per_item = tiles(e.len) + C::ITEM_UNITS, k = (int)quotient(e.t, per_item);
    return DecodePlace{e.b, k, (int)(e.t - (long long)k * per_item)};
  }
  __device__ __forceinline__ void enter(DecodeWalk& w, int b, int k) const {
    w.b = b;
    w.k = k;
    w.len = length(b);
    w.first = first(w.len);
    w.tiles = tiles(w.len);
    w.tile = w.begun = 0;
    w.end = w.tiles;
  }
  // From the item that the CTA's units begin in to the one that they end in.
  // False where they hold no tile at all.
  __device__ __forceinline__ bool begin(DecodeWalk& w, const DecodePlace& h, const DecodePlace& e) const {
    const int between = (e.b - h.b) * a.K + e.k - h.k;   // items
    enter(w, h.b, h.k);
    if (a.unsplit) {   // an item is done whole by the CTA that its first unit is in
      w.todo = between;
      return h.rem == 0 || next_item(w, DecodeEnd{});
    }
    w.tile = w.begun = max(0, h.rem - C::ITEM_UNITS);
    const int last_end = e.rem + 1 - C::ITEM_UNITS;   // of the last item
    w.todo = last_end > 0 ? between : between - 1;
    if (between == 0) w.end = min(w.end, last_end);
    return w.end > w.begun;
  }
  // `last`: of the CTA's last unit (read again: once an item costs less than a
  // register).
  __device__ __forceinline__ bool next_item(DecodeWalk& w, const DecodeEnd& last) const {
    if (w.todo <= 0) return false;
    --w.todo;
    if (w.k + 1 == a.K) {
      enter(w, w.b + 1, 0);
    } else {
      ++w.k;
      w.tile = w.begun = 0;
      w.end = w.tiles;
    }
    if (w.todo == 0 && !a.unsplit) {
      const int last_end = place(last).rem + 1 - C::ITEM_UNITS;
      if (last_end > 0) w.end = min(w.end, last_end);
    }
    return true;
  }
};

// What the CTAs share of the split's arithmetic.
template <class C>
struct DecodeShared {
  long long scan[C::WARPS];
  DecodeEnd ends[2];   // first and last unit
};

// Finds this CTA's units, by all its threads, and enters its first item; false
// where it has no tile.
template <class C>
__device__ __forceinline__ bool decode_units(const PagedDecodeArgs& a, DecodeShared<C>& sh, DecodeWalk& walk) {
  constexpr int threads = C::THREADS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const DecodeShape<C> shape{a};
  const int per = (a.B + threads - 1) / threads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    if (blockIdx.x == 0) {
      const int n = a.lens[b];
      if (n != shape.length(b)) atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
    }
    mine += (long long)(shape.tiles(shape.length(b)) + C::ITEM_UNITS) * a.K;
  }
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31) sh.scan[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  // CTA i: total / ctas units, and one more where i < total % ctas
  const int ctas = (int)min((long long)gridDim.x, total), i = blockIdx.x;
  if (i >= ctas) {
    if (tid == 0 && !a.by_item && !a.unsplit) a.splits[i] = PagedDecodeSplit{0, -1, 0, 0};
    return false;
  }
  const long long each = quotient(total, ctas), over = total - each * ctas;
  const long long t0 = i * each + min((long long)i, over), t1 = t0 + each + (i < over ? 1 : 0);
  const long long at = before + inc - mine;
  if (t0 < at + mine && t1 - 1 >= at) {   // the requests that hold the first and the last unit
    long long x = at;
    for (int b = b0; b < b1; ++b) {
      const int len = shape.length(b);
      const long long next = x + (long long)(shape.tiles(len) + C::ITEM_UNITS) * a.K;
      if (t0 >= x && t0 < next) sh.ends[0] = DecodeEnd{b, len, t0 - x};
      if (t1 - 1 >= x && t1 - 1 < next) sh.ends[1] = DecodeEnd{b, len, t1 - 1 - x};
      x = next;
    }
  }
  __syncthreads();
  const DecodePlace head = shape.place(sh.ends[0]), tail = shape.place(sh.ends[1]);
  if (tid == 32 && !a.unsplit) {
    // the item that the units end in, where it begins here and goes on in the
    // next CTA: for the join, with its last CTA
    const int tiles = shape.tiles(sh.ends[1].len);
    const long long first = t1 - 1 - tail.rem + C::ITEM_UNITS;   // its first tile's unit
    const bool split = tail.rem >= C::ITEM_UNITS && tail.rem + 1 < tiles + C::ITEM_UNITS && first >= t0;
    if (split || !a.by_item) {
      const long long unit = first + tiles - 1, cut = over * (each + 1);
      const long long last = unit < cut ? quotient(unit, each + 1) : over + quotient(unit - cut, each);
      const int item = tail.b * a.K + tail.k;
      a.splits[a.by_item ? item : i] = PagedDecodeSplit{item, split ? i : -1, (int)last, 0};
    }
  }
  return shape.begin(walk, head, tail);
}

// Whether any 16-bit (bf16) or 8-bit (e4m3) value of the `bytes` at `p` is not
// finite; warp-wide.
template <bool E4M3>
__device__ __forceinline__ bool any_not_finite(const char* p, int bytes, int lane) {
  bool bad = false;
  for (int i = lane * 16; i < bytes; i += 512) {
    const uint4 x = *reinterpret_cast<const uint4*>(p + i);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (E4M3) {   // all seven low bits of a byte set: NaN (e4m3 has no infinity)
        const uint32_t y = ~w[j] & 0x7f7f7f7fu;
        bad |= ((y - 0x01010101u) & ~y & 0x80808080u) != 0;
      } else {
        bad |= (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
      }
    }
  }
  return __any_sync(~0u, bad);
}

// --------------------------------------------------------------- results
// The four dims of row r of a joined or whole result, rounded to bf16 once.
__device__ __forceinline__ void put_result(void* o, float* lse, int H, int r, int d, float4 x, float M,
                                           float L, float vscale) {
  const float f = L == 0.0f ? 0.0f : vscale / L;
  const uint2 y = make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
  *reinterpret_cast<uint2*>((char*)o + ((int64_t)r * H + d) * 2) = y;
  if (d == 0) lse[r] = (M + log2f(L)) * 0.6931471805599453f;   // -inf with no key
}
__device__ __forceinline__ void put_partial(float* dst, int H, int P, int r, int d, float4 x, float M, float L) {
  *reinterpret_cast<float4*>(dst + (int64_t)r * H + d) = x;
  if (d == 0) {
    dst[(int64_t)P * H + r] = M;
    dst[(int64_t)P * (H + 1) + r] = L;
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::MIN_CTAS)
paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a) {
  constexpr int H = C::H, NT = C::NT, CK = C::CK, KT = CK / 16, KS = H / 16, S = C::STAGES;
  constexpr int WR = C::WR, WARPS = C::WARPS, threads = C::THREADS;
  constexpr bool E4M3 = C::E4M3, TEAM = C::TEAM;
  constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
  extern __shared__ __align__(1024) char smem[];
  __shared__ float sh_m[WARPS][16], sh_l[WARPS][16];
  __shared__ float4 sh_ml[TEAM ? WARPS : 1][32];
  __shared__ float sh_down[C::QTILES * 8];     // what undoes the scaling of a query row
  __shared__ DecodeShared<C> sh;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int R = a.G * a.T, P = paged_partial_rows(R);
  const DecodeShape<C> shape{a};

  // The join may be launched as soon as every CTA has got here; it waits.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's units
  DecodeWalk walk;
  if (!decode_units<C>(a, sh, walk)) return;
  DecodeWalk ahead = walk;   // where the copies are
  bool more = true;

  // ---- copies: lane r looks up key r of the next slot one slot early, then all
  // lanes copy 16-byte units of it
  const int team = warp / WR, wr = warp % WR;
  char* const ring = smem + team * S * C::SLOT;
  const uint32_t ring_u = smem_u32(ring);
  int64_t key_off = -1;   // lane r: byte offset of key r of the slot to come, -1: zeros
  int key_page = -1, key_in = 0, key_head = 0;
  bool key_live = false;
  // this lane's unit of the first rows copied: where it is and where it goes
  const int64_t lane_src = (lane / C::UPR) * a.lay.token + (lane % C::UPR) * 16;
  const int64_t row_step = a.lay.token * (32 / C::UPR);
  const uint32_t lane_dst = swz<C::UPR>(lane / C::UPR, lane % C::UPR);
  // the swizzle of rows j * 32 / UPR on from that of the first rows
  auto swz_step = [](int j) -> uint32_t {
    constexpr int RPJ = 32 / C::UPR;
    return C::UPR >= 8 ? ((j * RPJ) & 7) << 4 : ((j * RPJ >> 1) & 3) << 4;
  };
  auto look_up = [&]() {
    key_live = false;
    if (!more) return;
    const int s = ahead.first + (ahead.tile * C::TEAMS + team) * CK + (lane & (CK - 1));
    key_live = s >= shape.low(ahead.len) && s < ahead.len;
    key_in = s & ((1 << a.lay.page_shift) - 1);
    key_head = ahead.k;
    if (key_live) key_page = __ldg(a.block_table + (int64_t)ahead.b * a.max_pages + (s >> a.lay.page_shift));
  };
  auto issue = [&](int slot) {
    key_off = -1;
    if (key_live) {
      if (key_page >= 0 && key_page < a.lay.n_pages)
        key_off = key_page * a.lay.page + key_head * a.lay.head + key_in * a.lay.token;
      else
        atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
    }
    const uint32_t dst = ring_u + slot * C::SLOT;
    constexpr int NJ = CK * C::UPR / 32, RPJ = 32 / C::UPR;   // copies a lane, rows a copy
    if (a.lay.page_shift >= 3 && __all_sync(~0u, key_off >= 0)) {
      // whole slot, 8 keys or more a page: one offset per 8 keys, and steps
      constexpr int K8 = CK / 8;
#pragma unroll
      for (int k8 = 0; k8 < K8; ++k8) {
        const int64_t off = __shfl_sync(~0u, key_off, k8 * 8) + lane_src;
        const char *pk = (const char*)a.k_cache + off, *pv = (const char*)a.v_cache + off;
#pragma unroll
        for (int j = k8 * NJ / K8; j < (k8 + 1) * NJ / K8; ++j) {
          if (j % WR == wr) {
            const uint32_t d = (dst + lane_dst ^ swz_step(j)) + j * RPJ * C::ROWB;
            cp_async16(d, pk);
            cp_async16(d + C::HALF, pv);
          }
          pk += row_step;
          pv += row_step;
        }
      }
    } else if (__any_sync(~0u, key_live)) {
#pragma unroll 1
      for (int j = 0; j < NJ; ++j) {
        if (j % WR != wr) continue;
        const int row = j * RPJ + lane / C::UPR, u = lane % C::UPR;
        const int64_t off = __shfl_sync(~0u, key_off, row);
        const uint32_t d = dst + swz<C::UPR>(row, u);
        if (off >= 0) {
          cp_async16(d, (const char*)a.k_cache + off + u * 16);
          cp_async16(d + C::HALF, (const char*)a.v_cache + off + u * 16);
        } else {
          cp_zeros16(d, a.q);
          cp_zeros16(d + C::HALF, a.q);
        }
      }
    }
    cp_async_commit();
    if (more && ++ahead.tile == ahead.end) more = shape.next_item(ahead, sh.ends[1]);
    look_up();
  };
  look_up();
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) issue(i);

  // ---- items
  int cur = 0;
  const int row0 = wr * NT * 8;   // first query row of this warp
  uint4* const q_sm = reinterpret_cast<uint4*>(smem + C::RING);   // [pair of ks][n-tile][lane]
  const uint32_t q_u = smem_u32(q_sm + wr * NT * 32 + lane);
  // Query fragments: column n = lane / 4, dims as the key operand has them.
  auto load_q = [&](const DecodeWalk& w, int nt, uint2 (&x)[KS]) {
    const int r = nt * 8 + g;
    const char* src = (const char*)a.q + (((int64_t)w.b * a.K + w.k) * R + r) * (H * 2);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      x[ks] = make_uint2(0, 0);
      if (r < R) {
        if (E4M3) {
          x[ks] = __ldg(reinterpret_cast<const uint2*>(src + ks * 32 + c * 8));
        } else {
          x[ks].x = __ldg(reinterpret_cast<const uint32_t*>(src + ks * 32 + c * 4));
          x[ks].y = __ldg(reinterpret_cast<const uint32_t*>(src + ks * 32 + 16 + c * 4));
        }
      }
    }
  };
  // The rows of an n-tile, scaled and rounded to f16 for 8-bit caches.  Returns what
  // undoes it.
  auto scale_q = [&](uint2 (&x)[KS]) -> float {
    float big = 0.0f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const float2 p = unpack_bf16x2(x[ks].x), q = unpack_bf16x2(x[ks].y);
      big = fmaxf(fmaxf(big, fmaxf(fabsf(p.x), fabsf(p.y))), fmaxf(fabsf(q.x), fabsf(q.y)));
    }
    big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
    big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
    float up, down;
    e4m3_query_scale(big, up, down);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const float2 p = unpack_bf16x2(x[ks].x), q = unpack_bf16x2(x[ks].y);
      x[ks] = make_uint2(pack_f16x2(p.x * up, p.y * up), pack_f16x2(q.x * up, q.y * up));
    }
    return down;
  };
  // The next item's queries are read while this one's results are written,
  // where registers allow it.
  constexpr bool EARLY = !C::QSMEM && NT * KS <= 16;
  uint2 q_next[EARLY ? NT : 1][KS];
  if (EARLY) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) load_q(walk, nt, q_next[EARLY ? nt : 0]);
  }
  while (true) {
    const int64_t item = (int64_t)walk.b * a.K + walk.k;
    uint2 qf[C::QSMEM ? 1 : KS][NT];
    float sl2[NT][2];      // score to log2 units, per column
    const float kscale = a.k_scale ? __ldg(a.k_scale + walk.k) : 1.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) sl2[nt][0] = sl2[nt][1] = LOG2E;
    if constexpr (C::QSMEM) {
      // one copy for the CTA's warps, which take its n-tiles in turn
#pragma unroll
      for (int nt0 = 0; nt0 < C::QTILES; nt0 += WARPS) {
        const int nt = nt0 + warp;
        if (nt >= C::QTILES) continue;
        uint2 x[KS];
        load_q(walk, nt, x);
        if (E4M3) {
          const float down = scale_q(x);
          if (c == 0) sh_down[nt * 8 + g] = down;
        }
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2)
          q_sm[(ks / 2 * C::QTILES + nt) * 32 + lane] = make_uint4(x[ks].x, x[ks].y, x[ks + 1].x, x[ks + 1].y);
      }
      __syncthreads();
      if (E4M3) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) sl2[nt][j] = e4m3_score_scale(sh_down[row0 + nt * 8 + 2 * c + j], kscale);
      }
    } else {
      uint2 x[NT][KS];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (EARLY) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) x[nt][ks] = q_next[EARLY ? nt : 0][ks];
        } else {
          load_q(walk, nt, x[nt]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (E4M3) {
          const float down = scale_q(x[nt]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            sl2[nt][j] = e4m3_score_scale(__shfl_sync(~0u, down, (2 * c + j) * 4), kscale);
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[C::QSMEM ? 0 : ks][nt] = x[nt][ks];
        }
      }
    }
    // Keys that column (nt, j) keeps: [hi - window, hi)
    int col_hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        col_hi[nt][j] = walk.len - a.T + 1 + (a.T == 1 ? 0 : (row0 + nt * 8 + 2 * c + j) % a.T);
    const int full_hi = walk.len - a.T + 1;                              // all columns keep keys
    const int full_lo = a.window > 0 ? max(0, walk.len - a.window) : 0;   // in [full_lo, full_hi)

    float o[KS][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNoScore;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int ds = 0; ds < KS; ++ds) o[ds][nt][0] = o[ds][nt][1] = o[ds][nt][2] = o[ds][nt][3] = 0.0f;
    }

    for (; walk.tile < walk.end; ++walk.tile) {
      cp_async_wait<S - 2>();
      if (TEAM) named_bar_sync(1 + team, WR * 32); else __syncwarp();
      {
        const int next = cur == 0 ? S - 1 : cur - 1;   // the slot of the chunk before: free
        issue(next);
      }
      const uint32_t ks_u = ring_u + cur * C::SLOT, vs_u = ks_u + C::HALF;
      const char* const vs_p = ring + cur * C::SLOT + C::HALF;
      cur = cur + 1 == S ? 0 : cur + 1;
      const int key0 = walk.first + (walk.tile * C::TEAMS + team) * CK;
      if (key0 >= walk.len) continue;   // this team has no keys in the tile

      // A slot's keys at once, or with many rows (registers) 16 at a time.
      constexpr int KT2 = NT < 4 ? KT : 1;
      constexpr bool TWO = NT < 4;
#pragma unroll 1
      for (int k0 = 0; k0 < CK; k0 += KT2 * 16) {
        const int key1 = key0 + k0;
        if (k0 && key1 >= walk.len) break;
        const uint32_t k_u = ks_u + k0 * C::ROWB, v_u = vs_u + k0 * C::ROWB;
        // S^T = K Q^T
        float s[KT2][NT][4];
#pragma unroll
        for (int kt = 0; kt < KT2; ++kt) {
          float s2[TWO ? NT : 1][4];   // a second chain of products where there are few
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[kt][nt][i] = s2[TWO ? nt : 0][i] = 0.0f;
          const uint32_t k_lane = k_u + kt * 16 * C::ROWB + swz<C::UPR>(lane & 15, lane >> 4);
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
            uint32_t a0[4], a1[4];   // the keys' dims of two steps
            if (E4M3) {
              uint32_t x[4];
              ldsm4(k_lane ^ (ks << 4), x);
              e4m3x4_to_f16(x[0], a0[0], a0[2]);
              e4m3x4_to_f16(x[1], a0[1], a0[3]);
              e4m3x4_to_f16(x[2], a1[0], a1[2]);
              e4m3x4_to_f16(x[3], a1[1], a1[3]);
            } else {
              ldsm4(k_lane ^ (ks << 5), a0);
              ldsm4(k_lane ^ (ks << 5) ^ 32, a1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint4 q;
              if (C::QSMEM) {
                q = lds16(q_u + (ks / 2 * C::QTILES + nt) * 512);
              } else {
                const uint2 q0 = qf[C::QSMEM ? 0 : ks][nt], q1 = qf[C::QSMEM ? 0 : ks + 1][nt];
                q = make_uint4(q0.x, q0.y, q1.x, q1.y);
              }
              mma16816<E4M3>(s[kt][nt], a0, q.x, q.y);
              mma16816<E4M3>(TWO ? s2[TWO ? nt : 0] : s[kt][nt], a1, q.z, q.w);
            }
          }
          if (TWO) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[kt][nt][i] += s2[TWO ? nt : 0][i];
          }
        }
        const bool masked = key1 < full_lo || key1 + KT2 * 16 > full_hi;
        if (masked) {
#pragma unroll
          for (int kt = 0; kt < KT2; ++kt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = key1 + kt * 16 + g + (i >> 1) * 8, hi = col_hi[nt][i & 1];
                if (key >= hi || (a.window > 0 && key < hi - a.window)) s[kt][nt][i] = -INFINITY;
              }
        }

        // Online softmax, per column.  The base m of the exponents is raised only
        // where a score passes it by far (kRaise), so that most slots need neither the
        // maximum over the lanes nor a rescaling of o.
        bool high = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
            for (int kt = 1; kt < KT2; ++kt) mx = fmaxf(mx, fmaxf(s[kt][nt][j], s[kt][nt][j + 2]));
            high |= fmaf(mx, sl2[nt][j], -m[nt][j]) > kRaise<E4M3>;
          }
        if (__any_sync(~0u, high)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float alpha[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float mx = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
              for (int kt = 1; kt < KT2; ++kt) mx = fmaxf(mx, fmaxf(s[kt][nt][j], s[kt][nt][j + 2]));
              mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
              const float mn = fmaxf(m[nt][j], mx * sl2[nt][j] - kBelow<E4M3>);
              alpha[j] = fast_exp2(m[nt][j] - mn);
              m[nt][j] = mn;
              l[nt][j] *= alpha[j];
            }
#pragma unroll
            for (int ds = 0; ds < KS; ++ds) {
              o[ds][nt][0] *= alpha[0];
              o[ds][nt][1] *= alpha[1];
              o[ds][nt][2] *= alpha[0];
              o[ds][nt][3] *= alpha[1];
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float sum = 0.0f;
#pragma unroll
            for (int kt = 0; kt < KT2; ++kt) {
              s[kt][nt][j] = fast_exp2(fmaf(s[kt][nt][j], sl2[nt][j], -m[nt][j]));
              s[kt][nt][j + 2] = fast_exp2(fmaf(s[kt][nt][j + 2], sl2[nt][j], -m[nt][j]));
              sum += s[kt][nt][j] + s[kt][nt][j + 2];
            }
            l[nt][j] += sum;
          }

        // O^T += V^T P^T.  bf16 caches: the weights go in as two bf16 terms, cut
        // and rest (off by 2^-16 in all), so that o is rounded to bf16 once, at the
        // end.  The rest is kept above zero, or an infinite value would give
        // 0 x inf.  8-bit caches: one f16 term, off by 2^-11 (kRaise), against values off by 2^-4.
        uint32_t p[KT2][NT][2], pl[KT2][NT][2];
#pragma unroll
        for (int kt = 0; kt < KT2; ++kt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = s[kt][nt][2 * h], y = s[kt][nt][2 * h + 1];
              if (E4M3) {
                p[kt][nt][h] = transpose8x8(pack_f16x2(x, y));
              } else {
                const float hx = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
                const float hy = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
                p[kt][nt][h] = transpose8x8(__byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632));
                pl[kt][nt][h] = transpose8x8(pack_bf16x2(fmaf(x, 1 + 0x1p-20f, -hx), fmaf(y, 1 + 0x1p-20f, -hy)));
              }
            }
        // Operand V^T of 16 keys and 16 dims (8-bit: 32 dims, two operands).
        auto load_v = [&](int kt, int ds, uint32_t (&v0)[4], uint32_t (&v1)[4]) {
          if (E4M3) {
            uint32_t x[4];
            ldsm4_trans((v_u + kt * 16 * C::ROWB + swz<C::UPR>(lane & 15, lane >> 4)) ^ (ds << 4), x);
            // bytes (key 2c: dims 2g, 2g+1), (key 2c+1: the same) -> pairs of keys per dim
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __byte_perm(x[i], 0, 0x3120);
            e4m3x4_to_f16(x[0], v0[0], v0[1]);
            e4m3x4_to_f16(x[1], v0[2], v0[3]);
            e4m3x4_to_f16(x[2], v1[0], v1[1]);
            e4m3x4_to_f16(x[3], v1[2], v1[3]);
          } else {
            ldsm4_trans((v_u + kt * 16 * C::ROWB +
                         swz<C::UPR>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1)) ^ (ds << 5), v0);
          }
        };
        auto add_v = [&](float (&d)[4], const uint32_t (&v)[4], int kt, int nt) {
          mma16816<E4M3>(d, v, p[kt][nt][0], p[kt][nt][1]);
          if (!E4M3) mma16816<E4M3>(d, v, pl[kt][nt][0], pl[kt][nt][1]);
        };
        if (masked && a.T > 1 && any_not_finite<E4M3>(vs_p + k0 * C::ROWB, KT2 * 16 * C::ROWB, lane)) {
          // Some column does not keep a key whose value is an infinity or NaN, and
          // 0 x inf would reach it: each query position gets its own products, the
          // keys that it does not keep zeroed, and takes its columns of them.
#pragma unroll 1
          for (int t = 0; t < a.T; ++t) {
            const int hi = full_hi + t, lo = a.window > 0 ? hi - a.window : 0;
#pragma unroll
            for (int kt = 0; kt < KT2; ++kt) {
              uint32_t keep[2];   // of keys 2c, 2c + 1 and those + 8, as halves
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = key1 + kt * 16 + 2 * c + 8 * h;
                keep[h] = (key >= lo && key < hi ? 0xffffu : 0u) |
                          (key + 1 >= lo && key + 1 < hi ? 0xffff0000u : 0u);
              }
#pragma unroll
              for (int ds = 0; ds < KS; ds += E4M3 ? 2 : 1) {
                uint32_t v[2][4];
                load_v(kt, ds, v[0], v[1]);
#pragma unroll
                for (int i = 0; i < (E4M3 ? 2 : 1); ++i) {
                  v[i][0] &= keep[0];
                  v[i][1] &= keep[0];
                  v[i][2] &= keep[1];
                  v[i][3] &= keep[1];
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    add_v(d, v[i], kt, nt);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if (col_hi[nt][e & 1] == hi) o[ds + i][nt][e] += d[e];
                  }
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int kt = 0; kt < KT2; ++kt)
#pragma unroll
            for (int ds = 0; ds < KS; ds += E4M3 ? 2 : 1) {
              uint32_t v[2][4];
              load_v(kt, ds, v[0], v[1]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                add_v(o[ds][nt], v[0], kt, nt);
                if (E4M3) add_v(o[ds + (E4M3 ? 1 : 0)][nt], v[1], kt, nt);
              }
            }
        }
      }
    }

    // ---- end of the CTA's part of the item
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (m[nt][j] == kNoScore) m[nt][j] = -INFINITY;
        l[nt][j] += __shfl_xor_sync(~0u, l[nt][j], 4);
        l[nt][j] += __shfl_xor_sync(~0u, l[nt][j], 8);
        l[nt][j] += __shfl_xor_sync(~0u, l[nt][j], 16);
      }
    const bool whole = walk.begun == 0 && walk.end == walk.tiles;
    DecodeWalk then = walk;
    const bool go_on = shape.next_item(then, sh.ends[1]);
    if (EARLY && go_on) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) load_q(then, nt, q_next[EARLY ? nt : 0]);
    }
    const float vscale = a.v_scale ? __ldg(a.v_scale + walk.k) : 1.0f;
    const int64_t out_row = item * R;
    // Partials: slot 1 of a CTA holds the item that starts in it, slot 0 one
    // that started before.
    float* const mine = a.partials + ((int64_t)blockIdx.x * 2 + (walk.begun == 0 ? 1 : 0)) * paged_partial_floats(R, H);
    auto put = [&](int r, int d, float4 x, float M, float L) {   // four dims of row r
      if (whole) put_result((char*)a.o + out_row * H * 2, a.lse + out_row, H, r, d, x, M, L, vscale);
      else put_partial(mine, H, P, r, d, x, M, L);
    };
    // O^T goes through shared memory: the slot just used, free until the next
    // copies are issued.  Four dims stay together; dims move by 8 with the column
    // pair, against bank conflicts.  16 rows at a time.
    float* const so = reinterpret_cast<float*>(ring + (cur == 0 ? S - 1 : cur - 1) * C::SLOT);
    if (!TEAM) {
      constexpr int NR = NT < 2 ? NT : 2;   // n-tiles a round
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += NR) {
        if (n0 * 8 >= R) break;
        __syncwarp();
#pragma unroll
        for (int ds = 0; ds < KS; ++ds)
#pragma unroll
          for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float* const row = so + (nt * 8 + 2 * c + j) * H;
              if (E4M3) {
                *reinterpret_cast<float2*>(row + ((ds * 16 + 2 * g) ^ (c << 3))) =
                    make_float2(o[ds][n0 + nt][j], o[ds][n0 + nt][j + 2]);
              } else {
                row[(ds * 16 + g) ^ (c << 3)] = o[ds][n0 + nt][j];
                row[(ds * 16 + g + 8) ^ (c << 3)] = o[ds][n0 + nt][j + 2];
              }
            }
        if (g == 0) {
#pragma unroll
          for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              sh_m[warp][nt * 8 + 2 * c + j] = m[n0 + nt][j];
              sh_l[warp][nt * 8 + 2 * c + j] = l[n0 + nt][j];
            }
        }
        __syncthreads();
        const int rows = min(NR * 8, R - n0 * 8);
        for (int i = tid; i < rows * (H / 4); i += threads) {
          const int r = i / (H / 4), d = i % (H / 4) * 4;
          float M = sh_m[0][r], L = 0.0f;
#pragma unroll
          for (int w = 1; w < WARPS; ++w) M = fmaxf(M, sh_m[w][r]);
          const float base = M == -INFINITY ? 0.0f : M;
          float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          // every warp's ring has the same slot at the same place
          const float* at = reinterpret_cast<const float*>(smem + ((const char*)so - ring)) + r * H +
                            (d ^ (((r >> 1) & 3) << 3));
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            const float f = fast_exp2(sh_m[w][r] - base);
            const float4 y = *reinterpret_cast<const float4*>(at + w * (S * C::SLOT / 4));
            L += sh_l[w][r] * f;
            x.x += y.x * f;
            x.y += y.y * f;
            x.z += y.z * f;
            x.w += y.w * f;
          }
          put(n0 * 8 + r, d, x, M, L);
        }
        __syncthreads();
      }
    } else {
      // Teams are joined in pairs, an n-tile at a time: a lane of the one adds
      // what the same lane of the other left in the slots just used.
#pragma unroll
      for (int step = C::TEAMS / 2; step; step /= 2) {
        const int index = (team - step) * WR + wr, from = index + step * WR;   // of the writer, here and there
        auto area = [&](int i) {
          return reinterpret_cast<float4*>(smem + (step + i / 2) % (2 * step) * S * C::SLOT + ((char*)so - ring) +
                                           i % 2 * 32 * H) + lane;
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          __syncthreads();
          if (team >= step && team < 2 * step) {
            float4* const dst = area(index);
#pragma unroll
            for (int ds = 0; ds < KS; ++ds)
              dst[ds * 32] = make_float4(o[ds][nt][0], o[ds][nt][1], o[ds][nt][2], o[ds][nt][3]);
            sh_ml[warp][lane] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
          }
          __syncthreads();
          if (team < step) {
            const float4* const src = area(from);
            const float4 ml = sh_ml[warp + step * WR][lane];
            const float other[2] = {ml.x, ml.y}, sum[2] = {ml.z, ml.w};
            float f[2], h[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float mn = fmaxf(m[nt][j], other[j]), base = mn == -INFINITY ? 0.0f : mn;
              f[j] = fast_exp2(m[nt][j] - base);
              h[j] = fast_exp2(other[j] - base);
              m[nt][j] = mn;
              l[nt][j] = l[nt][j] * f[j] + sum[j] * h[j];
            }
#pragma unroll
            for (int ds = 0; ds < KS; ++ds) {
              const float4 y = src[ds * 32];
              o[ds][nt][0] = o[ds][nt][0] * f[0] + y.x * h[0];
              o[ds][nt][1] = o[ds][nt][1] * f[1] + y.y * h[1];
              o[ds][nt][2] = o[ds][nt][2] * f[0] + y.z * h[0];
              o[ds][nt][3] = o[ds][nt][3] * f[1] + y.w * h[1];
            }
          }
        }
      }
      __syncthreads();
      if (team == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = row0 + nt * 8 + 2 * c + j;
            const float L = l[nt][j], M = m[nt][j];
            f[j] = L == 0.0f ? 0.0f : vscale / L;
            if (r >= R) continue;
            if (whole) {
              if (g == 0) a.lse[out_row + r] = (M + log2f(L)) * LN2;
            } else {
              if (g == 0) {
                mine[(int64_t)P * H + r] = M;
                mine[(int64_t)P * (H + 1) + r] = L;
              }
#pragma unroll
              for (int ds = 0; ds < KS; ++ds) {
                const int d0 = ds * 16 + (E4M3 ? 2 * g : g), d1 = d0 + (E4M3 ? 1 : 8);
                mine[(int64_t)r * H + d0] = o[ds][nt][j];
                mine[(int64_t)r * H + d1] = o[ds][nt][j + 2];
              }
            }
          }
          if (whole) {   // transposed: row g, dims in pairs
            const int r = row0 + nt * 8 + g;
            char* const dst = (char*)a.o + (out_row + r) * (H * 2);
#pragma unroll
            for (int ds = 0; ds < KS; ++ds) {
              const uint32_t x = transpose8x8(pack_bf16x2(o[ds][nt][0] * f[0], o[ds][nt][1] * f[1]));
              const uint32_t y = transpose8x8(pack_bf16x2(o[ds][nt][2] * f[0], o[ds][nt][3] * f[1]));
              if (r >= R) continue;
              if (E4M3) {   // x: dims 4c and 4c + 2, y: dims 4c + 1 and 4c + 3
                *reinterpret_cast<uint2*>(dst + ds * 32 + c * 8) =
                    make_uint2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
              } else {
                *reinterpret_cast<uint32_t*>(dst + ds * 32 + c * 4) = x;
                *reinterpret_cast<uint32_t*>(dst + ds * 32 + 16 + c * 4) = y;
              }
            }
          }
        }
      }
    }

    if (whole && a.by_item && !a.unsplit && tid == 0) a.splits[item] = PagedDecodeSplit{(int)item, -1, 0, 0};
    if (!go_on) break;
    walk = then;
  }
  cp_async_wait<0>();
}

// Joins the partials of an item that several CTAs of the first kernel share: a
// thread per four dims of a row and share of the partials, `per` such elements a
// CTA, whose shares are then summed in order.  U: partials in flight a thread.  TC:
// partials of the tcgen05 kernel, of which a warp takes 4 x 4 dims of 8 rows.
// Few registers and threads a CTA, so that the whole grid starts at once as the
// first one ends (512 threads of 75 registers, one CTA an SM, took 4 us).
template <int H, bool TC, int U, int THREADS>
__global__ void __launch_bounds__(THREADS)
paged_join_kernel(const __grid_constant__ PagedDecodeArgs a, int ctas, int per) {
  __shared__ float4 sx[THREADS];
  __shared__ float2 sml[THREADS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (L2 loads: this grid may have started before the first one wrote)
  const int4 split = __ldcg(reinterpret_cast<const int4*>(a.splits) + blockIdx.x);
  const int item = split.x, first = split.y, n = split.z - first + 1;   // n partials
  // (an entry of a whole item holds anything where a wait of the first kernel ran out before it)
  if (first < 0 || split.z < first || split.z >= ctas || (unsigned)item >= (unsigned)(a.B * a.K)) return;
  const int R = a.G * a.T, P = paged_partial_rows(R), shares = blockDim.x / per;
  const int share = threadIdx.x / per, at = threadIdx.x % per;
  const int i = blockIdx.y * per + at;
  const int groups = P / 8, tile = i / 32;   // groups of 8 rows; the warp's tile
  const int r = TC ? (tile / (H / 16) < groups ? tile % groups * 8 + i % 8 : R) : i / (H / 4);
  const int d = TC ? (tile / groups * 4 + i % 32 / 8) * 4 : i % (H / 4) * 4;
  const int64_t at4 = TC ? ((int64_t)(d / 4) * P + r) * 4 : (int64_t)r * H + d;
  const int64_t part = paged_partial_floats(R, H);
  // partial 0 in slot 1 of its CTA, the others in slot 0 of theirs
  const float* const base = a.partials + (int64_t)first * 2 * part;
  float M = -INFINITY, L = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (r < R) {
    for (int p0 = share; p0 < n; p0 += U * shares) {
      float4 y[U];
      float m[U], l[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = p0 + u * shares;
        m[u] = -INFINITY;
        if (p < n) {
          const float* const src = base + (p ? p * 2 : 1) * part;
          y[u] = __ldcg(reinterpret_cast<const float4*>(src + at4));
          m[u] = __ldcg(src + P * H + r);
          l[u] = __ldcg(src + P * H + P + r);
        }
      }
      float mn = M;
#pragma unroll
      for (int u = 0; u < U; ++u) mn = fmaxf(mn, m[u]);
      const float low = mn == -INFINITY ? 0.0f : mn, f0 = fast_exp2(M - low);
      M = mn;
      L *= f0;
      x.x *= f0; x.y *= f0; x.z *= f0; x.w *= f0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (p0 + u * shares < n) {
          const float f = fast_exp2(m[u] - low);
          L += l[u] * f;
          x.x += y[u].x * f;
          x.y += y[u].y * f;
          x.z += y[u].z * f;
          x.w += y[u].w * f;
        }
      }
    }
  }
  if (shares > 1) {
    sx[threadIdx.x] = x;
    sml[threadIdx.x] = make_float2(M, L);
    __syncthreads();
    if (share == 0) {
      for (int w = 1; w < shares; ++w) M = fmaxf(M, sml[w * per + at].x);
      const float low = M == -INFINITY ? 0.0f : M;
      L = 0.0f;
      x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int w = 0; w < shares; ++w) {
        const float2 ml = sml[w * per + at];
        const float4 y = sx[w * per + at];
        const float f = fast_exp2(ml.x - low);
        L += ml.y * f;
        x.x += y.x * f;
        x.y += y.y * f;
        x.z += y.z * f;
        x.w += y.w * f;
      }
    }
  }
  if (share == 0 && r < R)
    put_result((char*)a.o + (int64_t)item * R * H * 2, a.lse + (int64_t)item * R, H, r, d, x, M, L,
               a.v_scale ? a.v_scale[item % a.K] : 1.0f);
}

}  // namespace fa
