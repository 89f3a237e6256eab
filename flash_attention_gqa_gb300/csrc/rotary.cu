// Rotary positions: pairs (a, b) of a head's dims turned by position times frequency,
//
//   a' = (a cos - b sin) scale,   b' = (b cos + a sin) scale,
//
// for queries and keys in one launch, and in the serving form with keys and values going
// straight into the cache's pages.  The gradient is the same with the angle's sign turned.
//
// Angles.  A position is a whole number, so only the fraction of frequency / 2 pi counts: as 64
// fixed-point bits, of which position times bits mod 2^64 is the turn, exact to position * 2^-64
// however far the position is (position * frequency in fp32 is off by 2^-24 of the angle: 0.03 at
// 500000).  Its upper half becomes an angle of fp32 precision in (-pi, pi].
//
// Bound by memory: every value is read and written once (16384 tokens x 40 heads x 128 dims: 54.8 us, 6.1
// TB/s; a decode step of 64 tokens 2.9 us, a launch and a chain of loads).
#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"
#include "rotary.h"

namespace fa {
namespace {

constexpr int kThreads = 256, kPer = 3;

// The fraction of f / (2 pi) in 2^-64 turns, rounded down in size: f = m 2^(e - 150), times
// floor(2^128 / (2 pi)).
__device__ __forceinline__ uint64_t turns_per_step(float f) {
  constexpr uint64_t HI = 0x28be60db9391054aull, LO = 0x7f09d5f47d4d3770ull;
  const uint32_t bits = __float_as_uint(f);
  const int e = max((int)(bits >> 23 & 255), 1);
  const uint64_t m = (bits & 0x7fffff) | ((bits >> 23 & 255) ? 0x800000 : 0);
  const uint64_t p0 = m * LO, h = m * HI;
  const uint64_t p1 = __umul64hi(m, LO) + h, p2 = __umul64hi(m, HI) + (p1 < h ? 1 : 0);
  const int s = 214 - e;   // the product's bits from here on; the 64 lowest of them
  uint64_t r;
  if (s >= 128) r = s >= 192 ? 0 : p2 >> (s - 128);
  else if (s >= 64) r = s == 64 ? p1 : p1 >> (s - 64) | p2 << (128 - s);
  else if (s > 0) r = p0 >> s | p1 << (64 - s);
  else r = p0 << -s;
  return bits >> 31 ? 0 - r : r;
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;   // nearest even, saturating at +-448; NaN stays NaN
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ void widen(uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_bf16x2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// A unit is two 16-byte vectors of a head: dims that turn together, or two vectors side by side
// in the lanes' order.  A CTA takes `tokens` tokens, a thread the same dims of every (kThreads * 16 / H)-th
// head of them in turn.  It loads its first units, then works out the CTA's angles, once for all
// heads, in shared memory in the order in which lanes read them, while the loads are on their way.
template <int TO, int PER>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryArgs a, int tokens) {
  extern __shared__ float4 turn[];   // [token][pairs / 2]: cos, sin of two pairs
  const int shift = a.H == 64 ? 2 : a.H == 128 ? 3 : 4;   // log2 of the units of a head
  const uint32_t upr = 1u << shift, u = threadIdx.x & (upr - 1);
  const uint32_t heads = a.QH + a.KH * (TO == ROTARY_PLAIN ? 1 : 2);
  const uint32_t N = (uint32_t)a.B * a.T, n0 = blockIdx.x * (uint32_t)tokens;
  const uint32_t here = min((uint32_t)tokens, N - n0);
  const uint32_t half = a.pairs / 8;   // vectors of one half of the turned dims
  // vectors u and u + half turn together; behind them those that stay as they are
  const uint32_t ux = a.adjacent || u < half ? u : u + half;
  const uint32_t uy = ux + (a.adjacent ? upr : u < half ? half : upr - half);

  struct Unit {
    uint4 x, y;       // the two vectors
    uint32_t token, b, t, head;
    bool live;
  };
  Unit w[PER];
  // the next unit's token of the CTA and head
  const uint32_t step = kThreads >> shift, step_token = step / heads, step_head = step - step_token * heads;
  uint32_t token = (threadIdx.x >> shift) / heads, head = (threadIdx.x >> shift) - token * heads;
  auto load = [&]() {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      Unit& c = w[j];
      c.live = token < here;
      if (!c.live) continue;
      c.token = token;
      c.head = head;
      const uint32_t n = n0 + token;
      c.b = a.B == 1 ? 0 : n / a.T;
      c.t = n - c.b * a.T;
      const bool isq = head < a.QH, isk = head < a.QH + a.KH;
      const RotaryRows& r = isq ? a.q : isk ? a.k : a.v;
      const uint32_t h = isq ? head : isk ? head - a.QH : head - a.QH - a.KH;
      const char* src = (const char*)r.at + c.b * r.batch + c.t * r.token + h * r.head;
      // (plain loads, not those of constant memory: outputs may be in the inputs' place)
      c.x = __ldcg(reinterpret_cast<const uint4*>(src + ux * 16));
      c.y = __ldcg(reinterpret_cast<const uint4*>(src + uy * 16));
      token += step_token;
      head += step_head;
      if (head >= heads) {
        head -= heads;
        ++token;
      }
    }
  };
  load();

  const uint32_t angles = here * a.pairs;
  for (uint32_t i = threadIdx.x; i < angles; i += kThreads) {
    const uint32_t t = i / a.pairs, p = i - t * a.pairs, n = n0 + t, b = n / a.T;
    int axis = a.axes ? a.axes[p] : 0;
    float f = a.inv_freq[p];
    if ((unsigned)axis >= (unsigned)a.n_axes || !(fabsf(f) < INFINITY)) {
      atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
      if ((unsigned)axis >= (unsigned)a.n_axes) axis = 0;
      if (!(fabsf(f) < INFINITY)) f = 0.0f;
    }
    const int64_t pos = a.positions[axis * a.pos_axis + b * a.pos_batch + (n - b * a.T) * a.pos_token];
    const uint64_t turned = (uint64_t)pos * turns_per_step(f);
    float s, c;
    sincospif((float)(int32_t)(turned >> 32) * 0x1p-31f, &s, &c);
    if (a.inverse) s = -s;
    const uint32_t group = a.adjacent ? p >> 2 : p >> 3, in = a.adjacent ? (p & 3) >> 1 : (p & 7) >> 1;
    const uint32_t groups = a.adjacent ? a.pairs / 4 : half;
    reinterpret_cast<float2*>(turn + t * (a.pairs / 2) + in * groups + group)[p & 1] = make_float2(c, s);
  }
  __syncthreads();

  for (;;) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const Unit& c = w[j];
      if (!c.live) continue;
      int64_t slot = 0;
      if (TO != ROTARY_PLAIN) {
        slot = a.slots[n0 + c.token];
        if (slot < 0) continue;   // padding
      }
      const bool isq = c.head < a.QH, isv = TO != ROTARY_PLAIN && c.head >= a.QH + a.KH;
      const uint32_t h = isq ? c.head : isv ? c.head - a.QH - a.KH : c.head - a.QH;
      float x[8], y[8];
      widen(c.x, x);
      widen(c.y, y);
      if (!isv) {
        const float4* const at = turn + c.token * (a.pairs / 2);
        if (a.adjacent) {
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t at_u = v ? uy : ux;
            if (at_u >= 2 * half) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 cs = at[i * (2 * half) + at_u];
              float(&f)[8] = v ? y : x;
              const float a0 = f[4 * i], b0 = f[4 * i + 1], a1 = f[4 * i + 2], b1 = f[4 * i + 3];
              f[4 * i] = a0 * cs.x - b0 * cs.y;
              f[4 * i + 1] = b0 * cs.x + a0 * cs.y;
              f[4 * i + 2] = a1 * cs.z - b1 * cs.w;
              f[4 * i + 3] = b1 * cs.z + a1 * cs.w;
            }
          }
        } else if (ux < half) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 cs = at[i * half + ux];
            const float a0 = x[2 * i], a1 = x[2 * i + 1];
            x[2 * i] = a0 * cs.x - y[2 * i] * cs.y;
            y[2 * i] = y[2 * i] * cs.x + a0 * cs.y;
            x[2 * i + 1] = a1 * cs.z - y[2 * i + 1] * cs.w;
            y[2 * i + 1] = y[2 * i + 1] * cs.z + a1 * cs.w;
          }
        }
        if (isq) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] *= a.q_scale;
            y[i] *= a.q_scale;
          }
        }
      }
      auto pack = [](const float (&f)[8]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
      };
      if (isq || TO == ROTARY_PLAIN) {
        const RotaryRows& r = isq ? a.q_out : a.k_out;
        char* const dst = (char*)r.at + c.b * r.batch + c.t * r.token + h * r.head;
        *reinterpret_cast<uint4*>(dst + ux * 16) = pack(x);
        *reinterpret_cast<uint4*>(dst + uy * 16) = pack(y);
        continue;
      }
      const int64_t page = slot >> a.lay.page_shift, in = slot & ((1 << a.lay.page_shift) - 1);
      if (page >= a.lay.n_pages) {
        atomicOr(a.err, (uint32_t)DEV_BAD_VALUE);
        continue;
      }
      char* const dst = (char*)(isv ? a.v_cache : a.k_cache) + page * a.lay.page + h * a.lay.head + in * a.lay.token;
      if (TO == ROTARY_BF16) {
        *reinterpret_cast<uint4*>(dst + ux * 16) = isv ? c.x : pack(x);
        *reinterpret_cast<uint4*>(dst + uy * 16) = isv ? c.y : pack(y);
      } else {
        // From fp32, by the scale's reciprocal: off by 2^-23 (its rounding and the product's) before the
        // rounding to e4m3's 2^-4 (a division per value takes twice the time of everything else).  `up` keeps
        // the reciprocal a normal number: 0 / 1e-39 is 0, and 0 times an infinite reciprocal is none.
        const float* const scales = isv ? a.v_scale : a.k_scale;
        const float scale = scales ? scales[h] : 1.0f;
        const float up = fabsf(scale) < 0x1p-64f ? 0x1p64f : fabsf(scale) > 0x1p64f ? 0x1p-64f : 1.0f;
        const float s = 1.0f / (scale * up);
        auto squeeze = [s, up](const float (&f)[8]) {
          return make_uint2(to_e4m3x4(f[0] * s * up, f[1] * s * up, f[2] * s * up, f[3] * s * up),
                            to_e4m3x4(f[4] * s * up, f[5] * s * up, f[6] * s * up, f[7] * s * up));
        };
        *reinterpret_cast<uint2*>(dst + ux * 8) = squeeze(x);
        *reinterpret_cast<uint2*>(dst + uy * 8) = squeeze(y);
      }
    }
    if (token >= here) break;
    load();
  }
}

template <int TO>
cudaError_t launch(const RotaryArgs& a, int sm_count, cudaStream_t st) {
  const int64_t N = (int64_t)a.B * a.T;
  const int64_t units = (int64_t)(a.QH + a.KH * (TO == ROTARY_PLAIN ? 1 : 2)) * (a.H / 16), all = N * units;
  // Three units of a thread in flight and two rounds of them, once that fills the GPU (4 CTAs on each of
  // its SMs); one unit below.  (16384 tokens x 40 heads x 128 dims: 61 us with four and one round, 54 with
  // two and two, 54.8 so; 8000 tokens x 80 heads into an e4m3 cache: 78, 64 and 55.)
  const bool many = all >= (int64_t)kPer * kThreads * 4 * sm_count;
  int64_t tokens = (many ? 2 * kPer : 1) * kThreads / units;
  if (tokens > 4096 / a.pairs) tokens = 4096 / a.pairs;   // 32 KB of angles
  if (tokens < 1) tokens = 1;
  auto* const kernel = many ? rotary_kernel<TO, kPer> : rotary_kernel<TO, 1>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((N + tokens - 1) / tokens));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)tokens * a.pairs * sizeof(float2);
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, a, (int)tokens);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, RotaryTo to, int sm_count, cudaStream_t st) {
  switch (to) {
    case ROTARY_PLAIN: return launch<ROTARY_PLAIN>(a, sm_count, st);
    case ROTARY_BF16: return launch<ROTARY_BF16>(a, sm_count, st);
    default: return launch<ROTARY_E4M3>(a, sm_count, st);
  }
}

}  // namespace fa
