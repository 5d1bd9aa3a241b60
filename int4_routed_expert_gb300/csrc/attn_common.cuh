// What the attention kernels share: the keys that a tile of rows sees, the
// conversions, the finish of a row.
#pragma once

#include <algorithm>

#include "attn_internal.cuh"

namespace moe {

// Weights are taken relative to 2^-kLift of the row's reference, which moves when it would grow by more than
// 2^kRescale: f16 weights lie below 2^15 and keep all their bits down to 2^-24 of the largest.
constexpr float kLift = 10.f, kRescale = 5.f;

// The tiles of TILE keys that some row of positions p0 .. p1 sees: n_a tiles
// from key 0 (the sinks), then those from tile t_b to key hi.
struct KeyTiles {
  int lo, hi;  // seen: [lo, hi) and the sinks below lo
  int n_a, t_b, n_t;
  int tile;
  int group, whole;  // Part::kBoth: of the prefix, whose are the first n_a tiles or the tokens below `whole`
  __device__ __forceinline__ int base(int t) const { return (t < n_a ? t : t_b + t - n_a) * tile; }
};

template <int TILE>
__device__ __forceinline__ KeyTiles key_tiles(const AttnArgs& a, int L, int p0, int p1) {
  KeyTiles k;
  k.tile = TILE;
  k.hi = a.causal ? max(p1 + 1, 0) : L;
  k.lo = a.window ? max(p0 - a.window + 1, 0) : 0;
  k.n_a = (min(a.sinks, k.hi) + TILE - 1) / TILE;
  k.t_b = k.lo / TILE;
  if (k.t_b <= k.n_a) k.n_a = k.t_b = 0;
  k.n_t = k.n_a + max((k.hi + TILE - 1) / TILE - k.t_b, 0);
  return k;
}

// An upper bound of n_t over the rows of a batch, for tiles of `rows` rows.
inline int64_t max_key_tiles(const KvView& c, const AttnArgs& a, int rows, int tile) {
  int64_t keys = c.max_kv;
  if (a.window)
    keys = std::min<int64_t>(keys, static_cast<int64_t>(a.window) + rows + a.sinks + 3 * tile);
  return std::max<int64_t>((keys + tile - 1) / tile, 1);
}

// The keys that one row sees: up to hi, from lo or below the sinks.
struct RowSees {
  int lo, hi, sinks;
  __device__ __forceinline__ bool operator()(int tok) const {
    return tok <= hi && (tok >= lo || tok < sinks);
  }
  // The same for keys tok .. tok + 31, a bit each.
  __device__ __forceinline__ uint32_t bits(int tok) const {
    return below(hi + 1 - tok) & (~below(lo - tok) | below(sinks - tok));
  }
  static __device__ __forceinline__ uint32_t below(int n) {  // the lowest n bits
    return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1u;
  }
};
__device__ __forceinline__ RowSees row_sees(const AttnArgs& a, int L, int p, bool live, int begin = 0) {
  RowSees r;
  r.hi = !live ? -1 : a.causal ? p : L - 1;
  r.lo = live && a.window ? p - a.window + 1 : begin;
  r.sinks = a.sinks;
  return r;
}

// Two e4m3 codes (low half word) as f16x2, exactly.
__device__ __forceinline__ void codes_to_half(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// 2^x, off by 2^-22 of itself at most, and 0 below 2^-126: a weight goes on with f16's 11 bits, and one of
// 2^-126 is 2^-136 of the row's reference.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^(TOP - floor(log2 amax)), the power of two that brings a query row to
// [2^TOP, 2^(TOP + 1)); rows below 2^-87 keep that of 2^-87.
template <int TOP>
__device__ __forceinline__ float row_factor(float amax) {
  const int e = max(static_cast<int>(__float_as_uint(amax) >> 23), 40);
  return __uint_as_float(static_cast<uint32_t>(min(127 + TOP + 127 - e, 254)) << 23);
}

// 1 / f of a power of two in [2^-126, 2^126]
__device__ __forceinline__ float inverse(float f) { return __uint_as_float((254u << 23) - __float_as_uint(f)); }

// Row `row` of the output (and of lse): sums over sum of weights, both
// relative to reference mm - kLift.  A row that saw nothing is 0.
template <int D>
__device__ __forceinline__ void finish_row(const AttnArgs& a, size_t row, int d4, const float4& v,
                                           float mm, float ll) {
  const bool any = ll > 0.f || ll != ll;
  const float f = any ? 1.f / ll : 0.f;
  const __nv_bfloat162 x0 = __floats2bfloat162_rn(v.x * f, v.y * f);
  const __nv_bfloat162 x1 = __floats2bfloat162_rn(v.z * f, v.w * f);
  *reinterpret_cast<uint2*>(a.out + row * D + 4 * d4) = make_uint2(
      *reinterpret_cast<const uint32_t*>(&x0), *reinterpret_cast<const uint32_t*>(&x1));
  if (a.lse && d4 == 0) a.lse[row] = any ? (mm - kLift + log2f(ll)) * 0.693147180559945f : -INFINITY;
}

// Joins a row's `n` partial results, `stride` rows apart, in their order: eight
// at a time, their loads under way together.
template <int D>
__device__ __forceinline__ void join_row(const AttnArgs& a, const AttnWs& ws, size_t first, int stride,
                                         int n, size_t row, int d4) {
  constexpr int kBatch = 8;
  float mm = -INFINITY, ll = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += kBatch) {
    float2 x[kBatch];
    float4 y[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const size_t at = first + static_cast<size_t>(min(s0 + i, n - 1)) * stride;
      x[i] = __ldcg(&ws.ml[at]);
      y[i] = __ldcg(reinterpret_cast<const float4*>(ws.o + at * D + 4 * d4));
    }
    float top = mm;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, x[i].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float back = ex2(mm - ref);
    mm = top;
    ll *= back;
    v.x *= back, v.y *= back, v.z *= back, v.w *= back;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i >= n) break;
      const float f = ex2(x[i].x - ref);
      ll = fmaf(x[i].y, f, ll);
      v.x = fmaf(y[i].x, f, v.x), v.y = fmaf(y[i].y, f, v.y);
      v.z = fmaf(y[i].z, f, v.z), v.w = fmaf(y[i].w, f, v.w);
    }
  }
  finish_row<D>(a, row, d4, v, mm, ll);
}

}  // namespace moe
