// Attention of sequences that share a prefix (moe_kv_attend_shared).
//
// With O_p, W_p the softmax's sums over the prefix's tokens and O_o, W_o those over a row's
// own ones, both relative to one reference, out = (O_p + O_o) / (W_p + W_o).  A group's rows
// see all of its prefix, whichever sequence they are of, so for the prefix the group is one
// sequence without a causal mask: its keys are read once for all of its rows, and the
// products have them all as one dimension.  The rows' own tokens are the ordinary batch, from
// the prefix's end on.  Both are launches of the two attention kernels, by their rows, that
// leave unnormalised sums in fp32, a reference and a weight sum for each split of the keys;
// a last kernel joins them, own splits first, in their order.
// The three launches overlap: the second does not need the first and begins as its
// CTAs leave SMs, the third is in place when they end.
//
// Short prefixes and few keys take one launch instead, in which each sequence goes over its
// prefix and its own tokens itself (Part::kBoth); the workspace is then the handle's, as for
// attention without prefixes.  Whichever of the two is to take less, the host's 7 us for two
// launches more counted (240 calls of 1 to 64 sequences of up to 1742 new tokens, prefixes of
// 20 to 125000, captured: 0.92 of the three launches' time, one by one 0.40 to 1.42 of it; a
// call of 3 tokens that is not captured: 14.7 us instead of 22.3).  24 tokens of 9 groups,
// prefixes of 133, 96 / 8 heads of 64: 13.0 us in one launch, 31.7 us in three; 10 prompts'
// last 536 tokens on 822, 24 / 8 heads: 88.8 and 155 us; 40 tokens of 3 groups on 2384, 8 / 8
// heads: 54.6 and 26.4 us.
#include <cmath>

#include "attn_tc.cuh"

namespace moe {
namespace {

constexpr int kJoinThreads = 256;

// One of the two launches: which kernel, its plan and its partial results.
struct Side {
  Plan pl;
  bool few;
  int rows;    // of a row tile
  int parts;   // results of a split: two where both M tiles have the same rows
  int ctas;    // not 0: the prefixes' work is dealt out to so many CTAs, pl.splits parts a row tile at most
  size_t cap;  // rows of results
};

// What a CTA of either kernel costs on a busy SM, in microseconds: a tile of keys, and its
// beginning and end; and how many share the SM.
struct CtaCost {
  double tile, start;
  int per_sm;
};
CtaCost cost_of(int64_t rows) {
  if (rows <= 16) return {1.9, 5., 2};
  if (rows <= 32) return {3.3, 6., 2};
  return {1.75, 10., 1};
}

// The kernel for a side's rows, and its row tiles: a launch has to count on row_tiles of each
// sequence, but `live` of all sequences and kv heads have rows, or about so many.
Side side_of(const KvView& c, int G, double& live) {
  const int64_t rows = static_cast<int64_t>(c.max_q) * G, all = static_cast<int64_t>(c.n_tokens) * G;
  Side x;
  x.few = rows <= 32;  // as moe_kv_attend chooses
  x.rows = x.few ? (rows <= 16 ? 16 : 32) : 256;
  x.parts = !x.few && rows <= 128 ? 2 : 1;
  x.ctas = 0;
  x.pl.row_tiles = static_cast<int>((rows + x.rows - 1) / x.rows);
  // (the sequences' rows add up to the call's, and half a tile of each is empty)
  live = std::min(static_cast<double>(x.pl.row_tiles) * c.n_seqs, static_cast<double>(all) / x.rows + 0.5 * c.n_seqs + 0.5) *
         c.hkv;
  return x;
}

void set_splits(Side& x, const KvView& c, int G, int64_t tiles, int64_t splits) {
  x.pl.tiles_per_split = static_cast<int>((tiles + splits - 1) / splits);
  x.pl.splits = static_cast<int>((tiles + x.pl.tiles_per_split - 1) / x.pl.tiles_per_split);
  x.cap = static_cast<size_t>(x.parts) * x.pl.splits * c.n_tokens * c.hkv * G;
}

// The prefixes as a batch: a group is a sequence.
KvView prefix_view(const KvView& c, const Share& sh) {
  KvView p = c;
  p.n_seqs = sh.n_groups;
  p.max_q = sh.max_tokens;
  p.max_kv = sh.max_len;
  p.table = sh.table;
  p.table_stride = sh.table_stride;
  return p;
}

struct Sides {
  KvView prefix;
  Side own, shared;
  bool wide;  // few rows: the join has a CTA for each
  bool one;   // neither: each sequence reads all of its keys, in one launch
};
// What one launch over all keys takes (Part::kBoth).
double one_launch_time(const KvView& c, int G, const Side& x, double live, int n_sm) {
  const int64_t tiles = (static_cast<int64_t>(c.max_kv) + kKeys - 1) / kKeys + 1;
  const int64_t base = static_cast<int64_t>(x.pl.row_tiles) * c.n_seqs * c.hkv;
  const CtaCost cost = cost_of(static_cast<int64_t>(c.max_q) * G);
  int64_t n = best_splits(base, n_sm, tiles, 256, c.n_seqs > 1, x.few ? Costs{2, 3., 0.25} : Costs{1, 6., 1. / 32});
  const int64_t per = (tiles + n - 1) / n;
  n = (tiles + per - 1) / per;
  const double cta = cost.tile * static_cast<double>(per) + cost.start;
  double join = 0;
  if (x.few && n > 1) join = 1.5 + 0.075 * cost.tile * static_cast<double>(n);
  if (!x.few && x.parts * n > 1)
    join = 2.5 + static_cast<double>(c.n_tokens) * c.hkv * G * static_cast<double>(x.parts * n) * c.D * 8 / 5e6;
  const double ctas = std::max(live * static_cast<double>(n), 1.);
  return static_cast<double>(static_cast<int64_t>((ctas - 1) / (n_sm * cost.per_sm)) + 1) * cta + join;
}
// How the keys are cut.  The launch over own tokens fills the SMs that the one over the
// prefixes leaves, so that one's CTAs go by the time of both: that of the longest ones, or
// all CTAs' time over the SMs, whichever is longer, and what a split more costs the join.
// The splits are alike, or (more than 128 rows, up to 32 groups) the row tiles' keys are
// dealt out evenly to CTAs that go from one to the next, which costs some at each change.
// (64 tokens on a prefix of 16384, 64 / 8 heads: 71 us in 5 splits, 87 us in 9, where the
// prefix alone is fastest, 79 us dealt out.  37 x 4 tokens on three prefixes of up to 66001,
// 48 / 4 heads: 265 us in 4 splits, 338 us in 6, whose second round of CTAs is a quarter
// full, 224 us dealt out.  5085 tokens of 12 questions on 24001, 32 / 2 heads of 64: 1546 us
// in 2 splits, 1437 us dealt out.)
Sides sides_of(const KvView& c, const Share& sh, int G, int n_sm) {
  constexpr int64_t kMost = 1 << 20;  // rows of results a side, where one split has fewer
  const int64_t rows = static_cast<int64_t>(c.n_tokens) * c.hkv * G;
  Sides s;
  s.prefix = prefix_view(c, sh);
  double own_live, live;
  s.own = side_of(c, G, own_live);
  s.shared = side_of(s.prefix, G, live);
  // The host knows no bound of a sequence's own tokens; where prefixes are alike it is this.  A
  // sequence that has many more gets no more splits (8 single tokens on a prefix of 65961, 64 / 8
  // heads: 54 us; with a ninth of 66001 own tokens 435 us, and 157 us as attention of each).
  const int64_t own_tiles = (std::max(c.max_kv - sh.max_len, 1) + kKeys - 1) / kKeys;
  const int64_t tiles = (sh.max_len + kKeys - 1) / kKeys;
  const CtaCost own_cost = cost_of(static_cast<int64_t>(c.max_q) * G), cost = cost_of(static_cast<int64_t>(s.prefix.max_q) * G);
  auto limit = [&](int64_t n, const Side& x) {
    return std::max<int64_t>(std::min({n, static_cast<int64_t>(256), kMost / (x.parts * rows)}), 1);
  };
  const int64_t own_splits =
      best_splits(static_cast<int64_t>(own_live + 0.5), n_sm, own_tiles, limit(own_tiles, s.own), c.n_seqs > 1,
                  s.own.few ? Costs{2, 3., 0.25} : Costs{1, 6., 1. / 32});
  set_splits(s.own, c, G, own_tiles, own_splits);
  // (sequences' lengths spread between none and the bound)
  const double own_time = own_live * (0.6 * static_cast<double>(own_tiles) * own_cost.tile + own_cost.start * s.own.pl.splits) /
                          own_cost.per_sm;
  // a split's sums written and read, at 5 TB/s, and read eight at a time, by one or all of a CTA's rows
  s.wide = rows <= 16 * n_sm;
  const double join = static_cast<double>(rows) * s.shared.parts * c.D * 8 / 5e6 + s.shared.parts * (s.wide ? 0.8 / 64 : 0.1);
  double least = 1e300;
  int64_t best = 1;
  for (int64_t k = 1, end = limit(tiles, s.shared); k <= end; ++k) {
    const double cta = cost.tile * static_cast<double>((tiles + k - 1) / k) + cost.start;
    const double ctas = std::max(live * static_cast<double>(k), 1.);
    const double rounds = static_cast<double>(static_cast<int64_t>((ctas - 1) / (n_sm * cost.per_sm)) + 1);
    const double time = std::max(rounds * cta, (ctas * cta / cost.per_sm + own_time) / n_sm) + join * static_cast<double>(k);
    if (time < least) least = time, best = k;
  }
  set_splits(s.shared, c, G, tiles, best);
  // The three launches as a whole: the longer of the two, what the own results cost the join,
  // and two launches more (4 us where they are captured, 7 us of the host's where not).
  const double one = one_launch_time(c, G, s.own, own_live, n_sm);
  auto decide = [&](double prefix) {
    const double own = own_cost.tile * s.own.pl.tiles_per_split + own_cost.start;
    s.one = one < std::max(prefix, own) + static_cast<double>(s.own.cap) * c.D * 8 / 5e6 + 7.;
    return s;
  };
  // (units are counted in 32 bits: room for those of groups whose offsets do not ascend, which are of the same rows)
  if (s.shared.few || s.shared.parts > 1 || sh.n_groups > 32 ||
      static_cast<double>(s.shared.pl.row_tiles) * sh.n_groups * c.hkv * static_cast<double>(tiles) > 1e9)
    return decide(least);
  const double units = live * static_cast<double>(tiles);
  int64_t ctas = 0;
  // (splits that are alike are so of groups that are not)
  if (sh.n_groups > 1) least += 0.15 * cost.tile * static_cast<double>(s.shared.pl.tiles_per_split);
  for (int64_t k = 1; k <= n_sm; ++k) {
    const double per = static_cast<double>(static_cast<int64_t>(units / static_cast<double>(k)) + 1);
    // (the deal itself, and half a beginning and end for each row tile but the first)
    const double cta = cost.tile * per + cost.start + 1.5 + 0.5 * cost.start * (1 + std::floor(per / static_cast<double>(tiles)));
    const double time = std::max(cta, (cta * static_cast<double>(k) + own_time) / n_sm) + join * (static_cast<double>(k) / live + 1);
    if (time < least) least = time, ctas = k;
  }
  if (ctas) {
    s.shared.ctas = static_cast<int>(ctas);
    // parts of a row tile: its keys over a CTA's, and one more where it begins within a CTA's;
    // half as much again, as the rows and lengths may be fewer than the host knows
    const int64_t parts = static_cast<int64_t>(1.5 * static_cast<double>(ctas) / live) + 3;
    s.shared.pl.splits = static_cast<int>(std::max<int64_t>(std::min(parts, kMost / rows), 2));
    s.shared.cap = static_cast<size_t>(s.shared.pl.splits) * rows;
  }
  return decide(least);
}

size_t align(size_t x) { return (x + 255) / 256 * 256; }
size_t side_bytes(const Side& x, int D) { return align(x.cap * D * 4) + align(x.cap * 8); }

// (one launch keeps its partial results where attention without prefixes does)
size_t bytes_of(const Sides& x, int D) { return x.one ? 0 : side_bytes(x.own, D) + side_bytes(x.shared, D); }

AttnWs side_ws(const Side& x, int D, char* base) {
  return AttnWs{reinterpret_cast<float*>(base), reinterpret_cast<float2*>(base + align(x.cap * D * 4)), nullptr, x.cap};
}

// What a row's partial results add up to, so far.
struct RowSum {
  float m, l;  // reference, sum of weights
  float4 v;
  // Takes on kBatch results at once, in their order; those from n on are none.
  template <int N>
  __device__ __forceinline__ void add(const float2 (&x)[N], const float4 (&y)[N], int n) {
    float top = m;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, x[i].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float back = ex2(m - ref);
    m = top;
    l *= back;
    v.x *= back, v.y *= back, v.z *= back, v.w *= back;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= n) break;
      const float f = ex2(x[i].x - ref);
      l = fmaf(x[i].y, f, l);
      v.x = fmaf(y[i].x, f, v.x), v.y = fmaf(y[i].y, f, v.y);
      v.z = fmaf(y[i].z, f, v.z), v.w = fmaf(y[i].w, f, v.w);
    }
  }
};

// A CTA joins a slice of the heads of one token, D / 4 threads a row.  WIDE: the whole CTA
// a row, D / 4 threads every eighth (heads of 64: sixteenth) of its results, whose sums are
// joined once more: for calls of few rows, whose keys are cut into many splits.  DEALT: the
// prefixes' results are of dealt out work.
template <int D, bool WIDE, bool DEALT>
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const KvView c, const AttnArgs a, const Share sh, const Side own, const Side shared, const AttnWs own_ws,
                const AttnWs shared_ws, int slices) {
  constexpr int kPer = kJoinThreads / (D / 4), kBatch = 8;
  const int t = blockIdx.x / slices, slice = blockIdx.x % slices;
  bool odd = false, covered;
  Seq q, g{0, 0, 0};
  InGroup in;
  for (int b = last_not_above(c.cu_q, c.n_seqs, t, odd), other = -1;; b = other) {
    in = group_of(sh, b);
    covered = load_seq(c, b, q) && t >= q.q0 && t < q.q0 + q.n;
    if (covered || other >= 0 || (other = range_of(c.cu_q, c.n_seqs, t, c.n_tokens, b, odd)) < 0) break;
  }
  const int begin = covered ? own_begin(sh, q, in) : 0;
  int n_shared = 0, per, before = 0, g_tiles = 0, g_per = 1;
  if constexpr (DEALT) {
    const Dealt d = deal_out(c, a, sh, shared.ctas, shared.pl.splits);
    const int lane_of = max(in.g, 0);
    before = __shfl_sync(0xffffffffu, d.before, lane_of);
    g_tiles = __shfl_sync(0xffffffffu, d.n_t, lane_of);
    g.q0 = __shfl_sync(0xffffffffu, d.q.q0, lane_of);
    g_per = d.per;
    if (!covered || in.g < 0) g_tiles = 0;
  } else if (covered && in.g >= 0 && load_group(c, sh, in.g, g)) {
    split_tiles(shared.pl, (g.L + kKeys - 1) / kKeys, n_shared, per);
    n_shared *= shared.parts;
  }
  pdl_wait();
  if (!covered) return;
  const int d4 = threadIdx.x % (D / 4), grp = threadIdx.x / (D / 4);
  const int h0 = static_cast<int>(static_cast<int64_t>(slice) * a.hq / slices);
  const int h1 = static_cast<int>((slice + static_cast<int64_t>(1)) * a.hq / slices);
  for (int h = h0 + (WIDE ? 0 : grp); h < h1; h += WIDE ? 1 : kPer) {
    const int hk = h / a.G, r = (t - q.q0) * a.G + h - hk * a.G;  // row of the sequence
    const int64_t tile_end = (static_cast<int64_t>(r) / own.rows + 1) * own.rows;
    const int last = static_cast<int>(min(static_cast<int64_t>(q.n) * a.G, tile_end) - 1) / a.G;
    int n_own;
    split_tiles(own.pl, own_tiles(a, q.L, begin, q.L - q.n + last), n_own, per);
    n_own *= own.parts;
    if (DEALT && g_tiles > 0) {  // the CTAs that its row tile's units went to
      const int unit = before + (((t - g.q0) * a.G + h - hk * a.G) / 256 * c.hkv + hk) * g_tiles;
      n_shared = (unit + g_tiles - 1) / g_per - unit / g_per + 1;
    }
    const size_t step = static_cast<size_t>(c.hkv) * c.n_tokens * a.G;
    const size_t first = (static_cast<size_t>(hk) * c.n_tokens + t) * a.G + h - hk * a.G;
    const int all = n_own + n_shared, mine = WIDE ? max((all - grp + kPer - 1) / kPer, 0) : all;
    RowSum sum{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int s0 = 0; s0 < mine; s0 += kBatch) {
      float2 x[kBatch];
      float4 y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int k = min(s0 + i, mine - 1), s = WIDE ? k * kPer + grp : k;
        const AttnWs& ws = s < n_own ? own_ws : shared_ws;
        const size_t at = first + (s < n_own ? s : s - n_own) * step;
        x[i] = __ldcg(&ws.ml[at]);
        y[i] = __ldcg(reinterpret_cast<const float4*>(ws.o + at * D + 4 * d4));
      }
      sum.add(x, y, mine - s0);
    }
    if constexpr (WIDE) {
      __shared__ float2 ml[kPer];
      __shared__ float4 part[kPer][D / 4];
      __syncthreads();  // (of the row before)
      if (d4 == 0) ml[grp] = make_float2(sum.m, sum.l);
      part[grp][d4] = sum.v;
      __syncthreads();
      if (grp > 0) continue;
      float2 x[kPer];
      float4 y[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = ml[i], y[i] = part[i][d4];
      sum = RowSum{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      sum.add(x, y, kPer);
    }
    finish_row<D>(a, static_cast<size_t>(t) * a.hq + h, d4, sum.v, sum.m, sum.l);
  }
}

}  // namespace

size_t attn_shared_workspace(const KvView& c, const Share& sh, int G, int n_sm) {
  return bytes_of(sides_of(c, sh, G, n_sm), c.D);
}

cudaError_t attn_shared_launch(const KvView& c, const AttnArgs& a, const Share& sh, const AttnWs& handle_ws, void* workspace,
                               size_t have, size_t* need, const KvMaps& maps, int n_sm, cudaStream_t s) {
  const Sides x = sides_of(c, sh, a.G, n_sm);
  *need = bytes_of(x, c.D);
  if (have < *need) return cudaErrorInvalidValue;
  if (x.one)
    return (x.own.few ? attn_few_both_launch : attn_tiles_both_launch)(c, a, handle_ws, sh, maps, n_sm, s);
  char* base = static_cast<char*>(workspace);
  const AttnWs own = side_ws(x.own, c.D, base), shared = side_ws(x.shared, c.D, base + side_bytes(x.own, c.D));
  AttnArgs all = a;
  all.causal = 0;
  cudaError_t e = x.shared.few
                      ? attn_few_part_launch(x.prefix, all, shared, x.shared.pl, sh, true, maps, s)
                      : attn_tiles_part_launch(x.prefix, all, shared, x.shared.pl, sh, true, x.shared.ctas, maps, s);
  if (e != cudaSuccess) return e;
  e = x.own.few ? attn_few_part_launch(c, a, own, x.own.pl, sh, false, maps, s)
                : attn_tiles_part_launch(c, a, own, x.own.pl, sh, false, 0, maps, s);
  if (e != cudaSuccess) return e;
  // a CTA for a pass of its threads over heads, while that is not more than the SMs hold at once
  const int64_t per = x.wide ? 1 : kJoinThreads / (c.D / 4), passes = (a.hq + per - 1) / per;
  const int64_t slices = x.wide ? passes : std::max<int64_t>(1, std::min<int64_t>(passes, 8LL * n_sm / c.n_tokens));
  const bool dealt = x.shared.ctas != 0;
  auto join = c.D == 128 ? (x.wide ? (dealt ? join_kernel<128, true, true> : join_kernel<128, true, false>)
                                   : (dealt ? join_kernel<128, false, true> : join_kernel<128, false, false>))
                         : (x.wide ? (dealt ? join_kernel<64, true, true> : join_kernel<64, true, false>)
                                   : (dealt ? join_kernel<64, false, true> : join_kernel<64, false, false>));
  return launch_kernel(join, c.n_tokens * slices, kJoinThreads, 0, s, true, c, a, sh, x.own, x.shared, own, shared,
                       static_cast<int>(slices));
}

}  // namespace moe
