// Attention over the 8-bit cache for few rows (single tokens, verify batches):
// split over the keys, on mma.sync, each warp streaming its own keys.
//
// Mathematics.  Row r (a query head of a new token) sees keys j with logits
// s_j = scale * q . k_j.  With the page's value scale v_j folded into the
// exponent, w_j = 2^(s_j log2 e + log2 v_j - m), the output is
//   o = sum_j w_j c_j / sum_j (w_j / v_j),   c_j the value's e4m3 code,
// so one running reference m serves both sums, the weights that the tensor
// cores take (16 bits) are relative to the largest contribution, and block
// scales cost one multiply-add a logit that the softmax needs anyway.
//
// Operands.  Codes become f16 exactly (two a conversion).  A query row is
// brought to [2^14, 2^15) by a power of two, so its bf16 values are exact in
// f16 down to 2^-28 of the row's largest.  Weights are rounded to f16
// (2^-12 relative); logits, sums and references are fp32.
//
// Layout.  A warp takes tiles of 32 keys: 16-byte cp.async copies into its own
// ring of stages, chunks swizzled so that ldmatrix is free of conflicts.  Both
// products use the freedom to permute the contracted index: for q.k the four
// bytes that ldmatrix gives a thread are the dims 4i .. 4i+3 and the query
// fragment is loaded in that order; for w.v the transposed 16-bit ldmatrix
// gives two dims of two keys, one byte permute pairs the keys, and the weights
// leave the softmax in the order the product needs.  No barrier inside the
// loop: the warps meet once, at the end.
//
// Bound by memory: 2 D bytes a key and kv head, 16 rows share them.
#include <climits>

#include "attn_common.cuh"
#include "smem_opt_in.cuh"
#include "stream_common.cuh"

namespace moe {
namespace {

constexpr int kRows = 16;    // rows of a CTA (one m16 fragment)
constexpr int kTile = 32;    // keys of a warp's tile
constexpr int kWarps = 4;
constexpr int kStages = 3;

template <int D>
struct Lay {
  static constexpr int kTileBytes = kTile * D;              // keys or values
  static constexpr int kStageBytes = 2 * kTileBytes + 128;  // + scales of the tile's pages
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kSmem = kWarps * kWarpBytes + kWarps * kRows * 8;
  static_assert(kRows * D * 4 <= kWarpBytes, "the merge reuses the ring");
};

// Byte offset of 16-byte chunk c of row r in a tile: rows of D bytes packed in
// 128-byte lines, chunks xor-swizzled by the line.
template <int D>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  const int line = r >> 1;
  return line * 128 + (((((r & 1) << 2) | c) ^ (line & 7)) << 4);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct Plan {
  int row_tiles, splits, tiles_per_split;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
    attn_rows_kernel(const KvView c, const AttnArgs a, const AttnWs ws, const Plan pl) {
  extern __shared__ __align__(128) char smem[];
  constexpr int C = D / 16;  // 16-dim chunks of a row
  using L_ = Lay<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, i4 = lane & 3;
  int idx = blockIdx.x;
  const int rt = idx % pl.row_tiles;
  idx /= pl.row_tiles;
  const int hk = idx % c.hkv;
  idx /= c.hkv;
  const int b = idx % c.n_seqs, split = idx / c.n_seqs;
  Seq q;
  if (!load_seq(c, b, q)) return;
  const int R = q.n * a.G, r0 = rt * kRows;
  if (r0 >= R) return;
  const int r1 = min(R, r0 + kRows);
  const int base_p = q.L - q.n;
  const int p0 = base_p + r0 / a.G, p1 = base_p + (r1 - 1) / a.G;
  const KeyTiles kt_ = key_tiles<kTile>(a, q.L, p0, p1);
  const int hi = kt_.hi, lo = kt_.lo, n_t = kt_.n_t;
  const int n_split = max((n_t + pl.tiles_per_split - 1) / pl.tiles_per_split, 1);
  if (split >= n_split) return;
  const int tile_end = min(n_t, (split + 1) * pl.tiles_per_split);
  const int tile0 = split * pl.tiles_per_split + warp;

  char* ring = smem + warp * L_::kWarpBytes;
  const uint32_t ring_u = smem_u32(ring);
  auto tile_base = [&](int t) { return kt_.base(t); };
  // table entries of the next tile to load, read one tile ahead
  int raw0 = 0, raw1 = 0;
  bool bad = false;
  auto next_pages = [&](int t) {
    if (t >= tile_end) return;
    const int base = tile_base(t);
    raw0 = raw_page(c, b, base >> c.page_log2);
    raw1 = c.page < kTile && base + 16 < hi ? raw_page(c, b, (base + 16) >> c.page_log2) : raw0;
  };
  auto issue = [&](int t, int stage) {
    if (t < tile_end) {
      const int base = tile_base(t);
      const int pg0 = checked_page(c, raw0, bad), pg1 = checked_page(c, raw1, bad);
      const uint32_t dst = ring_u + stage * L_::kStageBytes;
      constexpr int kPer = 32 / C;  // rows a pass of the warp
      const int c16 = lane % C;
#pragma unroll
      for (int p = 0; p < kTile / kPer; ++p) {
        const int r = p * kPer + lane / C;
        const int pg = r < 16 ? pg0 : pg1;
        const int tok = base + r;
        // what no row sees is zero: a NaN there would reach the rows through 0 * NaN
        const bool ok = tok < hi && (tok >= lo || tok < a.sinks) && pg >= 0;
        const size_t off =
            ok ? ((static_cast<size_t>(pg) * c.hkv + hk) * c.page + (tok & (c.page - 1))) * D + c16 * 16
               : 0;
        const uint32_t d = dst + tile_off<D>(r, c16);
        cp16(d, c.k + off, ok ? 16 : 0);
        cp16(d + L_::kTileBytes, c.v + off, ok ? 16 : 0);
      }
      if (lane < 4) {
        const int pg = (lane & 1) ? pg1 : pg0;
        const float* src = (lane & 2) ? c.v_scale : c.k_scale;
        cp4(dst + 2 * L_::kTileBytes + lane * 4,
            src + (pg >= 0 ? static_cast<size_t>(pg) * c.hkv + hk : 0), pg >= 0 ? 4 : 0);
      }
      next_pages(t + kWarps);
    }
    cp_commit();
  };

  next_pages(tile0);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(tile0 + s * kWarps, s);

  // the query fragments of rows g and g + 8: chunk x holds dims 16 x + 4 i4 ..
  uint32_t qa[C][4];
  float lscale[2];  // logit scale of the row, its power of two undone
  RowSees see[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + g + 8 * h;
    const bool ok = r < r1;
    const int tok = ok ? r / a.G : 0;
    see[h] = row_sees(a, q.L, base_p + tok, ok);
    const __nv_bfloat16* src = a.q + (static_cast<int64_t>(q.q0) + tok) * a.q_stride +
                               (static_cast<int64_t>(hk) * a.G + (ok ? r - tok * a.G : 0)) * D + 4 * i4;
    uint2 raw[C];
    float amax = 0.f;
#pragma unroll
    for (int x = 0; x < C; ++x) {
      raw[x] = ok ? __ldg(reinterpret_cast<const uint2*>(src + 16 * x)) : make_uint2(0, 0);
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[x].x << 16)),
                               fabsf(__uint_as_float(raw[x].x & 0xffff0000u))));
      amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(raw[x].y << 16)),
                               fabsf(__uint_as_float(raw[x].y & 0xffff0000u))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float f = row_factor<14>(amax);
    lscale[h] = a.scale_log2 / f;
#pragma unroll
    for (int x = 0; x < C; ++x) {
      qa[x][h] = half2_bits(__uint_as_float(raw[x].x << 16) * f,
                            __uint_as_float(raw[x].x & 0xffff0000u) * f);
      qa[x][2 + h] = half2_bits(__uint_as_float(raw[x].y << 16) * f,
                                __uint_as_float(raw[x].y & 0xffff0000u) * f);
    }
  }

  float o[C][2][4];  // chunk x, even / odd dims: rows g (0, 1) and g + 8 (2, 3)
#pragma unroll
  for (int x = 0; x < C; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[x][e][k] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  int stage = 0;
  for (int t = tile0; t < tile_end; t += kWarps) {
    cp_wait<kStages - 2>();
    __syncwarp();
    issue(t + (kStages - 1) * kWarps, stage == 0 ? kStages - 1 : stage - 1);
    const uint32_t kt = ring_u + stage * L_::kStageBytes, vt = kt + L_::kTileBytes;
    const float4 sc = *reinterpret_cast<const float4*>(ring + stage * L_::kStageBytes + 2 * L_::kTileBytes);
    float s[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[j][k] = 0.f;
#pragma unroll
      for (int x = 0; x < C; x += 4) {
        uint32_t r[4];
        ldsm4(kt + tile_off<D>(8 * j + (lane & 7), x + (lane >> 3)), r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t b0, b1;
          codes_to_half(r[k], b0, b1);
          mma16816(s[j], qa[x + k], b0, b1);
        }
      }
    }
    // logits in base 2 with the value scale folded in; what a row does not see
    const int base = tile_base(t);
    const float vs0 = fmaxf(sc.z, kMinBlockScale), vs1 = fmaxf(sc.w, kMinBlockScale);
    const float lv[2] = {__log2f(vs0), __log2f(vs1)};
    const float iv[2] = {__frcp_rn(vs0), __frcp_rn(vs1)};
    const bool whole = (a.causal ? base + kTile <= p0 + 1 : base + kTile <= q.L) &&
                       (a.window == 0 || base > p1 - a.window || base + kTile <= a.sinks);
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float ks = j < 2 ? sc.x : sc.y;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int h = k >> 1;
        float x = fmaf(s[j][k], lscale[h] * ks, lv[j >> 1]);
        if (!whole) {
          const int tok = base + 8 * j + 2 * i4 + (k & 1);
          const bool sees = see[h](tok);
          x = sees ? x : -INFINITY;
        }
        s[j][k] = x;
        top[h] = fmaxf(top[h], x);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
    }
    const bool move = top[0] > m[0] + kRescale || top[1] > m[1] + kRescale;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nm = fmaxf(m[h], top[h]);
        const float f = nm == m[h] ? 1.f : ex2(m[h] - nm);  // 0 from a row's first keys
        m[h] = nm;
        l[h] *= f;
#pragma unroll
        for (int x = 0; x < C; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            o[x][e][2 * h] *= f;
            o[x][e][2 * h + 1] *= f;
          }
      }
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0] - kLift, m[1] == -INFINITY ? 0.f : m[1] - kLift};
    uint32_t pa[2][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = ex2(s[j][k] - ref[k >> 1]);
        l[k >> 1] = fmaf(w[k], iv[j >> 1], l[k >> 1]);
      }
      pa[j >> 1][2 * (j & 1)] = half2_bits(w[0], w[1]);
      pa[j >> 1][2 * (j & 1) + 1] = half2_bits(w[2], w[3]);
    }
#pragma unroll
    for (int x = 0; x < C; x += 2) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t r[4];  // keys 16 kk .. + 7 and + 8 .. + 15 of chunk x, then of chunk x + 1
        ldsm4_t(vt + tile_off<D>(16 * kk + (lane & 15), x + (lane >> 4)), r);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t b0e, b0o, b1e, b1o;
          codes_to_half(__byte_perm(r[2 * e], 0, 0x3120), b0e, b0o);
          codes_to_half(__byte_perm(r[2 * e + 1], 0, 0x3120), b1e, b1o);
          mma16816(o[x + e][0], pa[kk], b0e, b1e);
          mma16816(o[x + e][1], pa[kk], b0o, b1o);
        }
      }
    }
    stage = stage == kStages - 1 ? 0 : stage + 1;
  }

  if (bad) atomicOr(c.err, kErrBadBatch);

  // the warps' results, each relative to its own reference, meet in shared memory
  cp_wait<0>();
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  float* ow = reinterpret_cast<float*>(ring);
  float2* ml = reinterpret_cast<float2*>(smem + kWarps * L_::kWarpBytes);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
#pragma unroll
    for (int x = 0; x < C; ++x)
      *reinterpret_cast<float4*>(ow + r * D + 16 * x + 4 * i4) =
          make_float4(o[x][0][2 * h], o[x][1][2 * h], o[x][0][2 * h + 1], o[x][1][2 * h + 1]);
    if (i4 == 0) ml[warp * kRows + r] = make_float2(m[h], l[h]);
  }
  __syncthreads();

  const size_t tile_id = (static_cast<size_t>(b) * c.hkv + hk) * pl.row_tiles + rt;
  const size_t prow = (tile_id * pl.splits + split) * kRows;
  auto out_row = [&](int r) {
    const int tok = (r0 + r) / a.G;
    return (static_cast<size_t>(q.q0) + tok) * a.hq + hk * a.G + (r0 + r) - tok * a.G;
  };
  for (int e = threadIdx.x; e < (r1 - r0) * (D / 4); e += kWarps * 32) {
    const int r = e / (D / 4), d4 = e % (D / 4);
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w * kRows + r].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 x = ml[w * kRows + r];
      const float f = ex2(x.x - ref);
      const float4 y = *reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(smem + w * L_::kWarpBytes) + r * D + 4 * d4);
      ll = fmaf(x.y, f, ll);
      v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y);
      v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
    }
    if (n_split == 1) {
      finish_row<D>(a, out_row(r), d4, v, mm, ll);
    } else {
      *reinterpret_cast<float4*>(ws.o + (prow + r) * D + 4 * d4) = v;
      if (d4 == 0) ws.ml[prow + r] = make_float2(mm, ll);
    }
  }
  if (n_split == 1) return;

  // the last CTA of the tile to arrive joins the splits, in their order
  __shared__ int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    s_last = atomicAdd(ws.count + tile_id, 1u) == static_cast<unsigned>(n_split - 1);
    if (s_last) ws.count[tile_id] = 0;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  const size_t first = tile_id * pl.splits * kRows;
  for (int e = threadIdx.x; e < (r1 - r0) * (D / 4); e += kWarps * 32) {
    const int r = e / (D / 4), d4 = e % (D / 4);
    join_row<D>(a, ws, first + r, kRows, n_split, out_row(r), d4);
  }
}

template <int D>
cudaError_t launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, int n_sm, cudaStream_t s) {
  static std::atomic<size_t> done[kMaxDevices];
  const void* fn = reinterpret_cast<const void*>(attn_rows_kernel<D>);
  if (const cudaError_t e = opt_in_smem(fn, done, Lay<D>::kSmem); e != cudaSuccess) return e;
  Plan pl;
  const int64_t rows = static_cast<int64_t>(c.max_q) * a.G;
  pl.row_tiles = static_cast<int>((rows + kRows - 1) / kRows);
  const int64_t base = static_cast<int64_t>(pl.row_tiles) * c.hkv * c.n_seqs;
  const int64_t tiles = max_key_tiles(c, a, kRows, kTile);
  // enough CTAs for four rounds of two a SM (ragged lengths), at least two
  // tiles a warp, and no more partial rows than the workspace has
  int64_t splits = (8LL * n_sm + base - 1) / base;
  splits = std::min(splits, (tiles + 2 * kWarps - 1) / (2 * kWarps));
  splits = std::min(splits, static_cast<int64_t>(ws.cap_rows) / (base * kRows));
  splits = std::max<int64_t>(splits, 1);
  pl.tiles_per_split = static_cast<int>((tiles + splits - 1) / splits);
  pl.splits = static_cast<int>((tiles + pl.tiles_per_split - 1) / pl.tiles_per_split);
  const int64_t grid = base * pl.splits;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  attn_rows_kernel<D><<<static_cast<unsigned>(grid), kWarps * 32, Lay<D>::kSmem, s>>>(c, a, ws, pl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_rows_launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, int n_sm,
                             cudaStream_t s) {
  return c.D == 128 ? launch<128>(c, a, ws, n_sm, s) : launch<64>(c, a, ws, n_sm, s);
}

}  // namespace moe
