// Attention over the 8-bit cache for many rows (prompts, chunks) on tcgen05.
//
// The mathematics is that of attn_rows.cu: weights 2^(s + log2 v - m + lift)
// with the block's value scale in the exponent, o = sum w c / sum w / v, an
// online softmax whose reference m moves only when it would grow by 2^5.
//
// One CTA takes 256 rows (a row is a query head of a token; the heads that
// share a kv head are packed into the rows, so K and V are converted once for
// all of them) as two M = 128 tiles, and walks over 128-key tiles:
//   4 warps   e4m3 codes -> f16 (exact), global -> registers -> the 128-byte
//             swizzled layout in shared memory; the next tile's codes are in
//             flight in registers meanwhile
//   1 thread  tcgen05.mma: S = Q K^T (both K-major, from shared memory), then
//             O += P V (P from tensor memory, V as it lies, MN-major)
//   2 x 4     softmax warps, one group a M tile, a thread a row: S from tensor
//             memory, weights back as f16 over S
// The two M tiles take turns, so one's softmax runs under the other's products.
// Tensor memory: S0, S1 (P in their first half), O0, O1: 512 columns.
// Bound by the tensor pipe: 2 * 2 * 128 * 128 * D flops a tile and M tile.
#include <climits>

#include "attn_common.cuh"
#include "smem_opt_in.cuh"
#include "stream_common.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kM = 128;        // rows of an M tile
constexpr int kRows = 2 * kM;  // rows of a CTA
constexpr int kTile = 128;     // keys of a tile
constexpr float kTiny = 1e-37f;  // keeps what is hidden at -inf where a block's scale is 0
constexpr int kThreads = 416;  // 4 + 4 softmax warps, 4 conversion warps, 1 MMA warp

template <int D>
struct Lay {
  static constexpr int kHalf = kTile * 128;        // 128 rows x 64 f16, swizzled
  static constexpr int kMat = kHalf * (D / 64);    // one operand tile
  static constexpr int kQ = 0;                     // two M tiles
  static constexpr int kK = kQ + 2 * kMat;         // two stages
  static constexpr int kV = kK + 2 * kMat;         // two stages
  static constexpr int kConst = kV + 2 * kMat;     // [4][8] float4: scales of a tile's 16-key groups
  static constexpr int kBar = kConst + 4 * 8 * 16;
  static constexpr int kEnd = kBar + 32 * 8;
  static constexpr int kSmem = kEnd + 1024;        // the base is rounded up to 1024
};

enum Bar { kQFull = 0, kKFull = 1, kKEmpty = 3, kVFull = 5, kVEmpty = 7, kSFull = 9, kPFull = 11, kOFull = 13, kBars = 15 };

__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand in the 128-byte swizzled layout: K rows of 128 bytes (64
// f16 along N), 8-row atoms of 1024 bytes apart; the next 64 along N are
// `lead` bytes on.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t smem_addr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}

// Waits for the loads into v; the operands keep their uses behind the wait.
__device__ __forceinline__ void tmem_wait_ld32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

struct Plan {
  int row_tiles, splits, tiles_per_split;
};

// Where a CTA of the grid, or a row of partial results, stands.
struct Work {
  Seq q;
  int b, hk, r0, r1, base_p;
  KeyTiles k;
  int n_split;
};

__device__ __forceinline__ bool work_of(const KvView& c, const AttnArgs& a, const Plan& pl, int b, int hk, int rt,
                                        Work& w) {
  if (!load_seq(c, b, w.q)) return false;
  const int64_t R = static_cast<int64_t>(w.q.n) * a.G;
  const int64_t r0 = static_cast<int64_t>(rt) * kRows;
  if (r0 >= R) return false;
  w.b = b;
  w.hk = hk;
  w.r0 = static_cast<int>(r0);
  w.r1 = static_cast<int>(min(R, r0 + kRows));
  w.base_p = w.q.L - w.q.n;
  w.k = key_tiles<kTile>(a, w.q.L, w.base_p + w.r0 / a.G, w.base_p + (w.r1 - 1) / a.G);
  w.n_split = max((w.k.n_t + pl.tiles_per_split - 1) / pl.tiles_per_split, 1);
  return true;
}

// ---- conversion warps --------------------------------------------------------
template <int D>
struct Converter {
  static constexpr int kChunks = D / 16;                 // 16-code chunks of a key
  static constexpr int kPer = 128 / kChunks;             // keys a pass
  static constexpr int kPasses = kTile / kPer;
  int pid[kPasses] = {};  // pages of the thread's keys of the tile to load
  int gpid = -1;          // page of 16-key group t (threads 0 .. 7)

  __device__ __forceinline__ void pages(const KvView& c, const AttnArgs& a, const Work& w, int t, int end, int tid) {
    if (t >= end) return;
    const int base = w.k.base(t);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int tok = base + p * kPer + tid / kChunks;
      // what no row sees reads as zero: a NaN there would reach the rows through 0 * NaN
      pid[p] = tok < w.k.hi && (tok >= w.k.lo || tok < a.sinks) ? load_page(c, w.b, tok >> c.page_log2) : -1;
    }
    if (tid < 8) {
      const int tok = base + 16 * tid;
      gpid = tok < w.k.hi ? load_page(c, w.b, tok >> c.page_log2) : -1;
    }
  }
  __device__ __forceinline__ void load(const KvView& c, const Work& w, const uint8_t* src, int t, int tid,
                                       uint4 (&raw)[kPasses]) const {
    const int base = w.k.base(t);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int tok = base + p * kPer + tid / kChunks;
      raw[p] = make_uint4(0, 0, 0, 0);
      if (pid[p] >= 0)
        raw[p] = __ldg(reinterpret_cast<const uint4*>(
            src + ((static_cast<size_t>(pid[p]) * c.hkv + w.hk) * c.page + (tok & (c.page - 1))) * D +
            (tid % kChunks) * 16));
    }
  }
  __device__ __forceinline__ void store(char* dst, int tid, const uint4 (&raw)[kPasses]) const {
    const int ch = tid % kChunks, half = ch >> 2;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int row = p * kPer + tid / kChunks;
      uint32_t h[8];
      codes_to_half(raw[p].x, h[0], h[1]);
      codes_to_half(raw[p].y, h[2], h[3]);
      codes_to_half(raw[p].z, h[4], h[5]);
      codes_to_half(raw[p].w, h[6], h[7]);
      char* line = dst + half * Lay<D>::kHalf + row * 128;
      const int c0 = 2 * (ch & 3);
      // lanes of the two halves take their two chunks in opposite order: no bank conflicts
      const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
      const bool swap = half != 0;
      *reinterpret_cast<uint4*>(line + (((c0 + (swap ? 1 : 0)) ^ (row & 7)) << 4)) = swap ? hi : lo;
      *reinterpret_cast<uint4*>(line + (((c0 + (swap ? 0 : 1)) ^ (row & 7)) << 4)) = swap ? lo : hi;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles_kernel(const KvView c, const AttnArgs a, const AttnWs ws, const Plan pl) {
  using L_ = Lay<D>;
  extern __shared__ char smem_raw[];
  __shared__ uint32_t s_tmem;
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base_u = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), wg = warp >> 2;  // uniform

  // long tiles first: the last rows of a causal prompt see the most keys
  int idx = blockIdx.x;
  const int hk = idx % c.hkv;
  idx /= c.hkv;
  const int b = idx % c.n_seqs;
  idx /= c.n_seqs;
  const int split = idx % pl.splits;
  const int rt = pl.row_tiles - 1 - idx / pl.splits;
  Work w;
  if (!work_of(c, a, pl, b, hk, rt, w) || split >= w.n_split) return;
  const int t_begin = split * pl.tiles_per_split;
  const int t_end = min(w.k.n_t, t_begin + pl.tiles_per_split);
  const int n = t_end - t_begin;  // 0 when the rows see nothing
  const int n_mt = w.r1 - w.r0 > kM ? 2 : 1;

  auto bar = [&](int i) { return base_u + L_::kBar + 8 * i; };
  if (threadIdx.x == 0) {
    const int count[kBars] = {128 * n_mt, 128, 128, 1, 1, 128, 128, 1, 1, 1, 1, 128, 128, 1, 1};
#pragma unroll
    for (int i = 0; i < kBars; ++i) mbar_init(bar(i), count[i]);
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = s_tmem;

  if (wg == 3) {
    if ((threadIdx.x & 31) == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_f16(kM, kTile);
      constexpr uint32_t id_o = idesc_f16(kM, D) | (1u << 16);  // V is MN-major
      auto issue_s = [&](int i, int stage) {
        const uint32_t qa = base_u + L_::kQ + i * L_::kMat, kb = base_u + L_::kK + stage * L_::kMat;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * L_::kHalf + (k & 3) * 32;
          mma_ss(tmem + i * 128, sdesc_sw128(qa + off), sdesc_sw128(kb + off), id_s, k != 0);
        }
        mma_commit(bar(kSFull + i));
      };
      bool ok = mbar_wait(bar(kQFull), 0, c.err) && mbar_wait(bar(kKFull), 0, c.err);
      if (ok) {
        fence_after_sync();
        for (int i = 0; i < n_mt; ++i) issue_s(i, 0);
        mma_commit(bar(kKEmpty));
      }
      for (int j = 0; ok && j < n; ++j) {
        const int st = j & 1;
        const uint32_t vb = base_u + L_::kV + st * L_::kMat;
        for (int i = 0; ok && i < n_mt; ++i) {
          ok = mbar_wait(bar(kPFull + i), j & 1, c.err) && (i > 0 || mbar_wait(bar(kVFull + st), (j >> 1) & 1, c.err));
          if (!ok) break;
          fence_after_sync();
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ts(tmem + 256 + i * 128, tmem + i * 128 + k * 8, sdesc_sw128_mn(vb + k * 2048, L_::kHalf), id_o,
                   (j | k) != 0);
          if (i == n_mt - 1) mma_commit(bar(kVEmpty + st));
          if (j == n - 1) {
            mma_commit(bar(kOFull + i));
          } else {
            const int s2 = (j + 1) & 1;
            ok = i > 0 || mbar_wait(bar(kKFull + s2), ((j + 1) >> 1) & 1, c.err);
            if (!ok) break;
            fence_after_sync();
            issue_s(i, s2);
            if (i == n_mt - 1) mma_commit(bar(kKEmpty + s2));
          }
        }
      }
      if (!ok) {
        // what was issued ends by itself; wait for it before the tensor memory goes back
        mma_commit(bar(kOFull));
        mbar_wait(bar(kOFull), 0, c.err);
      }
    }
  } else if (wg == 2) {
    const int tid = threadIdx.x - 256;
    if (n > 0) {
      Converter<D> cv;
      uint4 kr[Converter<D>::kPasses], vr[Converter<D>::kPasses];
      float4 cn = make_float4(0.f, 0.f, 1.f, 0.f);
      auto consts = [&]() {  // of the tile whose pages are in cv
        if (tid < 8) {
          float ks = 0.f, vs = 1.f;
          if (cv.gpid >= 0) {
            const size_t at = static_cast<size_t>(cv.gpid) * c.hkv + w.hk;
            ks = __ldg(c.k_scale + at);
            vs = __ldg(c.v_scale + at);
          }
          vs = fmaxf(vs, kMinBlockScale);
          cn = make_float4(ks, __log2f(vs), __frcp_rn(vs), 0.f);
        }
      };
      cv.pages(c, a, w, t_begin, t_end, tid);
      cv.load(c, w, c.k, t_begin, tid, kr);
      cv.load(c, w, c.v, t_begin, tid, vr);
      consts();
      cv.pages(c, a, w, t_begin + 1, t_end, tid);
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        const int st = j & 1;
        const uint32_t prev = ((j >> 1) & 1) ^ 1;  // parity of the stage's release two tiles ago
        if (j >= 2 && !(ok = mbar_wait(bar(kKEmpty + st), prev, c.err))) break;
        cv.store(smem + L_::kK + st * L_::kMat, tid, kr);
        // a ring of four: the softmax of tile j - 3 is done when the K stage of tile j is free
        if (tid < 8) reinterpret_cast<float4*>(smem + L_::kConst)[(j & 3) * 8 + tid] = cn;
        fence_proxy_async_smem();
        mbar_arrive(bar(kKFull + st));
        if (j + 1 < n) cv.load(c, w, c.k, t_begin + j + 1, tid, kr);
        if (j >= 2 && !(ok = mbar_wait(bar(kVEmpty + st), prev, c.err))) break;
        cv.store(smem + L_::kV + st * L_::kMat, tid, vr);
        fence_proxy_async_smem();
        mbar_arrive(bar(kVFull + st));
        if (j + 1 < n) {
          cv.load(c, w, c.v, t_begin + j + 1, tid, vr);
          consts();
          cv.pages(c, a, w, t_begin + j + 2, t_end, tid);
        }
      }
    }
  } else if (wg < n_mt) {
    const int i = wg, row = threadIdx.x & 127;
    const int r = w.r0 + i * kM + row;
    const bool live = r < w.r1;
    const int tok = live ? r / a.G : 0;
    const int head = w.hk * a.G + (live ? r - tok * a.G : 0);
    const RowSees sees = row_sees(a, w.q.L, w.base_p + tok, live);
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 * (warp % 4)
    const uint32_t ts = tmem + i * 128 + lanes, to = tmem + 256 + i * 128 + lanes;
    float m = -INFINITY, l = 0.f, lscale = 0.f;  // lscale >= 0: a negative scale turns the query's sign
    bool ok = true;
    if (n > 0) {
      // the row's query to f16, brought to [2^14, 2^15) by a power of two
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<int64_t>(w.q.q0) + tok) * a.q_stride + static_cast<int64_t>(head) * D);
      uint4 raw[D / 8];
      float amax = 0.f;
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        raw[x] = live ? __ldg(src + x) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u))));
      }
      const float f = copysignf(row_factor(amax), a.scale_log2);
      lscale = a.scale_log2 / f;
      char* dst = smem + L_::kQ + i * L_::kMat + row * 128;
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        const uint32_t u[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          h[k] = half2_bits(__uint_as_float(u[k] << 16) * f, __uint_as_float(u[k] & 0xffff0000u) * f);
        *reinterpret_cast<uint4*>(dst + (x >> 3) * L_::kHalf + (((x & 7) ^ (row & 7)) << 4)) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kQFull));
    }
    // the range that all rows of the CTA see whole
    const int p_lo = w.base_p + w.r0 / a.G, p_hi = w.base_p + (w.r1 - 1) / a.G;
    for (int j = 0; j < n; ++j) {
      // K's barrier orders this thread after the scales in shared memory, S's
      // after the products (and after O += P V of the tile before)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(kKFull + (j & 1)), (j >> 1) & 1, c.err) &&
                                       mbar_wait(bar(kSFull + i), j & 1, c.err));
      if (!ok) break;
      fence_after_sync();
      const float4* cn = reinterpret_cast<const float4*>(smem + L_::kConst) + (j & 3) * 8;
      const int base = w.k.base(t_begin + j);
      const bool whole = (a.causal ? base + kTile <= p_lo + 1 : base + kTile <= w.q.L) &&
                         (a.window == 0 || base > p_hi - a.window || base + kTile <= a.sinks);
      // S is read twice, 32 columns at a time and the next 32 under way: for the
      // row's largest logit (within 16 keys of one scale the largest product
      // gives it), then for the weights
      float s[2][32];
      auto hide = [&](int x) {
        if (!whole) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            s[x & 1][k] = sees(base + 32 * x + k) ? s[x & 1][k] : -INFINITY;
        }
      };
      float mt = -INFINITY;
      tmem_ld32(ts, s[0]);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        tmem_wait_ld32(s[x & 1]);
        tmem_ld32(ts + 32 * ((x + 1) & 3), s[(x + 1) & 1]);
        hide(x);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const float4 z = cn[2 * x + gg];
          const float* v = s[x & 1] + 16 * gg;
          float t0 = fmaxf(fmaxf(v[0], v[1]), v[2]), t1 = fmaxf(fmaxf(v[3], v[4]), v[5]);
#pragma unroll
          for (int k = 6; k < 16; k += 2) {
            float& t = (k & 2) ? t0 : t1;
            t = fmaxf(fmaxf(t, v[k]), v[k + 1]);
          }
          mt = fmaxf(mt, fmaf(fmaxf(t0, t1), fmaxf(lscale * z.x, kTiny), z.y));
        }
      }
      if (__any_sync(0xffffffffu, mt > m + kRescale)) {
        const float nm = fmaxf(m, mt);
        const float f = nm == m ? 1.f : ex2(m - nm);
        m = nm;
        l *= f;
        if (j > 0) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            uint32_t u[16];
            tmem_ld16(to + 16 * x, u);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * f);
            tmem_st16(to + 16 * x, u);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : m - kLift;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        tmem_wait_ld32(s[x & 1]);
        if (x < 3) tmem_ld32(ts + 32 * (x + 1), s[(x + 1) & 1]);
        hide(x);
        uint32_t u[16];
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const float4 z = cn[2 * x + gg];
          const float sc = fmaxf(lscale * z.x, kTiny), off = z.y - ref;
          const float* v = s[x & 1] + 16 * gg;
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float w0 = ex2(fmaf(v[k], sc, off)), w1 = ex2(fmaf(v[k + 1], sc, off));
            sum0 += w0;
            sum1 += w1;
            u[8 * gg + k / 2] = half2_bits(w0, w1);
          }
          l = fmaf(sum0 + sum1, z.z, l);
        }
        tmem_st16(ts + 16 * x, u);
      }
      tmem_wait_st();
      fence_before_sync();
      mbar_arrive(bar(kPFull + i));
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(kOFull + i), 0, c.err));
    if (ok) {
      fence_after_sync();
      const size_t orow = (static_cast<size_t>(w.q.q0) + tok) * a.hq + head;
      const size_t prow =
          (((static_cast<size_t>(b) * c.hkv + hk) * pl.row_tiles + rt) * pl.splits + split) * kRows + i * kM + row;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        float o[32];
        if (n > 0) {
          tmem_ld32(to + 32 * x, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; live && k < 8; ++k) {
          const float4 v = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          if (w.n_split == 1)
            finish_row<D>(a, orow, 8 * x + k, v, m, l);
          else
            *reinterpret_cast<float4*>(ws.o + prow * D + 32 * x + 4 * k) = v;
        }
        __syncwarp();
      }
      if (live && w.n_split > 1) ws.ml[prow] = make_float2(m, l);
    }
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// Joins the splits of every row that has more than one.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads)
    attn_join_kernel(const KvView c, const AttnArgs a, const AttnWs ws, const Plan pl) {
  constexpr int kPer = kJoinThreads / (D / 4);  // rows of a block
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kPer + threadIdx.x / (D / 4);
  const int row = static_cast<int>(item % kRows);
  const int64_t tile_id = item / kRows;
  const int rt = static_cast<int>(tile_id % pl.row_tiles);
  const int64_t s = tile_id / pl.row_tiles;
  const int hk = static_cast<int>(s % c.hkv), b = static_cast<int>(s / c.hkv);
  Work w;
  if (b >= c.n_seqs || !work_of(c, a, pl, b, hk, rt, w) || w.n_split == 1 || w.r0 + row >= w.r1) return;
  const int tok = (w.r0 + row) / a.G;
  const size_t orow = (static_cast<size_t>(w.q.q0) + tok) * a.hq + hk * a.G + (w.r0 + row) - tok * a.G;
  join_row<D>(a, ws, static_cast<size_t>(tile_id) * pl.splits * kRows + row, kRows, w.n_split, orow,
              threadIdx.x % (D / 4));
}

template <int D>
cudaError_t launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, int n_sm, cudaStream_t s) {
  static std::atomic<size_t> done[kMaxDevices];
  const void* fn = reinterpret_cast<const void*>(attn_tiles_kernel<D>);
  if (const cudaError_t e = opt_in_smem(fn, done, Lay<D>::kSmem); e != cudaSuccess) return e;
  Plan pl;
  const int64_t rows = static_cast<int64_t>(c.max_q) * a.G;
  pl.row_tiles = static_cast<int>((rows + kRows - 1) / kRows);
  const int64_t base = static_cast<int64_t>(pl.row_tiles) * c.hkv * c.n_seqs;
  const int64_t tiles = max_key_tiles(c, a, kRows, kTile);
  // one CTA a SM: split the keys when the row tiles leave SMs without work
  int64_t splits = base >= n_sm ? 1 : (2LL * n_sm + base - 1) / base;
  splits = std::min(splits, (tiles + 3) / 4);
  splits = std::min(splits, static_cast<int64_t>(ws.cap_rows) / (base * kRows));
  splits = std::max<int64_t>(splits, 1);
  pl.tiles_per_split = static_cast<int>((tiles + splits - 1) / splits);
  pl.splits = static_cast<int>((tiles + pl.tiles_per_split - 1) / pl.tiles_per_split);
  const int64_t grid = base * pl.splits;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  attn_tiles_kernel<D><<<static_cast<unsigned>(grid), kThreads, Lay<D>::kSmem, s>>>(c, a, ws, pl);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || pl.splits == 1) return e;
  const int64_t items = base * kRows, per = kJoinThreads / (D / 4);
  attn_join_kernel<D><<<static_cast<unsigned>((items + per - 1) / per), kJoinThreads, 0, s>>>(c, a, ws, pl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_tiles_launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, int n_sm,
                              cudaStream_t s) {
  return c.D == 128 ? launch<128>(c, a, ws, n_sm, s) : launch<64>(c, a, ws, n_sm, s);
}

}  // namespace moe
