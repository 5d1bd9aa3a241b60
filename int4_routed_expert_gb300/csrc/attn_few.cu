// Attention over the 8-bit cache for few rows (single tokens, verify batches)
// on tcgen05, the keys as the products' M dimension.
//
// Mathematics.  Row r (a query head of a new token) sees keys j with logits
// s_j = scale * q . k_j.  With the page's value scale v_j folded into the
// exponent, w_j = 2^(s_j log2 e + log2 v_j - m), the output is
//   o = sum_j w_j c_j / sum_j (w_j / v_j),   c_j the value's e4m3 code,
// so one running reference m serves both sums and the f16 weights are relative
// to the largest contribution, whatever the blocks' scales are.  m moves only
// when it would grow by 2^5.
//
// A CTA takes N = 16 or 64 rows of a kv head and walks over tiles of 128 keys:
//   S^T[128 keys x 2 N] = K [Q1; Q2]^T   e4m3; the bf16 query as two e4m3 terms
//   P[128 keys x N]                      a thread a key, f16
//   O^T[128 dims x N]  += V^T P          f16, V as it lies (M-major)
// With the keys in M the tensor pipe reads K and V once whatever N is, a
// thread's block scales are scalars, it writes its key's weights as they stand
// in one operand row, and no thread shuffles: only when a reference moves, the
// maxima over the keys are exchanged.  The keys are split over CTAs; the last
// CTA of a row tile to arrive joins them.
// Warps: 4 softmax for every 32 rows, 4 conversion of the value codes, MMA, load.
// Bound by memory: 2 D bytes a key and kv head.
#include "attn_tc.cuh"

namespace moe {
namespace {


enum Bar {
  kQFull = 0,
  kKFull = 1,    // [3] key codes
  kKEmpty = 4,   // [3]
  kRFull = 7,    // [3] value codes
  kREmpty = 10,  // [3]
  kVFull = 13,   // [2] values
  kSFull = 15,   // [2] S^T
  kPFull = 17,   // [2] P
  kODone = 19,   // [2] O^T += V^T P, by the parity of the tile
  kCFull = 21,   // [4] scales
  kDrain = 25,
  kBars = 26
};

// N = 16 keeps to half an SM, so that two CTAs cover each other's bubbles.
template <int D, int N>
struct Lay {
  static constexpr int kStages = N == 16 ? 2 : 3;   // of key codes and of value codes
  static constexpr int kVStages = N == 16 ? 1 : 2;  // of f16 values
  using Io = TileIo<D, kStages, kStages, kVStages>;
  static constexpr int kGroups = N == 16 ? 1 : 2;   // softmax groups of 128 threads
  static constexpr int kGroupRows = N / kGroups;
  static constexpr int kThreads = 128 * kGroups + 192;
  static constexpr int kQ = 0;                      // [2 N][D]
  static constexpr int kK = kQ + (2 * N * D + 1023) / 1024 * 1024;
  static constexpr int kV = kK + kStages * Io::kMat8;
  static constexpr int kRaw = kV + kVStages * Io::kMat;
  static constexpr int kP = kRaw + kStages * Io::kMat8;  // [2][128 keys][N] f16
  static constexpr int kConst = kP + 2 * kKeys * N * 2;
  static constexpr int kRow = kConst + kConstRing * 8 * 16;  // [6][N]: see Rows
  static constexpr int kRed = kRow + 6 * N * 4;              // [4][N] floats
  static constexpr int kBar = kRed + 4 * N * 4;
  static constexpr int kSmem = kBar + kBars * 8 + 1024;
  static constexpr int kTmem = N == 16 ? 128 : 512;          // S^T twice, then O^T
};

// What the softmax threads share of the rows.
template <int N>
struct Rows {
  float* lscale;  // logit scale, the query's power of two undone
  float* nref;    // lift - reference
  float* m;       // reference
  float* f;       // factor of a move
  int* lo;
  int* hi;
  __device__ __forceinline__ explicit Rows(char* p)
      : lscale(reinterpret_cast<float*>(p)), nref(lscale + N), m(nref + N), f(m + N),
        lo(reinterpret_cast<int*>(f + N)), hi(lo + N) {}
};

// P's operand layout: a key's N f16 in a row of 2 N bytes, rows swizzled in
// 2 N-byte patterns; byte offset of its 16-byte chunk c.
template <int N>
__device__ __forceinline__ uint32_t p_off(int key, int c) {
  return N == 64 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 32 + ((c ^ ((key >> 2) & 1)) << 4);
}
template <int N>
__device__ __forceinline__ uint64_t sdesc_p(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;  // (one swizzle pattern wide: no next block along N)
  d |= static_cast<uint64_t>((8 * 2 * N) >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(N == 64 ? 2u : 6u) << 61;
  return d;
}

// O^T[tmem] (+)= V^T[smem] P[smem] over 128 keys, 16 a step: both operands
// MN-major, V 2048 bytes a step, P 32 N.
template <int N>
__device__ __forceinline__ void mma_ot(uint32_t d_tmem, uint64_t v_desc, uint64_t p_desc, uint32_t idesc,
                                       uint32_t first) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 v<8>, b<8>;\n\t"
      "setp.eq.b32 p, %4, 0;\n\t"
      "add.s64 v1, %1, 128;\n\tadd.s64 v2, v1, 128;\n\tadd.s64 v3, v2, 128;\n\tadd.s64 v4, v3, 128;\n\t"
      "add.s64 v5, v4, 128;\n\tadd.s64 v6, v5, 128;\n\tadd.s64 v7, v6, 128;\n\t"
      "add.s64 b1, %2, %5;\n\tadd.s64 b2, b1, %5;\n\tadd.s64 b3, b2, %5;\n\tadd.s64 b4, b3, %5;\n\t"
      "add.s64 b5, b4, %5;\n\tadd.s64 b6, b5, %5;\n\tadd.s64 b7, b6, %5;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], v1, b1, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], v2, b2, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], v3, b3, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], v4, b4, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], v5, b5, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], v6, b6, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], v7, b7, %3, 1;\n\t}" ::"r"(d_tmem),
      "l"(v_desc), "l"(p_desc), "r"(idesc), "r"(first), "n"(static_cast<uint64_t>(32 * N) >> 4)
      : "memory");
}

// S^T[tmem] = K[smem] Q[smem]^T, e4m3, 32 codes a step.
template <int D>
__device__ __forceinline__ void mma_st(uint32_t d_tmem, uint64_t k_desc, uint64_t q_desc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .b64 k<2>, q<2>;\n\t"
      "add.s64 k1, %1, 2;\n\tadd.s64 q1, %2, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], k1, q1, %3, 1;\n\t}" ::"r"(d_tmem),
      "l"(k_desc), "l"(q_desc), "r"(idesc)
      : "memory");
  if constexpr (D == 128)
    asm volatile(
        "{\n\t.reg .b64 k<4>, q<4>;\n\t"
        "add.s64 k2, %1, 4;\n\tadd.s64 q2, %2, 4;\n\tadd.s64 k3, %1, 6;\n\tadd.s64 q3, %2, 6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], k2, q2, %3, 1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], k3, q3, %3, 1;\n\t}" ::"r"(d_tmem),
        "l"(k_desc), "l"(q_desc), "r"(idesc)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld16f(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

// Whether any of a softmax group's 128 threads says yes (a barrier among them).
__device__ __forceinline__ bool vote(int group, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(yes)), "r"(1 + group)
      : "memory");
  return r != 0;
}

template <int D, int N>
__global__ void __launch_bounds__(Lay<D, N>::kThreads, N == 16 ? 2 : 1)
    attn_few_kernel(const KvView c, const AttnArgs a, const AttnWs ws, const Plan pl,
                    const __grid_constant__ CUtensorMap k_map) {
  using L_ = Lay<D, N>;
  using Io = typename L_::Io;
  extern __shared__ char smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base_u = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  int idx = blockIdx.x;
  const int hk = idx % c.hkv;
  idx /= c.hkv;
  const int rt = idx % pl.row_tiles;
  idx /= pl.row_tiles;
  const int b = idx % c.n_seqs, split = idx / c.n_seqs;
  Work w;
  if (!work_of<N>(c, a, pl, b, hk, rt, w) || split >= w.n_split) return;
  const int t_begin = split * pl.tiles_per_split;
  const int n = min(w.k.n_t, t_begin + pl.tiles_per_split) - t_begin;  // 0 when the rows see nothing

  auto bar = [&](int i) { return base_u + L_::kBar + 8 * i; };
  if (threadIdx.x == 0) {
    constexpr int kS = 128 * L_::kGroups;
    const int count[kBars] = {kS, 1, 1, 1, L_::kGroups, L_::kGroups, L_::kGroups, 1, 1, 1, 128, 128, 128, 128, 128,
                              1, 1, kS, kS, 1, 1, 8, 8, 8, 8, 1};
#pragma unroll
    for (int i = 0; i < kBars; ++i) mbar_init(bar(i), count[i]);
    fence_barrier_init();
  }
  constexpr int kConv = 4 * L_::kGroups, kMma = kConv + 4;  // first conversion warp, MMA warp; then the load warp
  if (warp == kMma) {
    tmem_alloc(smem_u32(&s_tmem), L_::kTmem);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = s_tmem;
  const uint32_t ot = tmem + 4 * N;  // S^T: columns 0 .. 4 N - 1
  const Io io{base_u + L_::kK, base_u + L_::kRaw, base_u + L_::kV, smem, base_u, base_u + L_::kConst,
              bar(kKFull), bar(kKEmpty), bar(kRFull), bar(kREmpty), bar(kVFull), bar(kCFull)};
  const Rows<N> rows(smem + L_::kRow);

  if (warp == kMma + 1) {
    if (lane < 8 && n > 0) io.load(c, a, w.k, b, hk, t_begin, n, &k_map, lane);
  } else if (warp == kMma) {
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_f16(kKeys, 2 * N);                      // e4m3 is format 0 of its kind, too
      constexpr uint32_t id_o = idesc_f16(128, N) | (1u << 15) | (1u << 16);  // both MN-major
      const uint64_t q_desc = sdesc_k<D>(base_u + L_::kQ), k_desc = sdesc_k<D>(base_u + L_::kK);
      // heads of 64: the accumulator's other 64 rows take what lies behind, and are not read
      const uint64_t v_desc = sdesc_sw128_mn(base_u + L_::kV, D == 128 ? Io::kHalf : 1024);
      const uint64_t p_desc = sdesc_p<N>(base_u + L_::kP);
      auto issue_s = [&](int j) {
        const int ks = j % L_::kStages;
        if (!mbar_wait(bar(kKFull + ks), (j / L_::kStages) & 1, c.err)) return false;
        fence_after_sync();
        mma_st<D>(tmem + (j & 1) * 2 * N, k_desc + ks * (Io::kMat8 >> 4), q_desc, id_s);
        mma_commit(bar(kSFull + (j & 1)));
        return true;
      };
      bool ok = mbar_wait(bar(kQFull), 0, c.err) && issue_s(0) && (n < 2 || issue_s(1));
      for (int j = 0; ok && j < n; ++j) {
        const int vs = j % L_::kVStages;
        ok = mbar_wait(bar(kPFull + (j & 1)), (j >> 1) & 1, c.err) &&
             mbar_wait(bar(kVFull + vs), (j / L_::kVStages) & 1, c.err);
        if (!ok) break;
        fence_after_sync();
        mma_ot<N>(ot, v_desc + vs * (Io::kMat >> 4), p_desc + (j & 1) * (kKeys * 2 * N >> 4), id_o, j == 0);
        mma_commit(bar(kODone + (j & 1)));
        ok = j + 2 >= n || issue_s(j + 2);
      }
      if (!ok) {
        // what was issued ends by itself; wait for it before the tensor memory goes back
        mma_commit(bar(kDrain));
        mbar_wait(bar(kDrain), 0, c.err);
      }
    }
  } else if (warp >= kConv) {
    // the stage of tile j - VS is free when its product is done
    io.convert(c, a, w.k, t_begin, n, threadIdx.x - 32 * kConv, [&](int j) {
      const int i = j - L_::kVStages;
      return mbar_wait(bar(kODone + (i & 1)), (i >> 1) & 1, c.err);
    });
  } else {
    // ---- softmax: thread t is key t of a tile -----------------------------------
    constexpr int NG = L_::kGroupRows;
    const int t = threadIdx.x & 127, grp = warp >> 2, g0 = grp * NG;  // rows g0 .. of the group
    float l[NG];
#pragma unroll
    for (int r = 0; r < NG; ++r) l[r] = 0.f;
    // the rows' queries as two e4m3 terms, 128 kGroups / N threads a row
    {
      constexpr int kPer = 128 * L_::kGroups / N, kDims = D / kPer;  // threads a row, dims a thread
      const int r = threadIdx.x / kPer, part = threadIdx.x % kPer, gr = w.r0 + r;
      const bool live = gr < w.r1;
      const int tok = live ? gr / a.G : 0;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<int64_t>(w.q.q0) + tok) * a.q_stride +
          (static_cast<int64_t>(hk) * a.G + (live ? gr - tok * a.G : 0)) * D + part * kDims);
      uint4 raw[kDims / 8];
      float amax = 0.f;
#pragma unroll
      for (int x = 0; x < kDims / 8; ++x) {
        raw[x] = live ? __ldg(src + x) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = max3(amax, fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u)));
      }
#pragma unroll
      for (int o = kPer / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float f = copysignf(row_factor<7>(amax), a.scale_log2);
      const bool inf = !(amax < INFINITY);  // (codes saturate: such a row is NaN instead)
#pragma unroll
      for (int x = 0; x < kDims / 8; ++x) {
        const uint32_t u[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
        uint32_t t0[2], t1[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t a1, a2, b1, b2;
          split_query(u[2 * k], f, a1, a2);
          split_query(u[2 * k + 1], f, b1, b2);
          t0[k] = inf ? 0x7f7f7f7fu : a1 | (b1 << 16);
          t1[k] = a2 | (b2 << 16);
        }
        const int byte = part * kDims + 8 * x;
        char* dst = smem + L_::kQ + (byte & 8);
        *reinterpret_cast<uint2*>(dst + k_off<D>(r, byte >> 4)) = make_uint2(t0[0], t0[1]);
        *reinterpret_cast<uint2*>(dst + k_off<D>(N + r, byte >> 4)) = make_uint2(t1[0], t1[1]);
      }
      if (part == 0) {
        const RowSees s = row_sees(a, w.q.L, w.base_p + tok, live);
        rows.lscale[r] = fmaxf(a.scale_log2 / f, kTiny);
        rows.nref[r] = 0.f;
        rows.m[r] = -INFINITY;
        rows.lo[r] = s.lo;
        rows.hi[r] = s.hi;
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kQFull));
    }
    named_sync(3, 128 * L_::kGroups);
    const int p_lo = w.base_p + w.r0 / a.G, p_hi = w.base_p + (w.r1 - 1) / a.G;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 * (warp % 4)
    float* red = reinterpret_cast<float*>(smem + L_::kRed);
    bool ok = true, pending = true;  // a row has no reference yet
    for (int j = 0; j < n; ++j) {
      const int bf = j & 1, ph = (j >> 1) & 1;
      ok = mbar_wait(bar(kSFull + bf), ph, c.err) &&
           mbar_wait(bar(kCFull + j % kConstRing), (j / kConstRing) & 1, c.err) &&
           // P of tile j - 2 has been read
           (j < 2 || mbar_wait(bar(kODone + bf), ph ^ 1, c.err));
      ok = __all_sync(0xffffffffu, ok);
      if (vote(grp, !ok)) {
        ok = false;
        break;
      }
      fence_after_sync();
      if (t == 0) mbar_arrive(bar(kKEmpty + j % L_::kStages));
      const float4 cn = io.scales(j)[t >> 4];
      const float ks = fmaxf(cn.x, kTiny);
      const int tok = w.k.base(t_begin + j) + t, key0 = tok - t;
      const bool whole = (a.causal ? key0 + kKeys <= p_lo + 1 : key0 + kKeys <= w.q.L) &&
                         (a.window == 0 || key0 > p_hi - a.window || key0 + kKeys <= a.sinks);
      // exponents relative to the rows' references
      float z[NG];
      float top = -INFINITY;
      const uint32_t st = tmem + bf * 2 * N + lanes + g0;
#pragma unroll
      for (int x = 0; x < NG; x += 16) {
        float s2[16];
        tmem_ld16f(st + x, z + x);
        tmem_ld16f(st + N + x, s2);
        tmem_wait_ld16f(z + x);
        tmem_wait_ld16f(s2);
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const float4 ls = *reinterpret_cast<const float4*>(rows.lscale + g0 + x + r);
          const float4 nr = *reinterpret_cast<const float4*>(rows.nref + g0 + x + r);
          float* y = z + x + r;
          y[0] = fmaf((y[0] + s2[r]) * ks, ls.x, cn.y) + nr.x;
          y[1] = fmaf((y[1] + s2[r + 1]) * ks, ls.y, cn.y) + nr.y;
          y[2] = fmaf((y[2] + s2[r + 2]) * ks, ls.z, cn.y) + nr.z;
          y[3] = fmaf((y[3] + s2[r + 3]) * ks, ls.w, cn.y) + nr.w;
        }
        if (!whole) {
#pragma unroll
          for (int r = x; r < x + 16; ++r) {
            const bool sees = tok <= rows.hi[g0 + r] && (tok >= rows.lo[g0 + r] || tok < a.sinks);
            z[r] = sees ? z[r] : -INFINITY;
          }
        }
#pragma unroll
        for (int r = x; r < x + 16; r += 2) top = max3(top, z[r], z[r + 1]);
      }
      if (vote(grp, pending || top > kLift + kRescale)) {
        // some reference moves: the rows' maxima over the tile, warp by warp
#pragma unroll
        for (int r = 0; r < NG; ++r) {
          const int i = __float_as_int(z[r]);
          const int most = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7fffffff));  // ordered like floats
          if (lane == 0) red[(warp & 3) * N + g0 + r] = __int_as_float(most ^ ((most >> 31) & 0x7fffffff));
        }
        named_sync(1 + grp, 128);
        if (t < NG) {
          const int q = g0 + t;
          const float mx = fmaxf(fmaxf(red[q], red[N + q]), fmaxf(red[2 * N + q], red[3 * N + q])) - rows.nref[q];
          const float m = rows.m[q];
          const bool move = mx > m + kRescale;
          const float nm = move ? mx : m;
          rows.f[q] = move ? ex2(m - nm) : 1.f;
          red[q] = move ? (kLift - nm) - rows.nref[q] : 0.f;  // what the exponents change by
          rows.m[q] = nm;
          if (move) rows.nref[q] = kLift - nm;
        }
        named_sync(1 + grp, 128);
#pragma unroll
        for (int r = 0; r < NG; ++r) {
          z[r] += red[g0 + r];
          l[r] *= rows.f[g0 + r];
        }
        if (j > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(kODone + (bf ^ 1)), ((j - 1) >> 1) & 1, c.err));
          fence_after_sync();
#pragma unroll
          for (int x = 0; x < NG; x += 16) {
            uint32_t u[16];
            tmem_ld16(ot + lanes + g0 + x, u);
            tmem_wait_ld16(u);
#pragma unroll
            for (int r = 0; r < 16; ++r) u[r] = __float_as_uint(__uint_as_float(u[r]) * rows.f[g0 + x + r]);
            tmem_st16(ot + lanes + g0 + x, u);
          }
          tmem_wait_st();
        }
        // (a barrier, too: red and f are free again)
        pending = vote(grp, t < NG && rows.m[g0 + t % NG] == -INFINITY && rows.hi[g0 + t % NG] >= 0);
      }
      char* p = smem + L_::kP + bf * (kKeys * 2 * N);
#pragma unroll
      for (int x = 0; x < NG; x += 8) {
        uint32_t u[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w0 = ex2(z[x + 2 * r]), w1 = ex2(z[x + 2 * r + 1]);
          l[x + 2 * r] = fmaf(w0, cn.z, l[x + 2 * r]);
          l[x + 2 * r + 1] = fmaf(w1, cn.z, l[x + 2 * r + 1]);
          u[r] = half2_bits(w0, w1);
        }
        *reinterpret_cast<uint4*>(p + p_off<N>(t, (g0 + x) >> 3)) = make_uint4(u[0], u[1], u[2], u[3]);
      }
      fence_proxy_async_smem();
      fence_before_sync();
      mbar_arrive(bar(kPFull + bf));
    }
    // the weights' sums over the keys
#pragma unroll
    for (int r = 0; r < NG; ++r) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
      if (lane == 0) red[(warp & 3) * N + g0 + r] = l[r];
    }
    if (ok && n > 0)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(kODone + ((n - 1) & 1)), ((n - 1) >> 1) & 1, c.err));
    named_sync(1 + grp, 128);
    fence_after_sync();
    // thread t has dim t of every row
    const size_t tile_id = (static_cast<size_t>(b) * c.hkv + hk) * pl.row_tiles + rt;
    const size_t prow = (tile_id * pl.splits + split) * N;
    const int live = w.r1 - w.r0;
#pragma unroll
    for (int x = 0; x < NG; x += 16) {
      float o[16];
      if (n > 0 && ok) {
        tmem_ld16f(ot + lanes + g0 + x, o);
        tmem_wait_ld16f(o);
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) o[r] = 0.f;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = g0 + x + r;
        if (row < live && t < D) {
          const float ll = (red[row] + red[N + row]) + (red[2 * N + row] + red[3 * N + row]);
          if (w.n_split == 1) {
            const int gr = w.r0 + row, tk = gr / a.G;
            const size_t orow = (static_cast<size_t>(w.q.q0) + tk) * a.hq + hk * a.G + gr - tk * a.G;
            const bool any = ll > 0.f || ll != ll;
            a.out[orow * D + t] = __float2bfloat16_rn(any ? o[r] / ll : 0.f);
            if (a.lse && t == 0)
              a.lse[orow] = any ? (rows.m[row] - kLift + log2f(ll)) * 0.693147180559945f : -INFINITY;
          } else {
            ws.o[(prow + row) * D + t] = o[r];
            if (t == 0) ws.ml[prow + row] = make_float2(rows.m[row], ll);
          }
        }
      }
      __syncwarp();
    }
    if (w.n_split > 1) __threadfence();
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (warp == kMma) tmem_dealloc(tmem, L_::kTmem);
  if (w.n_split == 1) return;

  // the last CTA of the tile to arrive joins the splits, in their order
  const size_t tile_id = (static_cast<size_t>(b) * c.hkv + hk) * pl.row_tiles + rt;
  if (threadIdx.x == 0) {
    s_last = atomicAdd(ws.count + tile_id, 1u) == static_cast<unsigned>(w.n_split - 1);
    if (s_last) ws.count[tile_id] = 0;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int e = threadIdx.x; e < (w.r1 - w.r0) * (D / 4); e += L_::kThreads) {
    const int row = e / (D / 4), gr = w.r0 + row, tk = gr / a.G;
    join_row<D>(a, ws, tile_id * pl.splits * N + row, N, w.n_split,
                (static_cast<size_t>(w.q.q0) + tk) * a.hq + hk * a.G + gr - tk * a.G, e % (D / 4));
  }
}

template <int D, int N>
cudaError_t launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const CUtensorMap& k_map, int n_sm,
                   cudaStream_t s) {
  static std::atomic<size_t> done[kMaxDevices];
  const void* fn = reinterpret_cast<const void*>(attn_few_kernel<D, N>);
  if (const cudaError_t e = opt_in_smem(fn, done, Lay<D, N>::kSmem); e != cudaSuccess) return e;
  Plan pl;
  const int64_t rows = static_cast<int64_t>(c.max_q) * a.G;
  pl.row_tiles = static_cast<int>((rows + N - 1) / N);
  const int64_t base = static_cast<int64_t>(pl.row_tiles) * c.hkv * c.n_seqs;
  const int64_t tiles = max_key_tiles(c, a, N, kKeys);
  const int64_t resident = static_cast<int64_t>(n_sm) * (N == 16 ? 2 : 1);
  const int64_t splits = best_splits(base, resident, tiles, static_cast<int64_t>(ws.cap_rows) / (base * N));
  pl.tiles_per_split = static_cast<int>((tiles + splits - 1) / splits);
  pl.splits = static_cast<int>((tiles + pl.tiles_per_split - 1) / pl.tiles_per_split);
  const int64_t grid = base * pl.splits;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  attn_few_kernel<D, N><<<static_cast<unsigned>(grid), Lay<D, N>::kThreads, Lay<D, N>::kSmem, s>>>(c, a, ws, pl, k_map);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_few_launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const KvMaps& maps,
                            int n_sm, cudaStream_t s) {
  const bool small = static_cast<int64_t>(c.max_q) * a.G <= 16;
  if (c.D == 128)
    return small ? launch<128, 16>(c, a, ws, maps.k_tile, n_sm, s) : launch<128, 64>(c, a, ws, maps.k_tile, n_sm, s);
  return small ? launch<64, 16>(c, a, ws, maps.k_tile, n_sm, s) : launch<64, 64>(c, a, ws, maps.k_tile, n_sm, s);
}

}  // namespace moe
