// Attention over the 8-bit cache for many rows (prompts, chunks, verification of
// several tokens) on tcgen05.
//
// Mathematics.  Row r (a query head of a new token) sees keys j with logits
// s_j = scale * q . k_j.  With the block's value scale v_j in the exponent,
// w_j = 2^(s_j log2 e + log2 v_j - m + lift), the output is
//   o = sum_j w_j c_j / sum_j (w_j / v_j),   c_j the value's e4m3 code,
// an online softmax whose reference m moves only when it would grow by 2^5.
//
// One CTA takes 256 rows (a row is a query head of a token; the heads that
// share a kv head are packed into the rows, so K and V are read once for all
// of them) as two M = 128 tiles, and walks over 128-key tiles:
//   1 warp    TMA: key codes into the swizzled operand layout (three stages),
//             value codes as they lie (two stages), the blocks' scales
//   2 warps   value codes -> f16 (exact) in the swizzled operand layout
//   1 thread  tcgen05.mma: S = Q K^T in e4m3, then O += P V in f16 (P from
//             tensor memory, V as it lies, MN-major)
//   2 x 8     softmax warps, two groups a M tile, two threads a row, 64 keys
//             each: S from tensor memory, weights back as f16 over S
// Keys are multiplied as they are stored: a bf16 query (8 bits) is the sum of
// two e4m3 numbers of 4 bits each, exact down to 2^-18 of the row's largest,
// and e4m3 products run at twice the rate of f16 ones, so the two terms cost
// what one f16 product would and no key is converted.  Values stay f16
// operands: a weight of 11 bits would be three e4m3 terms.
// The two M tiles take turns, so one's softmax runs under the other's products.
// Tensor memory: S0, S1, O0, O1: 512 columns.  P stands in the second half of
// either 64 columns of S that a thread holds: the first half's second read is
// under way when the first weights are stored, and nothing orders a store behind
// a load of the same columns but a wait for it.
// The tensor pipe has 1024 clocks of products a tile and M tile of heads of 128
// (64 a step of M = N = 128; S two terms of four e4m3 steps, O eight f16 ones),
// the softmax warps about as many issue slots (a multiply-add, an exponential, a
// share of the sum, the maximum, the conversion and the tensor memory's traffic
// a logit).  What bounds it is the chain S -> weights -> O of either M tile, of
// which only two are under way: 696 us for a prompt of 8192 tokens with 48 query
// and 8 kv heads of 128, 1185 TFLOP/s, about half of the pipe's rate.  Of a
// tile's 3500 clocks 1024 are products, 1900 softmax and the rest the way from
// one to the other; a CTA's beginning and end cost as much as five tiles.  Heads
// of 64 have half the products to the same softmax: 716 TFLOP/s (16384 tokens).
// 20 warps leave 96 registers a thread (and 4 to 36 bytes of them spilt); two
// conversion warps instead of four (80 registers) brought 729 us down to 718 us at
// the time.
#include "attn_tc.cuh"

namespace moe {
namespace {

constexpr int kM = 128;        // rows of an M tile
constexpr int kRows = 2 * kM;  // rows of a CTA
constexpr int kSoftmax = 512;              // threads: 2 M tiles x 2 halves of the keys x 128 rows
constexpr int kConvert = 64;               // two conversion warps
constexpr int kThreads = kSoftmax + kConvert + 64;  // MMA warp, load warp
constexpr int kMmaWarp = (kSoftmax + kConvert) / 32;
constexpr int kKStages = 3;
constexpr int kPAt = 32;  // P's first column of the 64 columns of S that a thread holds

template <int D>
using Io = TileIo<D, kKStages, 2, 2, kConvert>;

template <int D>
struct Lay {
  static constexpr int kMat8 = Io<D>::kMat8, kMat = Io<D>::kMat;
  static constexpr int kQ = 0;                     // two M tiles of two terms
  static constexpr int kK = kQ + 4 * kMat8;
  static constexpr int kV = kK + kKStages * kMat8;
  static constexpr int kRaw = kV + 2 * kMat;
  static constexpr int kConst = kRaw + 2 * kMat8;
  static constexpr int kPair = kConst + kConstRing * 8 * 16;  // [2][2][2][128] floats between a row's threads
  static constexpr int kBar = kPair + 2 * 2 * 2 * 128 * 4;
  static constexpr int kEnd = kBar + 32 * 8;
  static constexpr int kSmem = kEnd + 1024;        // the base is rounded up to 1024
};

enum Bar {
  kQFull = 0,
  kKFull = 1,    // [3] key codes
  kKEmpty = 4,   // [3]
  kRFull = 7,    // [2] value codes
  kREmpty = 9,   // [2]
  kVFull = 11,   // [2] values
  kVEmpty = 13,  // [2]
  kSFull = 15,   // [2] by M tile
  kPFull = 17,
  kOFull = 19,   // [2]
  kCFull = 21,   // [8] scales
  kDrain = 29,
  kBars = 30
};

// DUAL: calls whose sequences have at most 128 rows a kv head.  The two M tiles
// are the same rows then, each with every other tile of keys and with sums of
// its own, which the join takes for two splits: one's softmax still runs under
// the other's products.  48 rows a kv head (four sequences of up to 131072
// keys, 4 kv heads): 142 us, and 198 us as one M tile.
template <int D, bool DUAL>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles_kernel(const KvView c, const AttnArgs a, const AttnWs ws, const Plan pl,
                      const __grid_constant__ CUtensorMap k_map) {
  using L_ = Lay<D>;
  extern __shared__ char smem_raw[];
  __shared__ uint32_t s_tmem;
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base_u = smem_u32(smem);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), wg = warp >> 2, lane = threadIdx.x & 31;

  // long tiles first: the last rows of a causal prompt see the most keys
  int idx = blockIdx.x;
  const int hk = idx % c.hkv;
  idx /= c.hkv;
  const int b = idx % c.n_seqs;
  idx /= c.n_seqs;
  const int split = idx % pl.splits;
  const int rt = pl.row_tiles - 1 - idx / pl.splits;
  Work w;
  if (!work_of<kRows>(c, a, pl, b, hk, rt, w) || split >= w.n_split) return;
  const int t_begin = split * pl.tiles_per_split;
  const int t_end = min(w.k.n_t, t_begin + pl.tiles_per_split);
  const int n = t_end - t_begin;  // 0 when the rows see nothing
  const int n_mt = DUAL || w.r1 - w.r0 > kM ? 2 : 1;

  // The softmax warps' queries are on their way while all else is set up, each
  // row to where its two terms will stand.  (This loop and the next two that run
  // once a CTA stay rolled: code met for the first time costs more to fetch than
  // to run.)
  constexpr int kLanes = D / 8, kPer = 32 / kLanes, kIts = 16 / kPer;  // lanes a row, rows a pass, passes
  const int sub = lane / kLanes, part = lane % kLanes, wrow = (warp & 7) * 16;
  const uint32_t q_tile = L_::kQ + (DUAL ? 0 : warp >> 3) * 2 * L_::kMat8;
  const uint32_t q_raw = q_tile + part / (D / 16) * L_::kMat8;
  if (n > 0 && warp < (DUAL ? 8 : 8 * n_mt)) {
#pragma unroll 2
    for (int x = 0; x < kIts; ++x) {
      const int r = wrow + x * kPer + sub, i = (DUAL ? 0 : (warp >> 3) * kM) + r;  // row of the M tile, of the CTA
      const bool in = w.r0 + i < w.r1;
      int tk, hd;
      w.row(a, in ? i : 0, tk, hd);
      cp_async16(base_u + q_raw + k_off<D>(r, part % (D / 16)),
                 a.q + (static_cast<int64_t>(w.q.q0) + tk) * a.q_stride + (static_cast<int64_t>(hk) * a.G + hd) * D +
                     8 * part,
                 in ? 16 : 0);
    }
  }

  auto bar = [&](int i) { return base_u + L_::kBar + 8 * i; };
  if (threadIdx.x == 0) {
    const int count[kBars] = {DUAL ? 256 : 256 * n_mt, 1, 1, 1, 1, 1, 1, 1, 1, kConvert, kConvert, kConvert, kConvert,
                              1, 1, 1, 1, 256, 256, 1, 1, 8, 8, 8, 8, 8, 8, 8, 8, 1};
#pragma unroll
    for (int i = 0; i < kBars; ++i) mbar_init(bar(i), count[i]);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = s_tmem;

  const Io<D> io{base_u + L_::kK, base_u + L_::kRaw, base_u + L_::kV, smem, base_u, base_u + L_::kConst,
                 bar(kKFull), bar(kKEmpty), bar(kRFull), bar(kREmpty), bar(kVFull), bar(kCFull)};
  if (warp == kMmaWarp + 1) {
    if (lane < 8 && n > 0) io.load(c, a, w.k, b, hk, t_begin, n, &k_map, nullptr, lane);
  } else if (warp == kMmaWarp) {
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_f16(kM, kKeys);           // e4m3 is format 0 of its kind, too
      constexpr uint32_t id_o = idesc_f16(kM, D) | (1u << 16);  // V is MN-major
      const uint64_t q_desc = sdesc_k<D>(base_u + L_::kQ), k_desc = sdesc_k<D>(base_u + L_::kK);
      const uint64_t v_desc = sdesc_sw128_mn(base_u + L_::kV, Io<D>::kHalf);
      auto issue_s = [&](int i, int stage) {
        mma_s<D>(tmem + i * 128, q_desc + (DUAL ? 0 : i) * (2 * L_::kMat8 >> 4),
                 k_desc + stage * (L_::kMat8 >> 4), id_s);
        mma_commit(bar(kSFull + i));
      };
      auto k_wait = [&](int j) { return mbar_wait(bar(kKFull + j % kKStages), (j / kKStages) & 1, c.err); };
      auto issue_o = [&](int i, int j, bool first) {
        const uint32_t ot = tmem + 256 + i * 128, pt = tmem + i * 128 + kPAt;
        const uint64_t vd = v_desc + (j & 1) * (L_::kMat >> 4);
        mma_o(ot, pt, vd, id_o, first);
        mma_o(ot, pt + 64, vd + (64 * 128 >> 4), id_o, 0);  // P's halves stand as far apart as S's
      };
      bool ok = mbar_wait(bar(kQFull), 0, c.err) && k_wait(0);
      if (ok) {
        fence_after_sync();
        issue_s(0, 0);
        if (!DUAL && n_mt == 2) issue_s(1, 0);
        mma_commit(bar(kKEmpty));
      }
      if (DUAL && ok && n > 1 && (ok = k_wait(1))) {
        fence_after_sync();
        issue_s(1, 1);
        mma_commit(bar(kKEmpty + 1));
      }
      // S of tile j + 1 goes straight behind O += P V of tile j, whose P it
      // overwrites: one thread's products run on the tensor pipe in the order of
      // their issue.  (Waiting for the product before issuing S costs a commit's
      // and a wait's latency, about 1000 clocks a tile: prompt of 8192, 822 us
      // to 1009 us; with a thread that looks in turn which M tile can go on,
      // 695 us to 884 us.)
      for (int j = 0; DUAL && ok && j < n; ++j) {
        const int i = j & 1, next = j + 2;
        ok = mbar_wait(bar(kPFull + i), (j >> 1) & 1, c.err) && mbar_wait(bar(kVFull + i), (j >> 1) & 1, c.err);
        if (!ok) break;
        fence_after_sync();
        issue_o(i, j, j < 2);
        mma_commit(bar(kVEmpty + i));
        if (next >= n) {
          mma_commit(bar(kOFull + i));
        } else if ((ok = k_wait(next))) {
          fence_after_sync();
          issue_s(i, next % kKStages);
          mma_commit(bar(kKEmpty + next % kKStages));
        }
      }
      for (int j = 0; !DUAL && ok && j < n; ++j) {
        for (int i = 0; ok && i < n_mt; ++i) {
          ok = mbar_wait(bar(kPFull + i), j & 1, c.err) &&
               (i > 0 || mbar_wait(bar(kVFull + (j & 1)), (j >> 1) & 1, c.err));
          if (!ok) break;
          fence_after_sync();
          issue_o(i, j, j == 0);
          if (i == n_mt - 1) mma_commit(bar(kVEmpty + (j & 1)));
          if (j == n - 1) {
            mma_commit(bar(kOFull + i));
          } else if ((ok = i > 0 || k_wait(j + 1))) {
            fence_after_sync();
            issue_s(i, (j + 1) % kKStages);
            if (i == n_mt - 1) mma_commit(bar(kKEmpty + (j + 1) % kKStages));
          }
        }
      }
      if (!ok) {
        // what was issued ends by itself; wait for it before the tensor memory goes back
        mma_commit(bar(kDrain));
        mbar_wait(bar(kDrain), 0, c.err);
      }
    }
  } else if (wg == 4) {
    io.convert(c, a, w.k, t_begin, n, threadIdx.x - kSoftmax,
               [&](int j) { return mbar_wait(bar(kVEmpty + (j & 1)), ((j >> 1) & 1) ^ 1, c.err); });
  } else if ((wg >> 1) < n_mt) {
    const int i = wg >> 1, half = wg & 1, row = threadIdx.x & 127;  // M tile, half of the keys
    const int row0 = w.r0 + (DUAL ? 0 : i * kM);  // of the M tile
    const int r = row0 + row;
    const bool live = r < w.r1;
    int tok = 0, head = 0;
    if (live) w.row(a, r - w.r0, tok, head);
    head += hk * a.G;
    const RowSees sees = row_sees(a, w.q.L, w.base_p + tok, live);
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 * (warp % 4)
    const uint32_t ts = tmem + i * 128 + lanes + half * 64, to = tmem + 256 + i * 128 + lanes + half * (D / 2);
    // What the row's two threads tell each other, two buffers in turn.  A warp
    // whose wait gave up waits no more but still comes to every barrier, and the
    // loop ends for all.
    bool ok = true;
    float* pair = reinterpret_cast<float*>(smem + L_::kPair) + i * 512;
    const int mine = DUAL ? (n + 1 - i) >> 1 : n;  // tiles of this M tile
    auto other = [&](int buf, float mine) {
      pair[buf * 256 + half * 128 + row] = mine;
      ok = !named_vote(1 + i, 256, !ok);
      return pair[buf * 256 + (half ^ 1) * 128 + row];
    };
    float m = -INFINITY, l = 0.f, lscale = 0.f;  // lscale >= 0: a negative scale turns the query's sign
    if (n > 0 && (!DUAL || i == 0)) {
      // The rows' queries, each brought to [2^7, 2^8) by a power of two, as two
      // e4m3 terms: a warp takes 16 of the M tile's rows, D / 8 lanes a row.
      char* dst = smem + q_tile;
      asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
      for (int x = 0; x < kIts; ++x) {
        const int qrow = wrow + x * kPer + sub;
        const uint4 raw = *reinterpret_cast<const uint4*>(smem + q_raw + k_off<D>(qrow, part % (D / 16)));
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
        // the row's largest magnitude: as bf16 bits magnitudes order like integers (NaN above all)
        uint32_t top = __vmaxu2(__vmaxu2(u[0] & 0x7fff7fffu, u[1] & 0x7fff7fffu),
                                __vmaxu2(u[2] & 0x7fff7fffu, u[3] & 0x7fff7fffu));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float amax = __uint_as_float(max(top << 16, top & 0xffff0000u));
        const float f = copysignf(row_factor<7>(amax), a.scale_log2);
        const bool inf = !(amax < INFINITY);  // (codes saturate: such a row is NaN instead)
        uint32_t t0[2], t1[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t a1, a2, b1, b2;
          split_query(u[2 * k], f, a1, a2);
          split_query(u[2 * k + 1], f, b1, b2);
          t0[k] = inf ? 0x7f7f7f7fu : a1 | (b1 << 16);
          t1[k] = a2 | (b2 << 16);
        }
        __syncwarp();  // the row's lanes have read it
        const uint32_t off = k_off<D>(qrow, part >> 1) + 8 * (part & 1);
        *reinterpret_cast<uint2*>(dst + off) = make_uint2(t0[0], t0[1]);
        *reinterpret_cast<uint2*>(dst + L_::kMat8 + off) = make_uint2(t1[0], t1[1]);
        if (part == 0) pair[256 + qrow] = fabsf(a.scale_log2) * inverse(fabsf(f));
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kQFull));
    }
    // (both barriers of one count: the second comes before the pair buffers' first use)
    auto all_sync = [&]() { DUAL ? named_sync(3, 512) : named_sync(1 + i, 256); };
    if (n > 0) {
      all_sync();
      lscale = reinterpret_cast<const float*>(smem + L_::kPair)[(DUAL ? 0 : i * 512) + 256 + row];
      all_sync();
    }
    // the range that all rows of the CTA see whole
    const int p_lo = w.p_lo, p_hi = w.p_hi;
    for (int t = 0; t < mine; ++t) {
      const int j = DUAL ? 2 * t + i : t;
      // (S of this tile says that O += P V of the tile before is done, too)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(kCFull + j % kConstRing), (j / kConstRing) & 1, c.err) &&
                                       mbar_wait(bar(kSFull + i), t & 1, c.err));
      fence_after_sync();
      const float4* cn = io.scales(j) + 4 * half;
      const int base = w.k.base(t_begin + j) + 64 * half;
      const bool whole = (a.causal ? base + 64 <= p_lo + 1 : base + 64 <= w.q.L) &&
                         (a.window == 0 || base > p_hi - a.window || base + 64 <= a.sinks);
      // S is read in halves of 32 keys, the first of them twice: for the row's
      // largest logit (within 16 keys of one scale the largest product gives
      // it), then for the weights
      float s[32];
      float mt = -INFINITY;
      auto hide = [&](int x) {
        const uint32_t seen = sees.bits(base + 32 * x);
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k] = seen & (1u << k) ? s[k] : -INFINITY;
      };
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        tmem_ld32(ts + 32 * x, s);
        tmem_wait_ld32(s);
        if (!whole) hide(x);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const float4 z = cn[2 * x + gg];
          const float* v = s + 16 * gg;
          float t0 = max3(v[0], v[1], v[2]), t1 = max3(v[3], v[4], v[5]);
          t0 = max3(t0, v[6], v[7]), t1 = max3(t1, v[8], v[9]);
          t0 = max3(t0, v[10], v[11]), t1 = max3(t1, v[12], v[13]);
          t0 = max3(t0, v[14], v[15]);
          mt = fmaxf(mt, fmaf(fmaxf(t0, t1), fmaxf(lscale * z.x, kTiny), z.y));
        }
      }
      mt = fmaxf(mt, other(t & 1, mt));
      if (!ok) break;
      if (__any_sync(0xffffffffu, mt > m + kRescale)) {
        const float nm = fmaxf(m, mt);
        const float f = nm == m ? 1.f : ex2(m - nm);
        m = nm;
        l *= f;
        if (t > 0) {
          // half of the output's columns a thread
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t u[16];
            tmem_ld16(to + 16 * x, u);
            tmem_wait_ld16(u);
#pragma unroll
            for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * f);
            tmem_st16(to + 16 * x, u);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.f : m - kLift;
      auto weigh = [&](int x) {
        uint32_t u[16];
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const float4 z = cn[2 * x + gg];
          const float sc = fmaxf(lscale * z.x, kTiny), off = z.y - ref;
          const float* v = s + 16 * gg;
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float w0, w1;
            fma2(w0, w1, v[k], v[k + 1], sc, off);
            w0 = ex2(w0), w1 = ex2(w1);
            add2(sum0, sum1, w0, w1);
            // (f16's 11 bits for the product: an output's error stays below its own rounding to
            // bf16's 8; the sum takes the weights as they are)
            u[8 * gg + k / 2] = half2_bits(w0, w1);
          }
          l = fmaf(sum0 + sum1, z.z, l);
        }
        // P takes the second half of this thread's S columns, those of keys 32 .. 63: they are in
        // registers or used up, while the load of the first half is still under way
        if (x == 1) tmem_ld32(ts, s);
        tmem_st16(ts + kPAt + 16 * x, u);
      };
      weigh(1);
      tmem_wait_ld32(s);
      if (!whole) hide(0);
      weigh(0);
      tmem_wait_st();
      fence_before_sync();
      mbar_arrive(bar(kPFull + i));
    }
    if (ok && mine > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(kOFull + i), 0, c.err));
    if (mine > 0) l += other(mine & 1, l);
    if (ok) {
      fence_after_sync();
      const size_t orow = (static_cast<size_t>(w.q.q0) + tok) * a.hq + head;
      const size_t prow =
          (((static_cast<size_t>(b) * c.hkv + hk) * pl.row_tiles + rt) * pl.splits + split) * kRows + i * kM + row;
      // A thread's half row goes through shared memory (the queries' room: the
      // last S of either M tile came before this O), D bytes a row, so that the
      // warp's stores are whole lines: D / 2 bf16 elements in one go, or fp32
      // partial sums in two.
      const bool any = l > 0.f || l != l;
      const float f = any ? 1.f / l : 0.f;
      char* stage = smem + L_::kQ + warp * (32 * D);
      const uint32_t olo = static_cast<uint32_t>(orow);
      const bool parts = DUAL || w.n_split > 1;
      constexpr int kCols = D / 4;  // columns a round
#pragma unroll 1
      for (int y = 0; y < 2; ++y) {
        float o[kCols];
#pragma unroll
        for (int k = 0; k < kCols; ++k) o[k] = 0.f;
        if (mine > 0) {
          if constexpr (D == 128) {
            tmem_ld32(to + kCols * y, o);
            tmem_wait_ld32(o);
          } else {
            tmem_ld16f(to + kCols * y, o);
            tmem_wait_ld16f(o);
          }
        }
        if (parts) {
#pragma unroll
          for (int k = 0; k < kCols / 4; ++k)
            *reinterpret_cast<uint4*>(stage + k_off<D>(lane, k)) =
                make_uint4(__float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]),
                           __float_as_uint(o[4 * k + 3]));
        } else {
#pragma unroll
          for (int k = 0; k < kCols / 8; ++k) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(o[8 * k + 2 * e] * f, o[8 * k + 2 * e + 1] * f);
              h[e] = *reinterpret_cast<const uint32_t*>(&x);
            }
            *reinterpret_cast<uint4*>(stage + k_off<D>(lane, y * (kCols / 8) + k)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        if (parts || y == 1) {
          __syncwarp();
          constexpr int kChunks = D / 16;  // 16-byte chunks of a row
          const int cc = lane % kChunks;
#pragma unroll
          for (int e = 0; e < kChunks; ++e) {
            const int rr = e * (32 / kChunks) + lane / kChunks;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + k_off<D>(rr, cc));
            const uint32_t to_row = __shfl_sync(0xffffffffu, olo, rr);
            if (__shfl_sync(0xffffffffu, static_cast<int>(live), rr)) {
              if (parts)
                *reinterpret_cast<uint4*>(ws.o + (prow - lane + rr) * D + half * (D / 2) + kCols * y + 4 * cc) = v;
              else
                *reinterpret_cast<uint4*>(a.out + static_cast<size_t>(to_row) * D + half * (D / 2) + 8 * cc) = v;
            }
          }
          __syncwarp();
        }
      }
      if (live && half == 0 && !parts && a.lse)
        a.lse[orow] = any ? (m - kLift + log2f(l)) * 0.693147180559945f : -INFINITY;
      if (live && half == 0 && parts) ws.ml[prow] = make_float2(m, l);
    }
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Joins the splits (and the M tiles of DUAL) of every row that has more than one.
constexpr int kJoinThreads = 256;
template <int D, bool DUAL>
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
  if (b >= c.n_seqs || !work_of<kRows>(c, a, pl, b, hk, rt, w) || (!DUAL && w.n_split == 1) || w.r0 + row >= w.r1) return;
  int tok, head;
  w.row(a, row, tok, head);
  const size_t orow = (static_cast<size_t>(w.q.q0) + tok) * a.hq + hk * a.G + head;
  join_row<D>(a, ws, static_cast<size_t>(tile_id) * pl.splits * kRows + row, DUAL ? kM : kRows,
              DUAL ? 2 * w.n_split : w.n_split, orow, threadIdx.x % (D / 4));
}

template <int D, bool DUAL>
cudaError_t launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const CUtensorMap& k_map, int n_sm,
                   cudaStream_t s) {
  static std::atomic<size_t> done[kMaxDevices];
  const void* fn = reinterpret_cast<const void*>(attn_tiles_kernel<D, DUAL>);
  if (const cudaError_t e = opt_in_smem(fn, done, Lay<D>::kSmem); e != cudaSuccess) return e;
  Plan pl;
  const int64_t rows = static_cast<int64_t>(c.max_q) * a.G;
  pl.row_tiles = static_cast<int>((rows + kRows - 1) / kRows);
  const int64_t base = static_cast<int64_t>(pl.row_tiles) * c.hkv * c.n_seqs;
  const int64_t tiles = max_key_tiles(c, a, kRows, kKeys);
  // one CTA a SM: split the keys when the row tiles do not fill the SMs evenly
  const int64_t most = static_cast<int64_t>(ws.cap_rows) / (base * kRows);
  const int64_t splits = best_splits(base, n_sm, tiles, most, c.n_seqs > 1, {1, 6., 1. / 32});
  pl.tiles_per_split = static_cast<int>((tiles + splits - 1) / splits);
  pl.splits = static_cast<int>((tiles + pl.tiles_per_split - 1) / pl.tiles_per_split);
  const int64_t grid = base * pl.splits;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  attn_tiles_kernel<D, DUAL><<<static_cast<unsigned>(grid), kThreads, Lay<D>::kSmem, s>>>(c, a, ws, pl, k_map);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!DUAL && pl.splits == 1)) return e;
  const int64_t items = base * kRows, per = kJoinThreads / (D / 4);
  attn_join_kernel<D, DUAL><<<static_cast<unsigned>((items + per - 1) / per), kJoinThreads, 0, s>>>(c, a, ws, pl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_tiles_launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const KvMaps& maps,
                              int n_sm, cudaStream_t s) {
  // (the two M tiles' sums have to fit the workspace)
  const bool dual = static_cast<int64_t>(c.max_q) * a.G <= kM &&
                    static_cast<size_t>(c.n_seqs) * c.hkv * kRows <= ws.cap_rows;
  if (c.D == 128) return (dual ? launch<128, true> : launch<128, false>)(c, a, ws, maps.k_tile, n_sm, s);
  return (dual ? launch<64, true> : launch<64, false>)(c, a, ws, maps.k_tile, n_sm, s);
}

}  // namespace moe
