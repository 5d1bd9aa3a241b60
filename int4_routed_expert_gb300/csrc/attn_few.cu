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
// A CTA takes N = 16 or 32 rows of a kv head and walks over tiles of 128
// keys, multiplied as they are stored:
//   S^T[128 keys x 2 N]   = K [Q1; Q2]^T         the bf16 query as two e4m3 terms
//   P[128 keys x 4 N]                            a thread a key
//   O^T[128 dims x 4 N]  += V^T [P1 P2 P3 P4]    V as it lies (M-major)
// A weight is rounded to f16 (11 bits) and cut into e4m3 terms of 4 bits, term
// i scaled by 32^(i - 1) into its own accumulator columns: exact for weights
// above 2^-15 of the row's largest, and to 2^-29 of the largest below (the
// lift of 5 and the reference within 2^3 of the largest see to that).  So no
// value is converted, shared memory carries each code once in and once out,
// and the extra columns are free: with the keys and dims in M the products are
// bound by reading K and V, whatever N is.  A thread's block scales are
// scalars, it writes its key's weights as they stand in one operand row, and
// no thread shuffles: only when a reference moves, the maxima over the keys
// are exchanged.  The keys are split over CTAs; the last CTA of a row tile to
// arrive joins them, in their order.
// Warps: 4 softmax for every 16 rows, MMA, load.
// Bound by memory: 2 D bytes a key and kv head.  64 sequences of up to 16384
// keys, 64 query and 8 kv heads of 128: 208 us, 5.1 TB/s; 32 rows a kv head
// (16 x 16384 keys, 4 kv heads) 89 us, 3.0 TB/s, where a tile's chain S -> weights
// -> O, twice as much softmax, bounds it; two such CTAs a SM leave 96 registers a
// thread, and 60 bytes are spilt.
#include "attn_tc.cuh"

namespace moe {
namespace {

constexpr float kFewLift = 5.f, kFewRescale = 3.f;  // weights below 2^8: an e4m3 ends at 448

enum Bar {
  kQFull = 0,
  kKFull = 1,    // [3] key codes
  kKEmpty = 4,   // [3]
  kVFull = 7,    // [3] value codes
  kVEmpty = 10,  // [3]
  kSFull = 13,   // [2] S^T
  kPFull = 15,   // P
  kODone = 16,   // O^T += V^T P
  kCFull = 17,   // [8] scales
  kDrain = 25,
  kJoin = 26,    // [2] partial results
  kBars = 28
};

// Most splits of a call: the join holds a reference and a sum of each and row.
constexpr int max_splits(int n) { return 4096 / n; }

// A CTA keeps to half an SM, so that two CTAs cover each other's bubbles.
template <int D, int N>
struct Lay {
  static constexpr int kStages = N == 16 ? 3 : 2;  // of key codes and of value codes
  static constexpr int kCtas = 2;                        // a SM
  using Io = TileIo<D, kStages, kStages, 0>;
  static constexpr int kGroups = N / 16;  // softmax groups of 128 threads
  static constexpr int kThreads = 128 * kGroups + 64;
  static constexpr int kQ = 0;            // [2 N][D]
  static constexpr int kK = kQ + (2 * N * D + 1023) / 1024 * 1024;
  static constexpr int kV = kK + kStages * Io::kMat8;
  static constexpr int kP = kV + kStages * Io::kMat8;  // [128 keys][4 N]
  static constexpr int kConst = kP + kKeys * 4 * N;
  static constexpr int kRow = kConst + kConstRing * 8 * 16;  // [7][N]: see Rows
  static constexpr int kRed = kRow + 7 * N * 4;              // [4][N] floats
  static constexpr int kBar = kRed + 4 * N * 4;
  static constexpr int kSmem = kBar + kBars * 8 + 1024;
  static constexpr int kTmem = 8 * N;                        // S^T twice, then O^T
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
  int* out;       // row of the output
  __device__ __forceinline__ explicit Rows(char* p)
      : lscale(reinterpret_cast<float*>(p)), nref(lscale + N), m(nref + N), f(m + N),
        lo(reinterpret_cast<int*>(f + N)), hi(lo + N), out(hi + N) {}
};

// P's operand layout: a key's terms in a row of 4 N bytes, term by term; rows
// of 64 or 128 bytes, swizzled.
// Byte offset of 16-byte chunk c of a key.
template <int N>
__device__ __forceinline__ uint32_t p_off(int key, int c) {
  if constexpr (N == 16) return key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
  return key * 128 + ((c ^ (key & 7)) << 4);
}

// MN-major operand of e4m3 codes: rows of `row` (64 or 128) bytes along M or N
// a key, swizzled in rows; 8-key atoms of 8 rows; the next block of rows `lead`
// bytes on.
__device__ __forceinline__ uint64_t sdesc_mn8(uint32_t smem_addr, uint32_t row, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((8 * row) >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(row == 128 ? 2u : 4u) << 61;
  return d;
}

// O^T[tmem] (+)= V^T[smem] P[smem] over 128 keys, 32 a step: both operands
// MN-major, VSTEP and PSTEP bytes a step.
template <int VSTEP, int PSTEP>
__device__ __forceinline__ void mma_ot(uint32_t d_tmem, uint64_t v_desc, uint64_t p_desc, uint32_t idesc,
                                       uint32_t first) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 v<4>, b<4>;\n\t"
      "setp.eq.b32 p, %4, 0;\n\t"
      "add.s64 v1, %1, %5;\n\tadd.s64 v2, v1, %5;\n\tadd.s64 v3, v2, %5;\n\t"
      "add.s64 b1, %2, %6;\n\tadd.s64 b2, b1, %6;\n\tadd.s64 b3, b2, %6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], v1, b1, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], v2, b2, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], v3, b3, %3, 1;\n\t}" ::"r"(d_tmem),
      "l"(v_desc), "l"(p_desc), "r"(idesc), "r"(first), "n"(static_cast<uint64_t>(VSTEP) >> 4),
      "n"(static_cast<uint64_t>(PSTEP) >> 4)
      : "memory");
}

// Two weights below 2^8 as four e4m3 pairs: h = t0 + t1 / 32 + t2 / 32^2 + t3 / 32^3
// (a term is off by at most 2^-5 of its binade, 8 at 2^8, and 8 * 32 is below 448).
__device__ __forceinline__ void split_weights(float w0, float w1, uint16_t (&t)[4]) {
  asm("{\n\t.reg .b32 h, k, n, b;\n\t"
      "cvt.rn.f16x2.f32 h, %5, %4;\n\t"
      "mov.b32 k, 0x50005000;\n\tmov.b32 n, 0xd000d000;\n\t"  // 32, -32
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, h;\n\tcvt.rn.f16x2.e4m3x2 b, %0;\n\t"
      "mul.rn.f16x2 h, h, k;\n\tfma.rn.f16x2 h, b, n, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %1, h;\n\tcvt.rn.f16x2.e4m3x2 b, %1;\n\t"
      "mul.rn.f16x2 h, h, k;\n\tfma.rn.f16x2 h, b, n, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %2, h;\n\tcvt.rn.f16x2.e4m3x2 b, %2;\n\t"
      "mul.rn.f16x2 h, h, k;\n\tfma.rn.f16x2 h, b, n, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %3, h;\n\t}"
      : "=&h"(t[0]), "=&h"(t[1]), "=&h"(t[2]), "=&h"(t[3])
      : "f"(w0), "f"(w1));
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

// Two waits whose first looks overlap.
__device__ __forceinline__ bool mbar_wait2(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, int* err) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(b0), "r"(p0), "r"(b1), "r"(p1)
      : "memory");
  return ok != 0 || (mbar_wait(b0, p0, err) && mbar_wait(b1, p1, err));
}

template <int D, int N>
__global__ void __launch_bounds__(Lay<D, N>::kThreads, Lay<D, N>::kCtas)
    attn_few_kernel(const KvView c, const AttnArgs a, const AttnWs ws, const Plan pl,
                    const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
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
    constexpr int kS = 128 * L_::kGroups, kG = L_::kGroups;
    const int count[kBars] = {kS, 1, 1, 1, kG, kG, kG, 1, 1, 1, 1, 1, 1, 1,
                              1,  kS, 1, 8, 8, 8, 8, 8, 8, 8, 8, 1, 1, 1};
#pragma unroll
    for (int i = 0; i < kBars; ++i) mbar_init(bar(i), count[i]);
    fence_barrier_init();
  }
  constexpr int kMma = 4 * L_::kGroups;  // the MMA warp; then the load warp
  if (warp == kMma) {
    tmem_alloc(smem_u32(&s_tmem), L_::kTmem);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = s_tmem;
  const uint32_t ot = tmem + 4 * N;  // S^T: columns 0 .. 4 N - 1
  const Io io{base_u + L_::kK, base_u + L_::kV, 0, smem, base_u, base_u + L_::kConst,
              bar(kKFull), bar(kKEmpty), bar(kVFull), bar(kVEmpty), 0, bar(kCFull)};
  const Rows<N> rows(smem + L_::kRow);

  if (warp == kMma + 1) {
    if (lane < 8 && n > 0) io.load(c, a, w.k, b, hk, t_begin, n, &k_map, &v_map, lane);
  } else if (warp == kMma) {
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_f16(kKeys, 2 * N);                      // e4m3 is format 0 of its kind, too
      constexpr uint32_t id_o = idesc_f16(128, 4 * N) | (1u << 15) | (1u << 16);  // both MN-major
      const uint64_t q_desc = sdesc_k<D>(base_u + L_::kQ), k_desc = sdesc_k<D>(base_u + L_::kK);
      // heads of 64: the accumulator's other 64 rows take the codes one atom on, and are not read
      const uint64_t v_desc = sdesc_mn8(base_u + L_::kV, D, 8 * D);
      const uint64_t p_desc = sdesc_mn8(base_u + L_::kP, 4 * N, 16);
      constexpr int kVStep = 32 * D, kPStep = 32 * 4 * N;
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
        const int vs = j % L_::kStages;
        ok = mbar_wait(bar(kPFull), j & 1, c.err) && mbar_wait(bar(kVFull + vs), (j / L_::kStages) & 1, c.err);
        if (!ok) break;
        fence_after_sync();
        mma_ot<kVStep, kPStep>(ot, v_desc + vs * (Io::kMat8 >> 4),
                             p_desc, id_o, j == 0);
        mma_commit(bar(kODone));
        ok = j + 2 >= n || issue_s(j + 2);
      }
      if (!ok) {
        // what was issued ends by itself; wait for it before the tensor memory goes back
        mma_commit(bar(kDrain));
        mbar_wait(bar(kDrain), 0, c.err);
      }
    }
  } else {
    // ---- softmax: thread t is key t of a tile -----------------------------------
    constexpr int NG = 16;
    const int t = threadIdx.x & 127, grp = warp >> 2, g0 = grp * NG;  // rows g0 .. of the group
    float l[NG];
#pragma unroll
    for (int r = 0; r < NG; ++r) l[r] = 0.f;
    // the rows' queries as two e4m3 terms, 128 kGroups / N threads a row
    {
      constexpr int kPer = 128 * L_::kGroups / N, kDims = D / kPer;  // threads a row, dims a thread
      const int r = threadIdx.x / kPer, part = threadIdx.x % kPer, gr = w.r0 + r;
      const bool live = gr < w.r1;
      int tok = 0, head = 0;
      if (live) w.row(a, r, tok, head);
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<int64_t>(w.q.q0) + tok) * a.q_stride +
          (static_cast<int64_t>(hk) * a.G + head) * D + part * kDims);
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
        rows.out[r] = (w.q.q0 + tok) * a.hq + hk * a.G + head;
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kQFull));
    }
    named_sync(8, 128 * L_::kGroups);
    const int p_lo = w.p_lo, p_hi = w.p_hi;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane 32 * (warp % 4)
    float* red = reinterpret_cast<float*>(smem + L_::kRed);
    bool ok = true, pending = true;  // a row has no reference yet
    for (int j = 0; j < n; ++j) {
      const int bf = j & 1;
      // (a thread whose wait gave up waits no more; the vote below ends the loop)
      ok = ok && mbar_wait2(bar(kSFull + bf), (j >> 1) & 1, bar(kCFull + j % kConstRing), (j / kConstRing) & 1, c.err);
      __syncwarp();
      fence_after_sync();
      const uint32_t st = tmem + bf * 2 * N + lanes + g0;
      float z[NG], s2[NG];
      tmem_ld16f(st, z);
      tmem_ld16f(st + N, s2);
      const float4 cn = io.scales(j)[t >> 4];
      const float ks = fmaxf(cn.x, kTiny);
      const int tok = w.k.base(t_begin + j) + t, key0 = tok - t;
      const bool whole = (a.causal ? key0 + kKeys <= p_lo + 1 : key0 + kKeys <= w.q.L) &&
                         (a.window == 0 || key0 > p_hi - a.window || key0 + kKeys <= a.sinks);
      // exponents relative to the rows' references
      float top = -INFINITY;
      tmem_wait_ld16f(z);
      tmem_wait_ld16f(s2);
#pragma unroll
      for (int r = 0; r < NG; r += 4) {
        const float4 ls = *reinterpret_cast<const float4*>(rows.lscale + g0 + r);
        const float4 nr = *reinterpret_cast<const float4*>(rows.nref + g0 + r);
        float* y = z + r;
        add2(y[0], y[1], s2[r], s2[r + 1]);
        add2(y[2], y[3], s2[r + 2], s2[r + 3]);
        float m0, m1, m2, m3, b0 = nr.x, b1 = nr.y, b2 = nr.z, b3 = nr.w;
        mul2(m0, m1, ls.x, ls.y, ks);
        mul2(m2, m3, ls.z, ls.w, ks);
        add2(b0, b1, cn.y, cn.y);
        add2(b2, b3, cn.y, cn.y);
        fma2(y[0], y[1], y[0], y[1], m0, m1, b0, b1);
        fma2(y[2], y[3], y[2], y[3], m2, m3, b2, b3);
      }
      if (!whole) {
#pragma unroll
        for (int r = 0; r < NG; ++r) {
          const bool sees = tok <= rows.hi[g0 + r] && (tok >= rows.lo[g0 + r] || tok < a.sinks);
          z[r] = sees ? z[r] : -INFINITY;
        }
      }
#pragma unroll
      for (int r = 0; r < NG; r += 2) top = max3(top, z[r], z[r + 1]);
      if (named_vote(1 + grp, 128, pending || top > kFewLift + kFewRescale || !ok)) {
        ok = !named_vote(1 + grp, 128, !ok);
        if (!ok) break;
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
          const bool move = mx > m + kFewRescale;
          const float nm = move ? mx : m;
          rows.f[q] = move ? ex2(m - nm) : 1.f;
          red[q] = move ? (kFewLift - nm) - rows.nref[q] : 0.f;  // what the exponents change by
          rows.m[q] = nm;
          if (move) rows.nref[q] = kFewLift - nm;
        }
        named_sync(1 + grp, 128);
#pragma unroll
        for (int r = 0; r < NG; ++r) {
          z[r] += red[g0 + r];
          l[r] *= rows.f[g0 + r];
        }
        if (j > 0) {
          ok = mbar_wait(bar(kODone), (j - 1) & 1, c.err);
          __syncwarp();
          fence_after_sync();
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t u[16];
            tmem_ld16(ot + lanes + x * N + g0, u);
            tmem_wait_ld16(u);
#pragma unroll
            for (int r = 0; r < 16; ++r) u[r] = __float_as_uint(__uint_as_float(u[r]) * rows.f[g0 + r]);
            tmem_st16(ot + lanes + x * N + g0, u);
          }
          tmem_wait_st();
        }
        // (a barrier, too: red and f are free again)
        pending = named_vote(1 + grp, 128, t < NG && rows.m[g0 + t % NG] == -INFINITY && rows.hi[g0 + t % NG] >= 0);
      }
      // the weights, and their terms: row pairs of term i in u[i]
      uint32_t u[4][4];
#pragma unroll
      for (int r = 0; r < NG; r += 4) {
        uint16_t t0[4], t1[4];
        const float w0 = ex2(z[r]), w1 = ex2(z[r + 1]), w2 = ex2(z[r + 2]), w3 = ex2(z[r + 3]);
        fma2(l[r], l[r + 1], w0, w1, cn.z, cn.z, l[r], l[r + 1]);
        fma2(l[r + 2], l[r + 3], w2, w3, cn.z, cn.z, l[r + 2], l[r + 3]);
        split_weights(w0, w1, t0);
        split_weights(w2, w3, t1);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i][r >> 2] = t0[i] | (static_cast<uint32_t>(t1[i]) << 16);
      }
      if (grp == 0 && !whole) {
        // the values that no row sees are zero: a NaN code there would reach the rows through 0 * NaN
        ok = ok && mbar_wait(bar(kVFull + j % L_::kStages), (j / L_::kStages) & 1, c.err);
        if (!(tok < w.k.hi && (tok >= w.k.lo || tok < a.sinks))) {
          uint4* v = reinterpret_cast<uint4*>(smem + L_::kV + (j % L_::kStages) * Io::kMat8 + t * D);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) v[x] = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      // P of the tile before has been read; through with its V (once for all groups) and with K of this one
      if (j > 0) ok = ok && mbar_wait(bar(kODone), (j - 1) & 1, c.err);
      if (t == 0) {
        mbar_arrive(bar(kKEmpty + j % L_::kStages));
        if (grp == 0 && j > 0) mbar_arrive(bar(kVEmpty + (j - 1) % L_::kStages));
      }
      char* p = smem + L_::kP;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(p + p_off<N>(t, (i * N + g0) >> 4)) = make_uint4(u[i][0], u[i][1], u[i][2], u[i][3]);
      fence_proxy_async_smem();
      fence_before_sync();
      mbar_arrive(bar(kPFull));
    }
    // the weights' sums over the warp's keys: half the rows go each way at a step,
    // so that lanes r and r + 16 end with row r's halves
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
#pragma unroll
      for (int r = 0; r < o; ++r) {
        const bool up = (lane & o) != 0;
        const float give = up ? l[r] : l[r + o], keep = up ? l[r + o] : l[r];
        l[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], 16);
    if (lane < NG) red[(warp & 3) * N + g0 + lane] = l[0];
    // (a lane whose wait gave up in the last tile has had no vote since: the warp decides here,
    // as its lanes go on to loads and barriers together)
    ok = __all_sync(0xffffffffu, ok && (n == 0 || mbar_wait(bar(kODone), (n - 1) & 1, c.err)));
    fence_after_sync();
    // thread t has dim t of every row: the terms' columns, the smallest first
    float o[NG];
#pragma unroll
    for (int r = 0; r < NG; ++r) o[r] = 0.f;
    if (n > 0 && ok) {
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        float y[NG];
        tmem_ld16f(ot + lanes + i * N + g0, y);
        tmem_wait_ld16f(y);
#pragma unroll
        for (int r = 0; r < NG; ++r) o[r] = fmaf(o[r], 0.03125f, y[r]);
      }
    }
    named_sync(1 + grp, 128);
    const int live = w.r1 - w.r0;
    const size_t prow = (((static_cast<size_t>(b) * c.hkv + hk) * pl.row_tiles + rt) * pl.splits + split) * N;
    if (t < NG && g0 + t < live) {
      const int row = g0 + t;
      const float ll = (red[row] + red[N + row]) + (red[2 * N + row] + red[3 * N + row]);
      const float mm = rows.m[row] + (kLift - kFewLift);  // as the other kernel counts
      const bool any = ll > 0.f || ll != ll;
      rows.f[row] = any ? 1.f / ll : 0.f;
      if (w.n_split > 1)
        ws.ml[prow + row] = make_float2(mm, ll);
      else if (a.lse)
        a.lse[rows.out[row]] = any ? (mm - kLift + log2f(ll)) * 0.693147180559945f : -INFINITY;
    }
    named_sync(1 + grp, 128);
#pragma unroll
    for (int r = 0; r < NG; ++r) {
      const int row = g0 + r;
      if (row < live && t < D) {
        if (w.n_split == 1)
          a.out[static_cast<size_t>(rows.out[row]) * D + t] = __float2bfloat16_rn(o[r] * rows.f[row]);
        else
          ws.o[(prow + row) * D + t] = o[r];
      }
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
  // Partial results come from SMs far away: as many splits as fit are on their
  // way over the key, value and weight stages, in two groups that take turns, a
  // lane a split, while the splits' factors are worked out.
  constexpr int kEach = (N * (D / 4) + L_::kThreads - 1) / L_::kThreads;
  constexpr int kRoom = L_::kConst - L_::kK;
  static_assert(kRoom - max_splits(N) * N * 8 >= 2 * N * D * 4, "a split in either group");
  const int live = w.r1 - w.r0;
  const int ml_bytes = w.n_split * N * 8, bytes = live * D * 4;
  const int group = (kRoom - ml_bytes) / (2 * bytes);
  const size_t first = tile_id * pl.splits * N;
  const uint32_t parts = L_::kK + ml_bytes;  // [2][group][live][D], behind [n_split][N] factors
  auto fetch = [&](int s0, int buf) {
    const int m = min(group, w.n_split - s0);
    if (lane == 0) mbar_arrive_expect_tx(bar(kJoin + buf), m * bytes);
    __syncwarp();
    for (int s = lane; s < m; s += 32)
      bulk_g2s(base_u + parts + (buf * group + s) * bytes, ws.o + (first + static_cast<size_t>(s0 + s) * N) * D, bytes,
               bar(kJoin + buf));
  };
  if (warp == 0) {
    asm volatile("fence.proxy.async;" ::: "memory");  // (the results were written by other threads' plain stores)
    fetch(0, 0);
    if (group < w.n_split) fetch(group, 1);
  }
  float2* ml = reinterpret_cast<float2*>(smem + L_::kK);
#pragma unroll 4
  for (int e = threadIdx.x; e < w.n_split * N; e += L_::kThreads) ml[e] = __ldcg(ws.ml + first + e);
  __syncthreads();
  if (const int row = threadIdx.x >> 3, sub = threadIdx.x & 7; row < N) {  // eight lanes a row
    float top = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int s = sub; s < w.n_split; s += 8) top = fmaxf(top, ml[s * N + row].x);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
    for (int s = sub; s < w.n_split; s += 8) {
      const float2 x = ml[s * N + row];
      const float f = ex2(x.x - ref);
      l = fmaf(x.y, f, l);
      ml[s * N + row].x = f;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (sub == 0) rows.m[row] = top, rows.f[row] = l;
  }
  __syncthreads();
  int el[kEach], of[kEach];
  float4 v[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int e = threadIdx.x + k * L_::kThreads;
    el[k] = e < live * (D / 4) ? e : 0;
    of[k] = el[k] / (D / 4);
    v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int s0 = 0, buf = 0, ph = 0, end = w.n_split; s0 < end; s0 += group) {
    const bool landed = mbar_wait(bar(kJoin + buf), ph, c.err);
    const int m = min(group, w.n_split - s0);
    const char* at = smem + parts + buf * group * bytes;
#pragma unroll 2
    for (int s = 0; s < m; ++s) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const float f = ml[(s0 + s) * N + of[k]].x;
        const float4 z = reinterpret_cast<const float4*>(at + s * bytes)[el[k]];
        v[k].x = fmaf(z.x, f, v[k].x), v[k].y = fmaf(z.y, f, v[k].y);
        v[k].z = fmaf(z.z, f, v[k].z), v[k].w = fmaf(z.w, f, v[k].w);
      }
    }
    // (after a timeout only what is under way is waited for)
    if (!__syncthreads_and(landed)) end = min(end, s0 + 2 * group);
    if (warp == 0 && s0 + 2 * group < end) {
      fence_proxy_async_smem();  // the buffer's last reads
      fetch(s0 + 2 * group, buf);
    }
    buf ^= 1, ph ^= buf == 0;
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if (threadIdx.x + k * L_::kThreads < live * (D / 4))
      finish_row<D>(a, rows.out[of[k]], el[k] % (D / 4), v[k], rows.m[of[k]], rows.f[of[k]]);
}

template <int D, int N>
cudaError_t launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const KvMaps& maps, int n_sm, cudaStream_t s) {
  static std::atomic<size_t> done[kMaxDevices];
  const void* fn = reinterpret_cast<const void*>(attn_few_kernel<D, N>);
  if (const cudaError_t e = opt_in_smem(fn, done, Lay<D, N>::kSmem); e != cudaSuccess) return e;
  Plan pl;
  const int64_t rows = static_cast<int64_t>(c.max_q) * a.G;
  pl.row_tiles = static_cast<int>((rows + N - 1) / N);
  const int64_t base = static_cast<int64_t>(pl.row_tiles) * c.hkv * c.n_seqs;
  const int64_t tiles = max_key_tiles(c, a, N, kKeys);
  // (32 rows of 8000 keys and 8 kv heads of 128, splits of 8, 4 and 2 tiles:
  // 27.3, 23.3 and 27.2 us)
  const int64_t most = std::min<int64_t>(static_cast<int64_t>(ws.cap_rows) / (base * N), max_splits(N));
  const int64_t splits = best_splits(base, n_sm, tiles, most, c.n_seqs > 1, {Lay<D, N>::kCtas, 3., 0.25});
  pl.tiles_per_split = static_cast<int>((tiles + splits - 1) / splits);
  pl.splits = static_cast<int>((tiles + pl.tiles_per_split - 1) / pl.tiles_per_split);
  const int64_t grid = base * pl.splits;
  if (grid > INT_MAX) return cudaErrorInvalidConfiguration;
  attn_few_kernel<D, N><<<static_cast<unsigned>(grid), Lay<D, N>::kThreads, Lay<D, N>::kSmem, s>>>(c, a, ws, pl,
                                                                                                     maps.k_tile, maps.v_tile);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_few_launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const KvMaps& maps,
                            int n_sm, cudaStream_t s) {
  // 16 rows a CTA cost less than 32: the 64 sequences above with 8 rows a kv
  // head take 208 us in the first and 304 us in the second
  const int64_t rows = static_cast<int64_t>(c.max_q) * a.G;
  if (c.D == 128)
    return (rows <= 16 ? launch<128, 16> : launch<128, 32>)(c, a, ws, maps, n_sm, s);
  return (rows <= 16 ? launch<64, 16> : launch<64, 32>)(c, a, ws, maps, n_sm, s);
}

}  // namespace moe
