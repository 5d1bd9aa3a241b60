// Attention over the 8-bit cache for many rows (prompts, chunks) on tcgen05.
//
// The mathematics is that of attn_rows.cu: weights 2^(s + log2 v - m + lift)
// with the block's value scale in the exponent, o = sum w c / sum w / v, an
// online softmax whose reference m moves only when it would grow by 2^5.
//
// One CTA takes 256 rows (a row is a query head of a token; the heads that
// share a kv head are packed into the rows, so K and V are read once for all
// of them) as two M = 128 tiles, and walks over 128-key tiles:
//   1 warp    TMA: key codes into the swizzled operand layout (three stages),
//             value codes as they lie (two stages), the blocks' scales
//   4 warps   value codes -> f16 (exact) in the swizzled operand layout
//   1 thread  tcgen05.mma: S = Q K^T in e4m3, then O += P V in f16 (P from
//             tensor memory, V as it lies, MN-major)
//   2 x 4     softmax warps, one group a M tile, a thread a row: S from tensor
//             memory, weights back as f16 over S
// Keys are multiplied as they are stored: a bf16 query (8 bits) is the sum of
// two e4m3 numbers of 4 bits each, exact down to 2^-18 of the row's largest,
// and e4m3 products run at twice the rate of f16 ones, so the two terms cost
// what one f16 product would and no key is converted.  Values stay f16
// operands: a weight of 11 bits would be three e4m3 terms.
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
constexpr int kThreads = 448;  // 4 + 4 softmax warps, 4 conversion warps, MMA warp, load warp
constexpr int kKStages = 3;

template <int D>
struct Lay {
  static constexpr int kHalf = kTile * 128;        // 128 rows x 64 f16, swizzled
  static constexpr int kMat8 = kTile * D;          // an operand tile of codes
  static constexpr int kMat = kHalf * (D / 64);    // an operand tile of f16
  static constexpr int kQ = 0;                     // two M tiles of two terms
  static constexpr int kK = kQ + 4 * kMat8;
  static constexpr int kV = kK + kKStages * kMat8; // two stages of f16
  static constexpr int kRaw = kV + 2 * kMat;       // two stages of value codes
  static constexpr int kConst = kRaw + 2 * kMat8;  // [4][8] float4: scales of a tile's 16-key groups
  static constexpr int kBar = kConst + 4 * 8 * 16;
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
  kOFull = 19,
  kCFull = 21,   // [4] scales
  kBars = 25
};

// The one thread that issues products is on every step's path: the MMAs of a
// product stand in one block, their descriptors a constant apart.
//
// S[tmem] = (Q1 + Q2) K^T: e4m3 operands, f32 accumulator; q and k step by 32
// codes (32 bytes) along the head, the second term `TERM` bytes behind Q1.
#define MOE_S_MMA(A, B, P) "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], " A ", " B ", %3, " P ";\n\t"
template <int D>
__device__ __forceinline__ void mma_s(uint32_t d_tmem, uint64_t q_desc, uint64_t k_desc, uint32_t idesc) {
  constexpr uint64_t kTerm = (kTile * D) >> 4;
  if constexpr (D == 128) {
    asm volatile(
        "{\n\t.reg .b64 q<8>, k<4>;\n\t"
        "add.s64 k1, %2, 2;\n\tadd.s64 k2, %2, 4;\n\tadd.s64 k3, %2, 6;\n\t"
        "add.s64 q1, %1, 2;\n\tadd.s64 q2, %1, 4;\n\tadd.s64 q3, %1, 6;\n\t"
        "add.s64 q4, %1, %4;\n\tadd.s64 q5, q4, 2;\n\tadd.s64 q6, q4, 4;\n\tadd.s64 q7, q4, 6;\n\t"
        MOE_S_MMA("%1", "%2", "0") MOE_S_MMA("q1", "k1", "1") MOE_S_MMA("q2", "k2", "1") MOE_S_MMA("q3", "k3", "1")
        MOE_S_MMA("q4", "%2", "1") MOE_S_MMA("q5", "k1", "1") MOE_S_MMA("q6", "k2", "1") MOE_S_MMA("q7", "k3", "1")
        "}" ::"r"(d_tmem), "l"(q_desc), "l"(k_desc), "r"(idesc), "n"(kTerm)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .b64 q<4>, k1;\n\t"
        "add.s64 k1, %2, 2;\n\tadd.s64 q1, %1, 2;\n\tadd.s64 q2, %1, %4;\n\tadd.s64 q3, q2, 2;\n\t"
        MOE_S_MMA("%1", "%2", "0") MOE_S_MMA("q1", "k1", "1") MOE_S_MMA("q2", "%2", "1") MOE_S_MMA("q3", "k1", "1")
        "}" ::"r"(d_tmem), "l"(q_desc), "l"(k_desc), "r"(idesc), "n"(kTerm)
        : "memory");
  }
}
#undef MOE_S_MMA

// O[tmem] (+)= P[tmem] V[smem] over 64 keys: P 8 columns, V 16 rows of 128
// bytes a K step; the first MMA overwrites O when `first`.
__device__ __forceinline__ void mma_o(uint32_t d_tmem, uint32_t p_tmem, uint64_t v_desc, uint32_t idesc,
                                      uint32_t first) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 v<4>;\n\t"
      "setp.eq.b32 p, %4, 0;\n\t"
      "add.s64 v1, %2, 128;\n\tadd.s64 v2, %2, 256;\n\tadd.s64 v3, %2, 384;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1 + 8], v1, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1 + 16], v2, %3, 1;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1 + 24], v3, %3, 1;\n\t}" ::"r"(d_tmem),
      "r"(p_tmem), "l"(v_desc), "r"(idesc), "r"(first)
      : "memory");
}

// K-major operand of D-byte rows in the D-byte swizzled layout (D = 64, 128):
// 8-row atoms of 8 D bytes.
template <int D>
__device__ __forceinline__ uint64_t sdesc_k(uint32_t smem_addr) {
  if constexpr (D == 128) return sdesc_sw128(smem_addr);
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(512u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(4u) << 61;  // 64-byte swizzle
  return d;
}
// Byte offset of 16-byte chunk c of row r in that layout.
template <int D>
__device__ __forceinline__ uint32_t k_off(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
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

__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Two fp32 operations an instruction.
__device__ __forceinline__ void fma2(float& x, float& y, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a0, float a1) {
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%0, %1};\n\t"
      "add.rn.f32x2 b, b, a;\n\tmov.b64 {%0, %1}, b;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

template <int D>
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
  if (!work_of(c, a, pl, b, hk, rt, w) || split >= w.n_split) return;
  const int t_begin = split * pl.tiles_per_split;
  const int t_end = min(w.k.n_t, t_begin + pl.tiles_per_split);
  const int n = t_end - t_begin;  // 0 when the rows see nothing
  const int n_mt = w.r1 - w.r0 > kM ? 2 : 1;

  auto bar = [&](int i) { return base_u + L_::kBar + 8 * i; };
  if (threadIdx.x == 0) {
    const int count[kBars] = {128 * n_mt, 1, 1, 1, 1, 1, 1, 1, 1, 128, 128, 128, 128,
                              1, 1, 1, 1, 128, 128, 1, 1, 8, 8, 8, 8};
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

  if (warp == 13) {
    // lane g (0 .. 7) looks after 16-key group g; the first group of a page
    // issues the page's copies
    if (lane < 8 && n > 0) {
      bool ok = true, bad = false;
      const int per = c.page >> 4;  // groups of a page
      const uint32_t bytes = static_cast<uint32_t>(c.page) * D;
      auto seen = [&](int t) {  // whether some row sees a key of the group's page
        const int tok = w.k.base(t) + 16 * (lane & ~(per - 1));
        return tok < w.k.hi && (tok + c.page > w.k.lo || tok < a.sinks);
      };
      auto entry = [&](int t) {
        return t < t_end && seen(t) ? raw_page(c, b, (w.k.base(t) + 16 * lane) >> c.page_log2) : INT_MIN;
      };
      int raw = entry(t_begin);
      int k_sent = 0, r_sent = 0;  // tiles whose copies are on their way
      for (int j = 0; ok && j < n; ++j) {
        const int ks = j % kKStages, rs = j & 1;
        const int page = raw == INT_MIN ? -1 : checked_page(c, raw, bad);
        float kscale = 0.f, vscale = 1.f;
        if (page >= 0) {
          const size_t at = static_cast<size_t>(page) * c.hkv + hk;
          kscale = __ldg(c.k_scale + at);
          vscale = __ldg(c.v_scale + at);
        }
        raw = entry(t_begin + j + 1);
        const bool copies = page >= 0 && (lane & (per - 1)) == 0;
        const uint32_t total = __popc(__ballot_sync(0xffu, copies)) * bytes;
        ok = j < kKStages || mbar_wait(bar(kKEmpty + ks), (j / kKStages - 1) & 1, c.err);
        ok = __all_sync(0xffu, ok);
        if (!ok) break;
        // a ring of four: the softmax of tile j - 4 is done when the K stage of tile j is free,
        // and has been through its slot's barrier (a parity tells neighbouring phases apart)
        vscale = fmaxf(vscale, kMinBlockScale);
        reinterpret_cast<float4*>(smem + L_::kConst)[(j & 3) * 8 + lane] =
            make_float4(kscale, __log2f(vscale), __frcp_rn(vscale), 0.f);
        mbar_arrive(bar(kCFull + (j & 3)));
        if (lane == 0) mbar_arrive_expect_tx(bar(kKFull + ks), total);
        __syncwarp(0xffu);
        if (copies)
          tma_load_3d(base_u + L_::kK + ks * L_::kMat8 + 16 * lane * D, &k_map, 0, hk * c.page, page,
                      bar(kKFull + ks));
        k_sent = j + 1;
        ok = j < 2 || mbar_wait(bar(kREmpty + rs), ((j >> 1) - 1) & 1, c.err);
        ok = __all_sync(0xffu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(kRFull + rs), total);
        __syncwarp(0xffu);
        if (copies)
          bulk_g2s(base_u + L_::kRaw + rs * L_::kMat8 + 16 * lane * D,
                   c.v + (static_cast<size_t>(page) * c.hkv + hk) * bytes, bytes, bar(kRFull + rs));
        r_sent = j + 1;
      }
      if (!ok) {  // the copies land before the CTA goes
        for (int j = max(k_sent - kKStages, 0); j < k_sent; ++j)
          mbar_wait(bar(kKFull + j % kKStages), (j / kKStages) & 1, c.err);
        for (int j = max(r_sent - 2, 0); j < r_sent; ++j) mbar_wait(bar(kRFull + (j & 1)), (j >> 1) & 1, c.err);
      }
      if (bad) atomicOr(c.err, kErrBadBatch);
    }
  } else if (warp == 12) {
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_f16(kM, kTile);           // e4m3 is format 0 of its kind, too
      constexpr uint32_t id_o = idesc_f16(kM, D) | (1u << 16);  // V is MN-major
      const uint64_t q_desc = sdesc_k<D>(base_u + L_::kQ), k_desc = sdesc_k<D>(base_u + L_::kK);
      const uint64_t v_desc = sdesc_sw128_mn(base_u + L_::kV, L_::kHalf);
      auto issue_s = [&](int i, int stage) {
        mma_s<D>(tmem + i * 128, q_desc + i * (2 * L_::kMat8 >> 4), k_desc + stage * (L_::kMat8 >> 4), id_s);
        mma_commit(bar(kSFull + i));
      };
      bool ok = mbar_wait(bar(kQFull), 0, c.err) && mbar_wait(bar(kKFull), 0, c.err);
      if (ok) {
        fence_after_sync();
        for (int i = 0; i < n_mt; ++i) issue_s(i, 0);
        mma_commit(bar(kKEmpty));
      }
      int ks = 0, kph = 0;  // K stage and parity of tile j
      for (int j = 0; ok && j < n; ++j) {
        const int st = j & 1;
        const uint64_t vd = v_desc + st * (L_::kMat >> 4);
        if (++ks == kKStages) ks = 0, kph ^= 1;  // those of tile j + 1
        for (int i = 0; ok && i < n_mt; ++i) {
          ok = mbar_wait(bar(kPFull + i), j & 1, c.err) && (i > 0 || mbar_wait(bar(kVFull + st), (j >> 1) & 1, c.err));
          if (!ok) break;
          fence_after_sync();
          const uint32_t ot = tmem + 256 + i * 128, pt = tmem + i * 128;
          mma_o(ot, pt, vd, id_o, j == 0);
          mma_o(ot, pt + 32, vd + (64 * 128 >> 4), id_o, 0);
          if (i == n_mt - 1) mma_commit(bar(kVEmpty + st));
          if (j == n - 1) {
            mma_commit(bar(kOFull + i));
          } else {
            ok = i > 0 || mbar_wait(bar(kKFull + ks), kph, c.err);
            if (!ok) break;
            fence_after_sync();
            issue_s(i, ks);
            if (i == n_mt - 1) mma_commit(bar(kKEmpty + ks));
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
    // value codes to f16: thread t takes 16-byte chunk t % (D / 16) of keys
    // t / (D / 16) + 0, kPer, ...; a chunk becomes two of the operand's
    const int tid = threadIdx.x - 256;
    constexpr int kChunks = D / 16, kPer = 128 / kChunks;
    const int ch = tid % kChunks, row0 = tid / kChunks;
    // the two halves' lanes store their two chunks in opposite order: no bank conflicts
    const int c0 = 2 * (ch & 3) + (ch >> 2);
    const uint32_t out = (ch >> 2) * L_::kHalf + row0 * 128;
    const uint32_t o0 = out + ((c0 ^ (row0 & 7)) << 4), o1 = out + (((c0 ^ 1) ^ (row0 & 7)) << 4);
    const bool swap = (ch >> 2) != 0;
    for (int j = 0; j < n; ++j) {
      const int st = j & 1, ph = (j >> 1) & 1;
      if (!mbar_wait(bar(kRFull + st), ph, c.err)) break;
      if (j >= 2 && !mbar_wait(bar(kVEmpty + st), ph ^ 1, c.err)) break;
      const int base = w.k.base(t_begin + j);
      const bool whole = base + kTile <= w.k.hi && (base >= w.k.lo || base + kTile <= a.sinks);
      const char* src = smem + L_::kRaw + st * L_::kMat8 + tid * 16;
      char* dst = smem + L_::kV + st * L_::kMat;
#pragma unroll
      for (int p = 0; p < kTile / kPer; ++p) {
        uint4 raw = *reinterpret_cast<const uint4*>(src + p * 2048);
        if (!whole) {
          // what no row sees is zero: a NaN there would reach the rows through 0 * NaN
          const int tok = base + p * kPer + row0;
          if (!(tok < w.k.hi && (tok >= w.k.lo || tok < a.sinks))) raw = make_uint4(0, 0, 0, 0);
        }
        uint4 lo, hi;
        codes_to_half(raw.x, lo.x, lo.y);
        codes_to_half(raw.y, lo.z, lo.w);
        codes_to_half(raw.z, hi.x, hi.y);
        codes_to_half(raw.w, hi.z, hi.w);
        // (kPer is a multiple of 8: the swizzle of a later pass is the first's)
        *reinterpret_cast<uint4*>(dst + o0 + p * kPer * 128) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(dst + o1 + p * kPer * 128) = swap ? lo : hi;
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kVFull + st));
      mbar_arrive(bar(kREmpty + st));
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
      // the row's query, brought to [2^7, 2^8) by a power of two, as two e4m3 terms
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
          amax = max3(amax, fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xffff0000u)));
      }
      const float f = copysignf(row_factor<7>(amax), a.scale_log2);
      lscale = a.scale_log2 / f;
      const bool inf = !(amax < INFINITY);  // (codes saturate: such a row is NaN instead)
      char* dst = smem + L_::kQ + i * 2 * L_::kMat8;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const uint32_t u[8] = {raw[2 * x].x,     raw[2 * x].y,     raw[2 * x].z,     raw[2 * x].w,
                               raw[2 * x + 1].x, raw[2 * x + 1].y, raw[2 * x + 1].z, raw[2 * x + 1].w};
        uint32_t t0[4], t1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w0 = 0, w1 = 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 v = make_float2(__uint_as_float(u[2 * k + e] << 16) * f,
                                         __uint_as_float(u[2 * k + e] & 0xffff0000u) * f);
            const uint32_t q1 = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
            const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q1), __NV_E4M3);
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hr));
            const uint32_t q2 =
                __nv_cvt_float2_to_fp8x2(make_float2(v.x - back.x, v.y - back.y), __NV_SATFINITE, __NV_E4M3);
            w0 |= q1 << (16 * e);
            w1 |= q2 << (16 * e);
          }
          t0[k] = inf ? 0x7f7f7f7fu : w0;
          t1[k] = w1;
        }
        const uint32_t off = k_off<D>(row, x);
        *reinterpret_cast<uint4*>(dst + off) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
        *reinterpret_cast<uint4*>(dst + L_::kMat8 + off) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kQFull));
    }
    // the range that all rows of the CTA see whole
    const int p_lo = w.base_p + w.r0 / a.G, p_hi = w.base_p + (w.r1 - 1) / a.G;
    for (int j = 0; j < n; ++j) {
      // (S of this tile says that O += P V of the tile before is done, too)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(kCFull + (j & 3)), (j >> 2) & 1, c.err) &&
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
      if (!whole) {
        // what the row does not see goes to -inf first, where it lies
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          tmem_ld32(ts + 32 * x, s[0]);
          tmem_wait_ld32(s[0]);
          uint32_t u[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) u[k] = sees(base + 32 * x + k) ? __float_as_uint(s[0][k]) : 0xff800000u;
          tmem_st32(ts + 32 * x, u);
        }
        tmem_wait_st();
      }
      float mt = -INFINITY;
      tmem_ld32(ts, s[0]);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        tmem_wait_ld32(s[x & 1]);
        tmem_ld32(ts + 32 * ((x + 1) & 3), s[(x + 1) & 1]);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const float4 z = cn[2 * x + gg];
          const float* v = s[x & 1] + 16 * gg;
          float t0 = max3(v[0], v[1], v[2]), t1 = max3(v[3], v[4], v[5]);
          t0 = max3(t0, v[6], v[7]), t1 = max3(t1, v[8], v[9]);
          t0 = max3(t0, v[10], v[11]), t1 = max3(t1, v[12], v[13]);
          t0 = max3(t0, v[14], v[15]);
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
            tmem_wait_ld16(u);
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
        uint32_t u[16];
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
          const float4 z = cn[2 * x + gg];
          const float sc = fmaxf(lscale * z.x, kTiny), off = z.y - ref;
          const float* v = s[x & 1] + 16 * gg;
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float w0, w1;
            fma2(w0, w1, v[k], v[k + 1], sc, off);
            w0 = ex2(w0), w1 = ex2(w1);
            add2(sum0, sum1, w0, w1);
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
          tmem_wait_ld32(o);
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
cudaError_t launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const CUtensorMap& k_map, int n_sm,
                   cudaStream_t s) {
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
  attn_tiles_kernel<D><<<static_cast<unsigned>(grid), kThreads, Lay<D>::kSmem, s>>>(c, a, ws, pl, k_map);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || pl.splits == 1) return e;
  const int64_t items = base * kRows, per = kJoinThreads / (D / 4);
  attn_join_kernel<D><<<static_cast<unsigned>((items + per - 1) / per), kJoinThreads, 0, s>>>(c, a, ws, pl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_tiles_launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const KvMaps& maps,
                              int n_sm, cudaStream_t s) {
  return c.D == 128 ? launch<128>(c, a, ws, maps.k_tile, n_sm, s) : launch<64>(c, a, ws, maps.k_tile, n_sm, s);
}

}  // namespace moe
