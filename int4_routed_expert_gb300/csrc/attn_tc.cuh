// What the two tcgen05 attention kernels share: operand layouts and products,
// and the warps that bring tiles of 128 keys into shared memory.
#pragma once

#include <climits>

#include "attn_common.cuh"
#include "smem_opt_in.cuh"
#include "stream_common.cuh"
#include "tc_ptx.cuh"

namespace moe {

using namespace tc;

constexpr int kKeys = 128;       // keys of a tile
constexpr int kConstRing = 8;    // tiles whose blocks' scales are kept
constexpr float kTiny = 1e-37f;  // keeps what is hidden at -inf where a block's scale is 0

// 16 bytes to shared memory, the last 16 - n of them zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Whether any of a barrier's `count` threads says yes.
__device__ __forceinline__ bool named_vote(int id, int count, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(yes)), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

// The one thread that issues products is on every step's path: the MMAs of a
// product stand in one block, their descriptors a constant apart.
//
// S[tmem] = (Q1 + Q2) K^T: e4m3 operands, f32 accumulator; q and k step by 32
// codes (32 bytes) along the head, the second term `TERM` bytes behind Q1.
#define MOE_S_MMA(A, B, P) "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], " A ", " B ", %3, " P ";\n\t"
template <int D>
__device__ __forceinline__ void mma_s(uint32_t d_tmem, uint64_t q_desc, uint64_t k_desc, uint32_t idesc) {
  constexpr uint64_t kTerm = (kKeys * D) >> 4;
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
// (x, y) = (a0, a1) * (b0, b1) + (c0, c1)
__device__ __forceinline__ void fma2(float& x, float& y, float a0, float a1, float b0, float b1, float c0,
                                     float c1) {
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& x, float& y, float a0, float a1, float b) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a0), "f"(a1), "f"(b));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ---- tiles of keys into shared memory ---------------------------------------------
//
// KS stages of key codes in the swizzled operand layout, RS stages of value
// codes (VS = 0: in the same layout; else as they lie, and VS stages of values
// in f16 in the swizzled layout [D / 64][128 keys][128 bytes]), and a ring of
// the blocks' scales by groups of 16 keys: {key scale, log2 value scale,
// 1 / value scale, 0}.
template <int D, int KS, int RS, int VS, int CT = 128>
struct TileIo {
  static constexpr int kMat8 = kKeys * D;
  static constexpr int kHalf = kKeys * 128;
  static constexpr int kMat = kHalf * (D / 64);
  uint32_t k, raw, v;  // shared-memory addresses of the stages
  char* smem;          // generic address of shared address `base`
  uint32_t base, consts;
  // barriers (addresses of the first of each): stages full and empty, scales
  uint32_t k_full, k_empty, r_full, r_empty, v_full, c_full;

  __device__ __forceinline__ const float4* scales(int j) const {
    return reinterpret_cast<const float4*>(smem + (consts - base)) + (j % kConstRing) * 8;
  }

  // One warp's lanes 0 .. 7: lane g looks after 16-key group g, the first group
  // of a page issues the page's copies.  A tile's table entries are read two
  // tiles ahead and its scales one tile ahead.  k_empty[s] is passed on by
  // the softmax, which then also is through with the scales of the tile
  // kConstRing - KS before.
  __device__ __forceinline__ void load(const KvView& c, const AttnArgs& a, const KeyTiles& kt, int b, int hk,
                                       int t_begin, int n, const CUtensorMap* k_map, const CUtensorMap* v_map,
                                       int lane) const {
    static_assert(kConstRing > KS, "the ring outlives the key stages");
    const int t_end = t_begin + n;
    bool ok = true, bad = false, odd = false;
    const int per = c.page >> 4;  // groups of a page
    const uint32_t bytes = static_cast<uint32_t>(c.page) * D;
    auto entry = [&](int t) {  // INT_MIN where no row sees a key of the group's page
      if (t >= t_end) return INT_MIN;
      const int base_key = kt.base(t), tok = base_key + 16 * (lane & ~(per - 1));
      if (!(tok < kt.hi && (tok + c.page > kt.lo || tok < a.sinks))) return INT_MIN;
      return raw_page(c, b, (base_key + 16 * lane) >> c.page_log2);
    };
    auto take = [&](int raw_entry, float& ks, float& vs) {
      const int page = raw_entry == INT_MIN ? -1 : checked_page(c, raw_entry, bad);
      ks = 0.f, vs = 1.f;
      if (page >= 0) {
        const size_t at = static_cast<size_t>(page) * c.hkv + hk;
        ks = __ldg(c.k_scale + at);
        vs = __ldg(c.v_scale + at);
      }
      return page;
    };
    float kscale, vscale;
    int page = take(entry(t_begin), kscale, vscale), raw1 = entry(t_begin + 1);
    int k_sent = 0, r_sent = 0;  // tiles whose copies are on their way
    for (int j = 0; j < n; ++j) {
      const int ks = j % KS, rs = j % RS;
      float kscale1, vscale1;
      const int page1 = take(raw1, kscale1, vscale1);
      raw1 = entry(t_begin + j + 2);
      const bool copies = page >= 0 && (lane & (per - 1)) == 0;
      const uint32_t total = __popc(__ballot_sync(0xffu, copies)) * bytes;
      ok = j < KS || mbar_wait(k_empty + 8 * ks, (j / KS - 1) & 1, c.err);
      ok = __all_sync(0xffu, ok);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(k_full + 8 * ks, total);
      __syncwarp(0xffu);
      if (copies) tma_load_3d(k + ks * kMat8 + 16 * lane * D, k_map, 0, hk * c.page, page, k_full + 8 * ks);
      k_sent = j + 1;
      // (looked at here, not where they are loaded: 64 sequences of up to 16384 keys, 208 us instead of 240)
      odd |= !(kscale >= 0.f && kscale < INFINITY && vscale >= 0.f && vscale < INFINITY);
      // (a smaller value scale, of a pool that write has not made, counts as the smallest: its values
      // are below 2^-55 either way, and 1 / v times a sum of weights stays within fp32)
      const float v = fmaxf(vscale, kMinBlockScale);
      reinterpret_cast<float4*>(smem + (consts - base))[(j % kConstRing) * 8 + lane] =
          make_float4(kscale, __log2f(v), __frcp_rn(v), 0.f);
      mbar_arrive(c_full + 8 * (j % kConstRing));
      ok = j < RS || mbar_wait(r_empty + 8 * rs, (j / RS - 1) & 1, c.err);
      ok = __all_sync(0xffu, ok);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(r_full + 8 * rs, total);
      __syncwarp(0xffu);
      if (copies && VS == 0)
        tma_load_3d(raw + rs * kMat8 + 16 * lane * D, v_map, 0, hk * c.page, page, r_full + 8 * rs);
      if (copies && VS != 0)
        bulk_g2s(raw + rs * kMat8 + 16 * lane * D, c.v + (static_cast<size_t>(page) * c.hkv + hk) * bytes, bytes,
                 r_full + 8 * rs);
      r_sent = j + 1;
      page = page1, kscale = kscale1, vscale = vscale1;
    }
    if (!ok) {  // the copies land before the CTA goes
      for (int j = max(k_sent - KS, 0); j < k_sent; ++j) mbar_wait(k_full + 8 * (j % KS), (j / KS) & 1, c.err);
      for (int j = max(r_sent - RS, 0); j < r_sent; ++j) mbar_wait(r_full + 8 * (j % RS), (j / RS) & 1, c.err);
    }
    if (bad) atomicOr(c.err, kErrBadBatch);
    if (odd) atomicOr(c.err, kErrNonFinite);
  }

  // CT threads: value codes to f16.  Thread t takes 16-byte chunk t % (D / 16)
  // of keys t / (D / 16) + 0, kPer, ...; a chunk becomes two of the operand's.
  // free(j) waits until the product that read the stage of tile j - VS is done.
  template <typename Free>
  __device__ __forceinline__ void convert(const KvView& c, const AttnArgs& a, const KeyTiles& kt, int t_begin, int n,
                                          int tid, Free free) const {
    constexpr int kChunks = D / 16, kPer = CT / kChunks;
    const int ch = tid % kChunks, row0 = tid / kChunks;
    // the two halves' lanes store their two chunks in opposite order: no bank conflicts
    const int c0 = 2 * (ch & 3) + (ch >> 2);
    const uint32_t out = (ch >> 2) * kHalf + row0 * 128;
    const uint32_t o0 = out + ((c0 ^ (row0 & 7)) << 4), o1 = out + (((c0 ^ 1) ^ (row0 & 7)) << 4);
    const bool swap = (ch >> 2) != 0;
    for (int j = 0; j < n; ++j) {
      const int rs = j % RS, vs = j % VS;
      if (!mbar_wait(r_full + 8 * rs, (j / RS) & 1, c.err) || (j >= VS && !free(j))) break;
      const int base_key = kt.base(t_begin + j);
      const bool whole = base_key + kKeys <= kt.hi && (base_key >= kt.lo || base_key + kKeys <= a.sinks);
      const char* src = smem + (raw - base) + rs * kMat8 + tid * 16;
      const char* src0 = src + (swap ? 8 : 0);
      const char* src1 = src + (swap ? 0 : 8);
      char* dst = smem + (v - base) + vs * kMat;
#pragma unroll
      for (int p = 0; p < kKeys / kPer; ++p) {
        uint2 u0 = *reinterpret_cast<const uint2*>(src0 + p * (CT * 16));
        uint2 u1 = *reinterpret_cast<const uint2*>(src1 + p * (CT * 16));
        if (!whole) {
          // what no row sees is zero: a NaN there would reach the rows through 0 * NaN
          const int tok = base_key + p * kPer + row0;
          if (!(tok < kt.hi && (tok >= kt.lo || tok < a.sinks))) u0 = u1 = make_uint2(0, 0);
        }
        uint4 h0, h1;
        codes_to_half(u0.x, h0.x, h0.y);
        codes_to_half(u0.y, h0.z, h0.w);
        codes_to_half(u1.x, h1.x, h1.y);
        codes_to_half(u1.y, h1.z, h1.w);
        // (kPer is a multiple of 8: the swizzle of a later pass is the first's)
        *reinterpret_cast<uint4*>(dst + o0 + p * kPer * 128) = h0;
        *reinterpret_cast<uint4*>(dst + o1 + p * kPer * 128) = h1;
      }
      fence_proxy_async_smem();
      mbar_arrive(v_full + 8 * vs);
      mbar_arrive(r_empty + 8 * rs);
    }
  }
};

// Two consecutive query elements (a bf16 pair times f, at most 2^8) as two e4m3
// terms: their sum is exact down to 2^-18 of the row's largest.  (f16 holds the
// product's 8 bits, from 2^-17 on rounded to 2^-25.)
__device__ __forceinline__ void split_query(uint32_t pair, float f, uint32_t& q1, uint32_t& q2) {
  const __half2 v = __floats2half2_rn(__uint_as_float(pair << 16) * f, __uint_as_float(pair & 0xffff0000u) * f);
  q1 = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q1), __NV_E4M3);
  q2 = __nv_cvt_halfraw2_to_fp8x2(__hsub2(v, __half2(back)), __NV_SATFINITE, __NV_E4M3);
}

// How a call's rows and keys are cut into CTAs.
struct Plan {
  int row_tiles, splits, tiles_per_split;
};

// What a kernel's CTAs cost, in the time that a CTA with an SM of its own takes
// for a tile of keys.
struct Costs {
  int per_sm;    // CTAs of an SM: the tiles of two take half as long again
  double start;  // set-up, first loads, results
  double join;   // a split's part of the join
};

// Splits of `tiles` tiles for `base` row tiles, at most `most`: the least time.
// Where there are several sequences, `tiles` comes from a bound that most of
// them stay below: the time is the sum over a batch at the bound and one at half
// of it, where empty CTAs leave their slots to others and half a round is lost
// at the end.
inline int64_t best_splits(int64_t base, int64_t n_sm, int64_t tiles, int64_t most, bool ragged, const Costs& k) {
  const int64_t end = std::max<int64_t>(std::min<int64_t>({tiles, most, 256}), 1);
  const int64_t resident = n_sm * k.per_sm;
  double least = 1e300;
  int64_t best = 1;
  for (int64_t s = 1; s <= end; ++s) {
    const double tile = base * s > n_sm && k.per_sm > 1 ? 1.5 : 1.;
    const double cta = tile * static_cast<double>((tiles + s - 1) / s) + k.start;
    const double full = static_cast<double>((base * s + resident - 1) / resident) * cta;
    const double half = std::max(0.5 * static_cast<double>(base * s) / static_cast<double>(resident) + 0.5, 1.0) * cta;
    const double cost = (ragged ? 0.5 * (full + half) : full) + k.join * static_cast<double>(s);
    if (cost < least) least = cost, best = s;
  }
  return best;
}

// Where a CTA, or a row of partial results, stands.
struct Work {
  Seq q;
  int b, hk, r0, r1, base_p;
  int tok0, rem0;  // token and head (of the kv head's) of row r0
  int p_lo, p_hi;  // positions of the first and the last row
  KeyTiles k;
  int n_split;

  // token and head of row r0 + i: (rem0 + i) / G by its reciprocal, exact as the
  // dividend is below 2^13 and half away from the next whole number
  __device__ __forceinline__ void row(const AttnArgs& a, int i, int& tok, int& head) const {
    const int x = rem0 + i, t = static_cast<int>((static_cast<float>(x) + 0.5f) * a.inv_g);
    tok = tok0 + t;
    head = x - t * a.G;
  }
};

template <int ROWS>
__device__ __forceinline__ bool work_of(const KvView& c, const AttnArgs& a, const Plan& pl, int b, int hk, int rt,
                                        Work& w) {
  if (!load_seq(c, b, w.q)) return false;
  const int64_t R = static_cast<int64_t>(w.q.n) * a.G;
  const int64_t r0 = static_cast<int64_t>(rt) * ROWS;
  if (r0 >= R) return false;
  w.b = b;
  w.hk = hk;
  w.r0 = static_cast<int>(r0);
  w.r1 = static_cast<int>(min(R, r0 + ROWS));
  w.base_p = w.q.L - w.q.n;
  w.tok0 = w.r0 / a.G;
  w.rem0 = w.r0 - w.tok0 * a.G;
  int last, head;
  w.row(a, w.r1 - 1 - w.r0, last, head);
  w.p_lo = w.base_p + w.tok0;
  w.p_hi = w.base_p + last;
  w.k = key_tiles<kKeys>(a, w.q.L, w.p_lo, w.p_hi);
  w.n_split = max((w.k.n_t + pl.tiles_per_split - 1) / pl.tiles_per_split, 1);
  return true;
}

}  // namespace moe
