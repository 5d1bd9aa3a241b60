// The 8-bit paged cache: quantising new tokens into their pages (moe_kv_write)
// and reading tokens back (moe_kv_read).
//
// Write.  One CTA owns one (page, kv head) block of keys and the same block of
// values, so a block's scale has a single writer.  It holds the block's new tokens in
// registers between the two passes that the mathematics needs (the largest
// magnitude, then the codes), so they are read from memory once.  Scales are
// powers of two: x / s and the re-encoding of earlier codes are then exact up
// to the one rounding to e4m3, whatever order tokens arrive in, and nothing is
// lost against a free scale, since e4m3 is a floating format.
//
// Read.  A thread turns chunks of 16 codes into 16 values.  Both are bound by
// memory, so a thread has several independent loads under way.  (Blocks of 64 x 128
// bf16: 3 x up to 8191 tokens written in 26.6 us, 4.5 TB/s; 5 x up to 16384 read
// in 55 us, 4.7 TB/s.)
#include <climits>

#include "attn_internal.cuh"

namespace moe {
namespace {

constexpr int kWriteThreads = 256;

// 8 consecutive elements of the input as fp32
__device__ __forceinline__ void unpack8(const uint4 (&r)[1], float (&f)[8]) {
  const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const uint4 (&r)[2], float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(r[i].x);
    f[4 * i + 1] = __uint_as_float(r[i].y);
    f[4 * i + 2] = __uint_as_float(r[i].z);
    f[4 * i + 3] = __uint_as_float(r[i].w);
  }
}

// The smallest power of two s >= 2^-64 with amax <= 448 s (amax finite, >= 0):
// amax = m 2^e, 1 <= m < 2, and 448 = 1.75 * 2^8.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, 127 - 64);  // biased; subnormal amax lands here too
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

__device__ __forceinline__ uint32_t encode2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// One CTA's block of keys or values: its new rows in registers.
template <int VEC, int PASSES>
struct Block {
  uint4 raw[PASSES][VEC];

  __device__ __forceinline__ void load(const void* x, int64_t stride, int64_t row0, int head, int D, int rows, int r0,
                                       int rstep, int col) {
    const size_t esz = VEC == 1 ? 2 : 4;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = r0 + p * rstep;
      if (r < rows) {
        const uint4* g = reinterpret_cast<const uint4*>(
            static_cast<const char*>(x) + ((row0 + r) * stride + static_cast<int64_t>(head) * D + col) * esz);
#pragma unroll
        for (int i = 0; i < VEC; ++i) raw[p][i] = __ldg(g + i);
      }
    }
  }
  // The warp's largest magnitude; NaN or infinity when there is one, unless
  // `finite`, which leaves them out.
  template <bool FINITE>
  __device__ __forceinline__ float most(int rows, int r0, int rstep) const {
    float amax = 0.f;
    __nv_bfloat162 pair = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      if (r0 + p * rstep < rows) {
        if constexpr (FINITE) {
          float f[8];
          unpack8(raw[p], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = fabsf(f[i]);
            amax = fmaxf(amax, a <= 3.4028234663852886e38f ? a : 0.f);
          }
        } else if constexpr (VEC == 1) {
          const uint32_t w[4] = {raw[p][0].x, raw[p][0].y, raw[p][0].z, raw[p][0].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            pair = __hmax2_nan(pair, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
        } else {
          float f[8];
          unpack8(raw[p], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(f[i]));
        }
      }
    }
    if constexpr (!FINITE && VEC == 1) amax = max_nan(__low2float(pair), __high2float(pair));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    return amax;
  }
  // dst: the block's codes; `at` earlier tokens stand before the new ones, in scale `old`
  __device__ __forceinline__ void store(uint8_t* dst, int D, int at, int rows, int r0, int rstep, int col, float old,
                                        float scale, bool odd) const {
    if (scale > old && at) {
      // the earlier tokens' codes in the new scale (their slots are not this call's)
      const float ratio = old / scale;
      for (int i = threadIdx.x; i < at * (D >> 3); i += kWriteThreads) {
        uint2* p = reinterpret_cast<uint2*>(dst) + i;
        const uint2 u = *p;
        uint32_t w[2] = {u.x, u.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 lo = decode2(w[j] & 0xffffu), hi = decode2(w[j] >> 16);
          w[j] = encode2(lo.x * ratio, lo.y * ratio) | (encode2(hi.x * ratio, hi.y * ratio) << 16);
        }
        *p = make_uint2(w[0], w[1]);
      }
    }
    const float inv = 1.f / scale;  // exact: a power of two within [2^-120, 2^64]
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = r0 + p * rstep;
      if (r < rows) {
        float f[8];
        unpack8(raw[p], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv;
        if (odd) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = f[i] == f[i] ? f[i] : 0.f;
        }
        const uint32_t a = encode2(f[0], f[1]) | (encode2(f[2], f[3]) << 16);
        const uint32_t z = encode2(f[4], f[5]) | (encode2(f[6], f[7]) << 16);
        *reinterpret_cast<uint2*>(dst + static_cast<size_t>(at + r) * D + col) = make_uint2(a, z);
      }
    }
  }
};

// VEC = 16-byte loads of 8 elements (1: bf16, 2: fp32); PASSES: row groups of
// a page that a thread holds.
template <int VEC, int PASSES>
__global__ void __launch_bounds__(kWriteThreads)
    kv_write_kernel(const KvView c, const void* kx, int64_t ks, const void* vx, int64_t vs) {
  __shared__ float s_max[2][kWriteThreads / 32];
  const int b = blockIdx.y, head = blockIdx.z;
  Seq q;
  if (!load_seq(c, b, q)) return;
  const int first = max(q.L - q.n, 0);  // rows at negative positions are skipped
  if (q.n == 0 || first >= q.L) return;
  const int pi = (first >> c.page_log2) + blockIdx.x;
  const int t0 = max(first, pi << c.page_log2), t1 = min(q.L, (pi + 1) << c.page_log2);
  if (t0 >= t1) return;
  const int entry = raw_page(c, b, pi);
  const int rows = t1 - t0, at = t0 & (c.page - 1);
  const int dv = c.D >> 3;  // 8-element vectors of a row
  const int r0 = threadIdx.x / dv, col = (threadIdx.x % dv) * 8;
  const int rstep = kWriteThreads / dv;
  // row t0's place among the call's rows: its position less the first row's
  const int64_t row0 = static_cast<int64_t>(q.q0) + (t0 - (q.L - q.n));
  Block<VEC, PASSES> k, v;
  k.load(kx, ks, row0, head, c.D, rows, r0, rstep, col);
  v.load(vx, vs, row0, head, c.D, rows, r0, rstep, col);
  bool bad = false;
  const int page = checked_page(c, entry, bad);
  if (bad) {
    if (threadIdx.x == 0) atomicOr(c.err, kErrBadBatch);
    return;
  }
  const size_t block = static_cast<size_t>(page) * c.hkv + head;
  const float k_old = at ? c.k_scale[block] : 0.f, v_old = at ? c.v_scale[block] : 0.f;
  float km = k.template most<false>(rows, r0, rstep), vm = v.template most<false>(rows, r0, rstep);
  auto join = [&]() {
    if ((threadIdx.x & 31) == 0) {
      s_max[0][threadIdx.x >> 5] = km;
      s_max[1][threadIdx.x >> 5] = vm;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWriteThreads / 32; ++i) {
      km = max_nan(km, s_max[0][i]);
      vm = max_nan(vm, s_max[1][i]);
    }
  };
  join();
  const bool odd = !(km <= 3.4028234663852886e38f && vm <= 3.4028234663852886e38f);
  if (odd) {  // for all threads: again, without what is not finite
    if (threadIdx.x == 0) atomicOr(c.err, kErrNonFinite);
    __syncthreads();
    km = k.template most<true>(rows, r0, rstep);
    vm = v.template most<true>(rows, r0, rstep);
    join();
  }
  const float k_new = fmaxf(block_scale(km), k_old), v_new = fmaxf(block_scale(vm), v_old);
  const size_t base = block * (static_cast<size_t>(c.page) * c.D);
  k.store(c.k + base, c.D, at, rows, r0, rstep, col, k_old, k_new, odd);
  v.store(c.v + base, c.D, at, rows, r0, rstep, col, v_old, v_new, odd);
  // (every thread has read the old scales before the barriers above)
  if (threadIdx.x == 0) {
    c.k_scale[block] = k_new;
    c.v_scale[block] = v_new;
  }
}

constexpr int kReadThreads = 256;

// 16 codes times a scale to 16 values
template <typename T>
__device__ __forceinline__ void put16(T* dst, const uint4& u, float s) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float f[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = decode2(w[i] & 0xffffu), hi = decode2(w[i] >> 16);
    f[4 * i] = lo.x * s, f[4 * i + 1] = lo.y * s, f[4 * i + 2] = hi.x * s, f[4 * i + 3] = hi.y * s;
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(dst)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  } else {
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      o[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// A thread takes kReadItems chunks of 16 codes, of keys and of values, with
// their loads under way together.
constexpr int kReadItems = 2;
template <typename T>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const KvView c, T* ko, T* vo) {
  const int b = blockIdx.y;
  Seq q;
  if (!load_seq(c, b, q)) return;
  const int per_head = c.D >> 4, per_tok = c.hkv * per_head;
  const int64_t it0 = static_cast<int64_t>(blockIdx.x) * (kReadItems * kReadThreads) + threadIdx.x;
  const int64_t items = static_cast<int64_t>(q.n) * per_tok;
  int raw[kReadItems], t[kReadItems], head[kReadItems], col[kReadItems];
#pragma unroll
  for (int i = 0; i < kReadItems; ++i) {
    const int64_t it = it0 + i * kReadThreads;
    const int row = static_cast<int>(min(it, items) / per_tok), r = static_cast<int>(it - static_cast<int64_t>(row) * per_tok);
    head[i] = r / per_head;
    col[i] = (r - head[i] * per_head) * 16;
    t[i] = q.L - q.n + row;
    raw[i] = INT_MIN;
    if (it < items && t[i] >= 0) raw[i] = raw_page(c, b, t[i] >> c.page_log2);
  }
  uint4 ku[kReadItems], vu[kReadItems];
  float ks[kReadItems], vs[kReadItems];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kReadItems; ++i) {
    ku[i] = vu[i] = make_uint4(0, 0, 0, 0);
    ks[i] = vs[i] = 0.f;
    const int page = raw[i] == INT_MIN ? -1 : checked_page(c, raw[i], bad);
    if (page >= 0) {
      const size_t block = static_cast<size_t>(page) * c.hkv + head[i];
      const size_t at = (block * c.page + (t[i] & (c.page - 1))) * c.D + col[i];
      if (ko) ku[i] = __ldg(reinterpret_cast<const uint4*>(c.k + at)), ks[i] = __ldg(c.k_scale + block);
      if (vo) vu[i] = __ldg(reinterpret_cast<const uint4*>(c.v + at)), vs[i] = __ldg(c.v_scale + block);
    }
  }
#pragma unroll
  for (int i = 0; i < kReadItems; ++i) {
    const int64_t it = it0 + i * kReadThreads;
    if (it >= items) break;
    const size_t dst = static_cast<size_t>(q.q0) * per_tok * 16 + static_cast<size_t>(it) * 16;
    if (ko) put16(ko + dst, ku[i], ks[i]);
    if (vo) put16(vo + dst, vu[i], vs[i]);
  }
  if (bad) atomicOr(c.err, kErrBadBatch);
}

template <int VEC>
cudaError_t write_dtype(const KvView& c, const void* k, int64_t ks, const void* v, int64_t vs,
                        cudaStream_t s) {
  // pages that n new tokens can touch
  const unsigned pages = static_cast<unsigned>((static_cast<int64_t>(c.max_q) + c.page - 2) / c.page + 1);
  const dim3 grid(pages, c.n_seqs, c.hkv);
  const int need = (c.page * (c.D >> 3) + kWriteThreads - 1) / kWriteThreads;
  if (need <= 1)
    kv_write_kernel<VEC, 1><<<grid, kWriteThreads, 0, s>>>(c, k, ks, v, vs);
  else if (need <= 2)
    kv_write_kernel<VEC, 2><<<grid, kWriteThreads, 0, s>>>(c, k, ks, v, vs);
  else if (need <= 4)
    kv_write_kernel<VEC, 4><<<grid, kWriteThreads, 0, s>>>(c, k, ks, v, vs);
  else
    kv_write_kernel<VEC, 8><<<grid, kWriteThreads, 0, s>>>(c, k, ks, v, vs);
  return cudaGetLastError();
}

}  // namespace

cudaError_t kv_write_launch(const KvView& c, const void* k, int64_t ks, const void* v, int64_t vs,
                            moe_dtype_t dt, cudaStream_t s) {
  return dt == MOE_BF16 ? write_dtype<1>(c, k, ks, v, vs, s) : write_dtype<2>(c, k, ks, v, vs, s);
}

cudaError_t kv_read_launch(const KvView& c, void* k, void* v, moe_dtype_t dt, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(c.max_q) * c.hkv * (c.D >> 4);
  constexpr int kPer = kReadItems * kReadThreads;
  const dim3 grid(static_cast<unsigned>((items + kPer - 1) / kPer), c.n_seqs);
  if (dt == MOE_BF16)
    kv_read_kernel<__nv_bfloat16><<<grid, kReadThreads, 0, s>>>(
        c, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v));
  else
    kv_read_kernel<float><<<grid, kReadThreads, 0, s>>>(c, static_cast<float*>(k),
                                                        static_cast<float*>(v));
  return cudaGetLastError();
}

}  // namespace moe
