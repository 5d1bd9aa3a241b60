// The 8-bit paged cache: quantising new tokens into their pages (moe_kv_write)
// and reading tokens back (moe_kv_read).
//
// Write.  One CTA owns one (page, kv head) block of keys or of values, so a
// block's scale has a single writer.  It holds the block's new tokens in
// registers between the two passes that the mathematics needs (the largest
// magnitude, then the codes), so they are read from memory once.  Scales are
// powers of two: x / s and the re-encoding of earlier codes are then exact up
// to the one rounding to e4m3, whatever order tokens arrive in, and nothing is
// lost against a free scale, since e4m3 is a floating format.
//
// Read.  A thread turns 16 codes into 16 values.  Both are bound by memory.
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

// VEC = 16-byte loads of 8 elements (1: bf16, 2: fp32); PASSES: row groups of
// a page that a thread holds.
template <int VEC, int PASSES>
__global__ void __launch_bounds__(kWriteThreads)
    kv_write_kernel(const KvView c, const void* kx, int64_t ks, const void* vx, int64_t vs) {
  __shared__ float s_max[kWriteThreads / 32];
  const int b = blockIdx.y;
  const bool is_v = (blockIdx.z & 1) != 0;
  const int head = blockIdx.z >> 1;
  Seq q;
  if (!load_seq(c, b, q)) return;
  const int first = max(q.L - q.n, 0);  // rows at negative positions are skipped
  if (q.n == 0 || first >= q.L) return;
  const int pi = (first >> c.page_log2) + blockIdx.x;
  const int t0 = max(first, pi << c.page_log2), t1 = min(q.L, (pi + 1) << c.page_log2);
  if (t0 >= t1) return;
  const int page = load_page(c, b, pi);
  if (page < 0) return;
  const int rows = t1 - t0, at = t0 & (c.page - 1);
  const int dv = c.D >> 3;                       // 8-element vectors of a row
  const int r0 = threadIdx.x / dv, col = (threadIdx.x % dv) * 8;
  const int rstep = kWriteThreads / dv;
  const int64_t stride = is_v ? vs : ks;
  const char* src = static_cast<const char*>(is_v ? vx : kx);
  // row t0's place among the call's rows: its position less the first row's
  const int64_t row0 = static_cast<int64_t>(q.q0) + (t0 - (q.L - q.n));
  const size_t esz = VEC == 1 ? 2 : 4;
  uint4 raw[PASSES][VEC];
  float amax = 0.f;
  bool odd = false;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = r0 + p * rstep;
    if (r < rows) {
      const uint4* g = reinterpret_cast<const uint4*>(
          src + ((row0 + r) * stride + static_cast<int64_t>(head) * c.D + col) * esz);
#pragma unroll
      for (int i = 0; i < VEC; ++i) raw[p][i] = __ldg(g + i);
    }
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    if (r0 + p * rstep < rows) {
      float f[8];
      unpack8(raw[p], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = fabsf(f[i]);
        const bool finite = a <= 3.4028234663852886e38f;
        odd |= !finite;
        amax = fmaxf(amax, finite ? a : 0.f);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + static_cast<size_t>(page) * c.hkv + head;
  const float old = at ? *scale_at : 0.f;
  if (__syncthreads_or(odd) && threadIdx.x == 0) atomicOr(c.err, kErrNonFinite);
#pragma unroll
  for (int i = 0; i < kWriteThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
  const float need = block_scale(amax);
  const float scale = fmaxf(need, old);
  uint8_t* dst = (is_v ? c.v : c.k) +
                 (static_cast<size_t>(page) * c.hkv + head) * (static_cast<size_t>(c.page) * c.D);
  if (need > old && at) {
    // the earlier tokens' codes in the new scale (their slots are not this call's)
    const float ratio = old / scale;
    for (int i = threadIdx.x; i < at * dv; i += kWriteThreads) {
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
      for (int i = 0; i < 8; ++i) f[i] = f[i] == f[i] ? f[i] * inv : 0.f;
      const uint32_t a = encode2(f[0], f[1]) | (encode2(f[2], f[3]) << 16);
      const uint32_t z = encode2(f[4], f[5]) | (encode2(f[6], f[7]) << 16);
      *reinterpret_cast<uint2*>(dst + static_cast<size_t>(at + r) * c.D + col) = make_uint2(a, z);
    }
  }
  // (every thread has read the old scale before the barrier above)
  if (threadIdx.x == 0) *scale_at = scale;
}

constexpr int kReadThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const KvView c, T* ko, T* vo) {
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  T* out = is_v ? vo : ko;
  if (!out) return;
  Seq q;
  if (!load_seq(c, b, q)) return;
  const int per_head = c.D >> 4, per_tok = c.hkv * per_head;
  const int64_t it = static_cast<int64_t>(blockIdx.x) * kReadThreads + threadIdx.x;
  const int64_t row = it / per_tok;
  if (row >= q.n) return;
  const int r = static_cast<int>(it - row * per_tok), head = r / per_head, col = (r - head * per_head) * 16;
  const int t = q.L - q.n + static_cast<int>(row);
  uint4 u = make_uint4(0, 0, 0, 0);
  float s = 0.f;
  if (t >= 0) {
    const int page = load_page(c, b, t >> c.page_log2);
    if (page >= 0) {
      const size_t block = static_cast<size_t>(page) * c.hkv + head;
      s = (is_v ? c.v_scale : c.k_scale)[block];
      u = *reinterpret_cast<const uint4*>((is_v ? c.v : c.k) +
                                          (block * c.page + (t & (c.page - 1))) * c.D + col);
    }
  }
  T* dst = out + ((static_cast<size_t>(q.q0) + row) * c.hkv + head) * c.D + col;
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

template <int VEC>
cudaError_t write_dtype(const KvView& c, const void* k, int64_t ks, const void* v, int64_t vs,
                        cudaStream_t s) {
  // pages that n new tokens can touch
  const unsigned pages = static_cast<unsigned>((static_cast<int64_t>(c.max_q) + c.page - 2) / c.page + 1);
  const dim3 grid(pages, c.n_seqs, c.hkv * 2);
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
  const dim3 grid(static_cast<unsigned>((items + kReadThreads - 1) / kReadThreads), c.n_seqs, 2);
  if (dt == MOE_BF16)
    kv_read_kernel<__nv_bfloat16><<<grid, kReadThreads, 0, s>>>(
        c, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v));
  else
    kv_read_kernel<float><<<grid, kReadThreads, 0, s>>>(c, static_cast<float*>(k),
                                                        static_cast<float*>(v));
  return cudaGetLastError();
}

}  // namespace moe
