// Rotary positions (moe_rope_apply).
//
// One CTA a token: the angles' sines and cosines go to shared memory once for
// all heads, then the threads stream the token's heads, 16 elements (8 pairs,
// or 16 copied elements) an item.  The angle of pair i at position p is p *
// inc[i] mod 2^64, a 64-bit fraction of a turn: an integer product wraps
// exactly, so far positions lose nothing.  Bound by memory: x is read once and
// y written once.
#include "attn_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct RopeParams {
  uint64_t inc[128];  // fraction of a turn per position, 64-bit fixed point
  const void* x[2];
  void* y[2];
  int64_t xs[2], ys[2];
  const int32_t* pos;
  float amplitude;
  int heads[2];
  int rot, head_dim;
};

struct V8 {
  float f[8];
};

template <typename T>
__device__ __forceinline__ V8 load8(const T* p);
template <>
__device__ __forceinline__ V8 load8<float>(const float* p) {
  V8 v;
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v.f[0] = a.x, v.f[1] = a.y, v.f[2] = a.z, v.f[3] = a.w;
  v.f[4] = b.x, v.f[5] = b.y, v.f[6] = b.z, v.f[7] = b.w;
  return v;
}
template <>
__device__ __forceinline__ V8 load8<__nv_bfloat16>(const __nv_bfloat16* p) {
  V8 v;
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.f[2 * i] = __uint_as_float(w[i] << 16);
    v.f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return v;
}
__device__ __forceinline__ void store8(float* p, const V8& v) {
  *reinterpret_cast<float4*>(p) = make_float4(v.f[0], v.f[1], v.f[2], v.f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v.f[4], v.f[5], v.f[6], v.f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const V8& v) {
  uint4 a;
  uint32_t* w = &a.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.f[2 * i], v.f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = a;
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams P) {
  __shared__ float2 cs[128];  // cosine, sine
  const int t = blockIdx.x;
  const int half = P.rot >> 1;
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(P.pos[t])) * P.inc[i];
    // the top 32 bits as a signed number of half turns in [-1, 1)
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.6566128730773926e-10f, &s, &c);
    cs[i] = make_float2(c * P.amplitude, s * P.amplitude);
  }
  __syncthreads();
  const int per_head = P.head_dim >> 4;
  const int turned = P.rot >> 4;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const T* x = static_cast<const T*>(P.x[w]) + t * P.xs[w];
    T* y = static_cast<T*>(P.y[w]) + t * P.ys[w];
    const int items = P.heads[w] * per_head;
    for (int it = threadIdx.x; it < items; it += kThreads) {
      const int h = it / per_head, c = it - h * per_head;
      const size_t base = static_cast<size_t>(h) * P.head_dim;
      size_t ia = base + 16 * c, ib = ia + 8;
      if (!INTERLEAVED && c < turned) ia = base + 8 * c, ib = ia + half;
      V8 a = load8<T>(x + ia), b = load8<T>(x + ib);
      if (c < turned) {
        const float2* q = cs + 8 * c;
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 r = q[i], z = q[i + 4];
            const float a0 = a.f[2 * i], a1 = a.f[2 * i + 1];
            a.f[2 * i] = a0 * r.x - a1 * r.y;
            a.f[2 * i + 1] = a0 * r.y + a1 * r.x;
            const float b0 = b.f[2 * i], b1 = b.f[2 * i + 1];
            b.f[2 * i] = b0 * z.x - b1 * z.y;
            b.f[2 * i + 1] = b0 * z.y + b1 * z.x;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 r = q[i];
            const float a0 = a.f[i], b0 = b.f[i];
            a.f[i] = a0 * r.x - b0 * r.y;
            b.f[i] = a0 * r.y + b0 * r.x;
          }
        }
      }
      store8(y + ia, a);
      store8(y + ib, b);
    }
  }
}

}  // namespace

cudaError_t rope_launch(const uint64_t* inc, int rot_dim, float amplitude, bool interleaved,
                        const moe_rope_tensor_t* q, const moe_rope_tensor_t* k, int head_dim,
                        moe_dtype_t dt, const int32_t* pos, int T, cudaStream_t s) {
  RopeParams P;
  for (int i = 0; i < 128; ++i) P.inc[i] = i < rot_dim / 2 ? inc[i] : 0;
  const moe_rope_tensor_t* ts[2] = {q, k};
  for (int w = 0; w < 2; ++w) {
    P.x[w] = ts[w] ? ts[w]->x : nullptr;
    P.y[w] = ts[w] ? ts[w]->y : nullptr;
    P.xs[w] = ts[w] ? ts[w]->x_stride : 0;
    P.ys[w] = ts[w] ? ts[w]->y_stride : 0;
    P.heads[w] = ts[w] ? ts[w]->n_heads : 0;
  }
  P.pos = pos;
  P.amplitude = amplitude;
  P.rot = rot_dim;
  P.head_dim = head_dim;
  if (dt == MOE_BF16) {
    if (interleaved)
      rope_kernel<__nv_bfloat16, true><<<T, kThreads, 0, s>>>(P);
    else
      rope_kernel<__nv_bfloat16, false><<<T, kThreads, 0, s>>>(P);
  } else {
    if (interleaved)
      rope_kernel<float, true><<<T, kThreads, 0, s>>>(P);
    else
      rope_kernel<float, false><<<T, kThreads, 0, s>>>(P);
  }
  return cudaGetLastError();
}

}  // namespace moe
