// Rotary positions (moe_rope_apply).
//
// The angles' sines and cosines of a CTA's tokens go to shared memory once for
// all heads; then a thread holds its 8 pairs' ones in registers and streams
// its place of the token's heads (8 pairs, or 16 copied elements).  The angle
// of pair i at position p is p * inc[i] mod 2^64, a 64-bit fraction of a turn:
// an integer product wraps exactly, so far positions lose nothing.  The nearest
// quarter turn is taken off in integers, and what fp32 cannot hold of the rest's
// 30 bits turns the sine and cosine by their derivatives: the angle that goes in
// is exact to 2^-33 turns, where the phase as one fp32 number would be off by up
// to 2^-26.  Several axes are a position for each pair, picked where its phase is worked out.
//
// Bound by memory: x is read once and y written once.  A thread's next heads are on their
// way while it turns the ones at hand, the first ones under the angles, and small CTAs,
// seven of them a SM in bf16, are in different phases (8192 tokens of 56 heads of 128, bf16:
// 36.8 us, 6.4 TB/s; CTAs of 256 threads and four tokens 40.8 us, without the loads ahead
// 42.8 us; fp32, whose registers allow four of the CTAs, 70.2 us, 6.7 TB/s).
#include "attn_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kItems = 2;   // heads of a thread under way, twice
constexpr int kTokens = 2;  // most tokens of a CTA

struct RopeParams {
  uint64_t inc[128];  // fraction of a turn per position, 64-bit fixed point
  const void* x[2];
  const void* y[2];
  int64_t xs[2], ys[2];
  const int32_t* pos;
  int64_t pos_stride;  // between axes
  float amplitude;
  int heads[2];
  int rot, head_dim, T, tokens;
  uint8_t axis[128];
};

// 8 elements as they lie, and as fp32
template <typename T>
struct Raw {
  static constexpr int kVec = sizeof(T) / 2;
  uint4 v[kVec];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (kVec == 1) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(v[i].x), f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z), f[4 * i + 3] = __uint_as_float(v[i].w);
      }
    }
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    if constexpr (kVec == 1) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
    }
  }
};

template <typename T, bool INTERLEAVED, bool AXES>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 7 : 1) rope_kernel(const __grid_constant__ RopeParams P) {
  __shared__ float2 cs[kTokens][128];  // cosine, sine
  const int half = P.rot >> 1;
  const int t0 = blockIdx.x * P.tokens, tn = min(P.tokens, P.T - t0);
  // a thread's place c in a head is fixed: elements ia .. ia + 7 and ib .. ib + 7
  const int per_head = P.head_dim >> 4;
  const int h0 = threadIdx.x / per_head, c = threadIdx.x - h0 * per_head;
  const int hstep = blockDim.x / per_head, heads = P.heads[0] + P.heads[1];
  const bool turned = c < (P.rot >> 4);
  int ia = 16 * c, ib = 16 * c + 8;
  if (!INTERLEAVED && turned) ia = 8 * c, ib = 8 * c + half;
  auto at = [&](const void* const (&base)[2], const int64_t (&stride)[2], int t, int h) {
    const int w = h >= P.heads[0];
    return static_cast<const T*>(base[w]) + (t0 + t) * stride[w] + (h - (w ? P.heads[0] : 0)) * P.head_dim;
  };
  Raw<T> a[kItems], b[kItems], a1[kItems], b1[kItems];
  auto load = [&](Raw<T>(&x)[kItems], Raw<T>(&y)[kItems], int t, int h) {
#pragma unroll
    for (int n = 0; n < kItems; ++n) {
      if (t < tn && h + n * hstep < heads) {
        const T* p = at(P.x, P.xs, t, h + n * hstep);
        x[n].load(p + ia);
        y[n].load(p + ib);
      }
    }
  };
  // the first heads are on their way while the angles are worked out
  load(a, b, 0, h0);
  for (int i = threadIdx.x; i < tn * half; i += blockDim.x) {
    const int tk = i / half, pair = i - tk * half;
    const int32_t* pos = P.pos + t0 + tk;
    if constexpr (AXES) pos += P.axis[pair] * P.pos_stride;
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(__ldg(pos))) * P.inc[pair];
    const uint32_t turn = static_cast<uint32_t>((phase + 0x80000000u) >> 32);  // in 2^-32 turns
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(turn - (quarter << 30));  // [-2^29, 2^29)
    const float hi = static_cast<float>(rest);
    const float lo = static_cast<float>(rest - static_cast<int32_t>(hi)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    float s0, c0;
    sincospif(hi * 4.6566128730773926e-10f, &s0, &c0);  // 2^-31: half turns
    const float s1 = fmaf(c0, lo, s0), c1 = fmaf(-s0, lo, c0);
    float s = quarter & 1 ? c1 : s1, c = quarter & 1 ? s1 : c1;
    s = quarter & 2 ? -s : s;
    c = (quarter + 1) & 2 ? -c : c;
    cs[tk][pair] = make_float2(c * P.amplitude, s * P.amplitude);
  }
  __syncthreads();
  for (int t = 0; t < tn; ++t) {
    float2 r[8];
    if (turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = cs[t][8 * c + i];
    }
    for (int h = h0; h < heads; h += kItems * hstep) {
      // the next heads, this token's or the next one's
      const bool more = h + kItems * hstep < heads;
      load(a1, b1, more ? t : t + 1, more ? h + kItems * hstep : h0);
#pragma unroll
      for (int n = 0; n < kItems; ++n) {
        if (h + n * hstep >= heads) break;
        if (turned) {
          float f[8], g[8];
          a[n].get(f);
          b[n].get(g);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float& u = !INTERLEAVED ? f[i] : i < 4 ? f[2 * i] : g[2 * i - 8];
            float& v = !INTERLEAVED ? g[i] : i < 4 ? f[2 * i + 1] : g[2 * i - 7];
            const float u0 = u, v0 = v;
            u = u0 * r[i].x - v0 * r[i].y;
            v = u0 * r[i].y + v0 * r[i].x;
          }
          a[n].put(f);
          b[n].put(g);
        }
        T* y = const_cast<T*>(at(P.y, P.ys, t, h + n * hstep));
        a[n].store(y + ia);
        b[n].store(y + ib);
      }
#pragma unroll
      for (int n = 0; n < kItems; ++n) a[n] = a1[n], b[n] = b1[n];
    }
  }
}

template <bool AXES>
cudaError_t launch(const uint64_t* inc, const uint8_t* axis, int rot_dim, float amplitude, bool interleaved,
                   const moe_rope_tensor_t* q, const moe_rope_tensor_t* k, int head_dim, moe_dtype_t dt, const int32_t* pos,
                   int64_t pos_stride, int T, cudaStream_t s) {
  RopeParams P;
  for (int i = 0; i < 128; ++i) {
    P.inc[i] = i < rot_dim / 2 ? inc[i] : 0;
    P.axis[i] = axis && i < rot_dim / 2 ? axis[i] : 0;
  }
  const moe_rope_tensor_t* ts[2] = {q, k};
  for (int w = 0; w < 2; ++w) {
    P.x[w] = ts[w] ? ts[w]->x : nullptr;
    P.y[w] = ts[w] ? ts[w]->y : nullptr;
    P.xs[w] = ts[w] ? ts[w]->x_stride : 0;
    P.ys[w] = ts[w] ? ts[w]->y_stride : 0;
    P.heads[w] = ts[w] ? ts[w]->n_heads : 0;
  }
  P.pos = pos;
  P.pos_stride = pos_stride;
  P.amplitude = amplitude;
  P.rot = rot_dim;
  P.head_dim = head_dim;
  P.T = T;
  // one token a CTA while that fills the device once; two share the angles' phase then
  // (8192 tokens of 32 + 2 heads of 64: 15.2 us, and 17.8 us with one)
  P.tokens = T >= 2048 ? kTokens : 1;
  const int per_head = head_dim / 16, threads = kThreads / per_head * per_head;
  const int grid = (T + P.tokens - 1) / P.tokens;
  if (dt == MOE_BF16) {
    if (interleaved)
      rope_kernel<__nv_bfloat16, true, AXES><<<grid, threads, 0, s>>>(P);
    else
      rope_kernel<__nv_bfloat16, false, AXES><<<grid, threads, 0, s>>>(P);
  } else {
    if (interleaved)
      rope_kernel<float, true, AXES><<<grid, threads, 0, s>>>(P);
    else
      rope_kernel<float, false, AXES><<<grid, threads, 0, s>>>(P);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t rope_launch(const uint64_t* inc, int rot_dim, float amplitude, bool interleaved,
                        const moe_rope_tensor_t* q, const moe_rope_tensor_t* k, int head_dim,
                        moe_dtype_t dt, const int32_t* pos, int T, cudaStream_t s) {
  return launch<false>(inc, nullptr, rot_dim, amplitude, interleaved, q, k, head_dim, dt, pos, 0, T, s);
}

cudaError_t rope_axes_launch(const uint64_t* inc, const uint8_t* axis, int rot_dim, float amplitude, bool interleaved,
                             const moe_rope_tensor_t* q, const moe_rope_tensor_t* k, int head_dim, moe_dtype_t dt,
                             const int32_t* pos, int64_t pos_stride, int T, cudaStream_t s) {
  return launch<true>(inc, axis, rot_dim, amplitude, interleaved, q, k, head_dim, dt, pos, pos_stride, T, s);
}

}  // namespace moe
