// Internal declarations of the attention-side operators (include/moe_attn.h).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe_attn.h"

namespace moe {

constexpr int kErrBadBatch = 2;   // device error bit: a batch broke its bounds
constexpr int kErrNonFinite = 4;  // device error bit: NaN or infinity written to the cache, or a scale not in [0, inf) met
constexpr float kMinBlockScale = 5.421010862427522e-20f;  // 2^-64

// What the kernels know of the cache and of a batch (by value).
struct KvView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* table;
  int table_stride;
  int n_seqs, n_tokens, max_q, max_kv;
  int n_pages, hkv, D, page, page_log2;
  int* err;
};

// One sequence of a batch: rows q0 .. q0 + n - 1, length L; row i's position
// is L - n + i.
struct Seq {
  int q0, n, L;
};

// False (and bit 1 of the error word) when the device arrays break the bounds
// that the launch was sized for.
__device__ __forceinline__ bool load_seq(const KvView& c, int b, Seq& s) {
  const int q0 = __ldg(c.cu_q + b), q1 = __ldg(c.cu_q + b + 1), L = __ldg(c.kv_len + b);
  s.q0 = q0;
  s.n = q1 - q0;
  s.L = L;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= c.n_tokens && s.n <= c.max_q && L >= 0 &&
                  L <= c.max_kv && ((L + c.page - 1) >> c.page_log2) <= c.table_stride;
  if (!ok) atomicOr(c.err, kErrBadBatch);
  return ok;
}

// The same in two steps, so that a prefetched entry is looked at only when it
// is used: the entry as it is, then its check.
__device__ __forceinline__ int raw_page(const KvView& c, int b, int i) {
  return __ldg(c.table + static_cast<size_t>(b) * c.table_stride + i);
}
__device__ __forceinline__ int checked_page(const KvView& c, int p, bool& bad) {
  const bool ok = static_cast<unsigned>(p) < static_cast<unsigned>(c.n_pages);
  bad |= !ok;
  return ok ? p : -1;
}

// Workspace of attend: partial results of row tiles whose keys are split over
// several CTAs, and the tiles' arrival counters (0 between calls: the last
// CTA of a tile resets its counter).
struct AttnWs {
  float* o;        // [cap_rows][D] unnormalised sums
  float2* ml;      // [cap_rows] running reference and weight sum
  unsigned* count; // [cap_rows / 16]
  size_t cap_rows;
};

struct AttnArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  float* lse;
  float scale_log2;  // softmax scale * log2(e)
  int causal, window, sinks;
  int hq, G;      // query heads, and those of a kv head
  float inv_g;    // 1 / G
};

// Groups of a batch's sequences that share a prefix (moe_kv_prefix_t).
struct Share {
  const int32_t* cu_seq;
  const int32_t* prefix_len;
  const int32_t* table;
  int table_stride, n_groups, max_tokens, max_len;
  int n_seqs;  // of the batch
};

cudaError_t rope_launch(const uint64_t* inc, int rot_dim, float amplitude, bool interleaved,
                        const moe_rope_tensor_t* q, const moe_rope_tensor_t* k, int head_dim,
                        moe_dtype_t dt, const int32_t* pos, int T, cudaStream_t s);
cudaError_t rope_axes_launch(const uint64_t* inc, const uint8_t* axis, int rot_dim, float amplitude, bool interleaved,
                             const moe_rope_tensor_t* q, const moe_rope_tensor_t* k, int head_dim, moe_dtype_t dt,
                             const int32_t* pos, int64_t pos_stride, int T, cudaStream_t s);
cudaError_t kv_write_launch(const KvView& c, const void* k, int64_t ks, const void* v, int64_t vs,
                            moe_dtype_t dt, cudaStream_t s);
cudaError_t kv_read_launch(const KvView& c, void* k, void* v, moe_dtype_t dt, cudaStream_t s);
// TMA maps of the code arrays as [n_pages][n_kv_heads * page_size][D] bytes, boxes
// of one page of one head, swizzled in D-byte rows.
struct KvMaps {
  CUtensorMap k_tile, v_tile;
};
bool kv_create_maps(const moe_kv_config_t& cfg, const moe_kv_store_t& st, KvMaps* m);
cudaError_t attn_few_launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const KvMaps& maps,
                            int n_sm, cudaStream_t s);
// Attention of a batch whose sequences share prefixes; the workspace holds the partial
// results of rows over their prefix and over their own tokens; nothing is launched where
// it has fewer bytes than *need.
size_t attn_shared_workspace(const KvView& c, const Share& sh, int G, int n_sm);
cudaError_t attn_shared_launch(const KvView& c, const AttnArgs& a, const Share& sh, const AttnWs& handle_ws, void* workspace,
                               size_t have, size_t* need, const KvMaps& maps, int n_sm, cudaStream_t s);
cudaError_t attn_tiles_launch(const KvView& c, const AttnArgs& a, const AttnWs& ws, const KvMaps& maps,
                              int n_sm, cudaStream_t s);

}  // namespace moe
