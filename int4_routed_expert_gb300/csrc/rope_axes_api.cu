// C ABI of rotary positions with several axes (include/moe_attn.h): argument checks.
#include "attn_host.cuh"

extern "C" moe_status_t moe_rope_apply_axes(const moe_rope_t* r, const moe_rope_tensor_t* q, const moe_rope_tensor_t* k,
                                            int head_dim, moe_dtype_t dtype, const int32_t* positions,
                                            int64_t position_stride, int n_tokens, void* stream) {
  using namespace moe;
  moe_rope_tensor_t t[2];
  int device;
  if (const moe_status_t st = rope_args(r, q, k, head_dim, dtype, n_tokens, t, device); st != MOE_OK) return st;
  if (position_stride < n_tokens || position_stride > (1LL << 40)) {
    fail(nullptr, "position_stride must be at least n_tokens, got %lld", static_cast<long long>(position_stride));
    return MOE_ERR_INVALID_ARG;
  }
  if (n_tokens == 0) return MOE_OK;
  const void* pos = positions;
  if (const moe_status_t st = tensor(nullptr, &device, "positions", &pos); st != MOE_OK) return st;
  const OnDevice on(device);
  if (on.error != cudaSuccess) return launched(nullptr, on.error, "moe_rope_apply_axes");
  return launched(nullptr,
                  rope_axes_launch(r->inc, r->axis, r->rot_dim, r->amplitude, r->interleaved, &t[0], k ? &t[1] : nullptr,
                                   head_dim, dtype, static_cast<const int32_t*>(pos), position_stride, n_tokens,
                                   static_cast<cudaStream_t>(stream)),
                  "moe_rope_apply_axes");
}
