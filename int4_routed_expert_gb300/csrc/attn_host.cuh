// What the host sides of the attention-side entry points share: handles, messages,
// argument checks, the device that a call works on.
#pragma once

#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "attn_internal.cuh"
#include "moe_internal.cuh"

namespace moe {

// What every handle of these entry points has.
struct HandleBase {
  int device;
  char msg[512];
};

}  // namespace moe

struct moe_rope {
  int rot_dim;
  float amplitude;
  bool interleaved;
  int n_axes;
  uint64_t inc[128];
  uint8_t axis[128];  // of each pair
};

struct moe_kv : moe::HandleBase {
  moe_kv_config_t cfg;
  moe_kv_store_t st;
  int n_sm;
  void* base;  // workspace
  moe::AttnWs ws;
  moe::KvMaps maps;
  size_t count_bytes;
  int* err;  // device error word
};

namespace moe {

inline void fail(HandleBase* h, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  if (h)
    snprintf(h->msg, sizeof(h->msg), "%s", text);
  else
    set_thread_error("%s", text);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A tensor as the kernels address it, or NULL with the reason in *why.  Device
// memory has to lie on *device; -1 becomes the tensor's device.
inline const void* resolve(const void* p, int* device, const char** why) {
  if (!p) {
    *why = "is NULL";
    return nullptr;
  }
  if (!aligned16(p)) {
    *why = "must be 16-byte aligned";
    return nullptr;
  }
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    *why = "is not known to the CUDA driver";
    return nullptr;
  }
  if (at.type == cudaMemoryTypeDevice && *device < 0) *device = at.device;
  if (at.type == cudaMemoryTypeDevice && at.device != *device) {
    *why = "lies on another device than the handle or the first tensor";
    return nullptr;
  }
  if (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) return p;
  if (at.type == cudaMemoryTypeHost && at.devicePointer) return at.devicePointer;
  *why = "must be device memory or mapped pinned host memory";
  return nullptr;
}

inline const char* check_dtype(moe_dtype_t dt) {
  return dt == MOE_F32 || dt == MOE_BF16 ? nullptr : "dtype must be MOE_F32 or MOE_BF16";
}

// Checks a batch (shapes, bounds, pointers); fills the kernels' view of it.
inline moe_status_t view(moe_kv_t* h, const moe_kv_batch_t* b, KvView* v) {
  const moe_kv_config_t& c = h->cfg;
  if (!b) {
    fail(h, "batch is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  if (b->n_seqs < 0 || b->n_tokens < 0 || b->max_q_len < 0 || b->max_kv_len < 0) {
    fail(h, "batch sizes must not be negative");
    return MOE_ERR_INVALID_ARG;
  }
  if (b->n_seqs > c.max_seqs || b->n_tokens > c.max_tokens || b->max_kv_len > c.max_kv_len) {
    fail(h, "batch of %d sequences, %d tokens and %d cached tokens exceeds the handle's %d, %d, %d",
         b->n_seqs, b->n_tokens, b->max_kv_len, c.max_seqs, c.max_tokens, c.max_kv_len);
    return MOE_ERR_CAPACITY;
  }
  if (b->n_seqs == 0 || b->n_tokens == 0) return MOE_OK;
  if (b->max_q_len < 1 || b->max_q_len > b->n_tokens) {
    fail(h, "max_q_len must be in [1, n_tokens], got %d", b->max_q_len);
    return MOE_ERR_INVALID_ARG;
  }
  if (b->table_stride < 1) {
    fail(h, "table_stride must be at least 1");
    return MOE_ERR_INVALID_ARG;
  }
  const void* p[3] = {b->cu_q, b->kv_len, b->page_table};
  const char* name[3] = {"cu_q", "kv_len", "page_table"};
  for (int i = 0; i < 3; ++i) {
    const char* why = nullptr;
    p[i] = resolve(p[i], &h->device, &why);
    if (!p[i]) {
      fail(h, "%s %s", name[i], why);
      return MOE_ERR_INVALID_ARG;
    }
  }
  int log2 = 0;
  while ((1 << log2) < c.page_size) ++log2;
  *v = KvView{h->st.k, h->st.v, h->st.k_scale, h->st.v_scale,
              static_cast<const int32_t*>(p[0]), static_cast<const int32_t*>(p[1]),
              static_cast<const int32_t*>(p[2]), b->table_stride, b->n_seqs, b->n_tokens,
              b->max_q_len, b->max_kv_len, c.n_pages, c.n_kv_heads, c.head_dim, c.page_size,
              log2, h->err};
  return MOE_OK;
}

inline moe_status_t check_stride(HandleBase* h, const char* name, int64_t stride, int64_t row, size_t esz) {
  if (stride < row || (stride * static_cast<int64_t>(esz)) % 16 != 0 || stride > (1LL << 40)) {
    fail(h, "%s must be at least %lld elements and a multiple of 16 bytes, got %lld", name,
         static_cast<long long>(row), static_cast<long long>(stride));
    return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

inline moe_status_t tensor(HandleBase* h, int* device, const char* name, const void** p) {
  const char* why = nullptr;
  const void* r = resolve(*p, device, &why);
  if (!r) {
    fail(h, "%s %s", name, why);
    return MOE_ERR_INVALID_ARG;
  }
  *p = r;
  return MOE_OK;
}

// Checks a rotation's arguments: its tensors as the kernels address them, and their device.
inline moe_status_t rope_args(const moe_rope_t* r, const moe_rope_tensor_t* q, const moe_rope_tensor_t* k, int head_dim,
                              moe_dtype_t dtype, int n_tokens, moe_rope_tensor_t (&t)[2], int& device) {
  if (!r || !q) {
    fail(nullptr, "the rope handle or q is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  if (head_dim % 16 != 0 || head_dim < r->rot_dim || head_dim > 256) {
    fail(nullptr, "head_dim must be a multiple of 16 in [%d, 256], got %d", r->rot_dim, head_dim);
    return MOE_ERR_UNSUPPORTED;
  }
  if (const char* m = check_dtype(dtype)) {
    fail(nullptr, "%s", m);
    return MOE_ERR_INVALID_ARG;
  }
  if (n_tokens < 0) {
    fail(nullptr, "n_tokens must be >= 0 (got %d)", n_tokens);
    return MOE_ERR_INVALID_ARG;
  }
  const size_t esz = dtype == MOE_BF16 ? 2 : 4;
  const moe_rope_tensor_t* in[2] = {q, k};
  const char* names[2][4] = {{"q.x", "q.y", "q.x_stride", "q.y_stride"},
                             {"k.x", "k.y", "k.x_stride", "k.y_stride"}};
  device = -1;
  for (int w = 0; w < 2; ++w) {
    if (!in[w]) continue;
    t[w] = *in[w];
    if (t[w].n_heads < 1 || t[w].n_heads > 4096) {
      fail(nullptr, "n_heads must be in [1, 4096], got %d", t[w].n_heads);
      return MOE_ERR_UNSUPPORTED;
    }
    const int64_t row = static_cast<int64_t>(t[w].n_heads) * head_dim;
    moe_status_t st = check_stride(nullptr, names[w][2], t[w].x_stride, row, esz);
    if (st == MOE_OK) st = check_stride(nullptr, names[w][3], t[w].y_stride, row, esz);
    if (st != MOE_OK) return st;
    if (n_tokens == 0) continue;
    if ((st = tensor(nullptr, &device, names[w][0], &t[w].x)) != MOE_OK) return st;
    const void* y = t[w].y;
    if ((st = tensor(nullptr, &device, names[w][1], &y)) != MOE_OK) return st;
    t[w].y = const_cast<void*>(y);
    if (t[w].x == t[w].y && t[w].x_stride != t[w].y_stride) {
      fail(nullptr, "in place, %s and %s must be equal", names[w][2], names[w][3]);
      return MOE_ERR_INVALID_ARG;
    }
  }
  return MOE_OK;
}

// Checks attention's arguments; fills the kernels' view of the batch (n_seqs is 0 where
// there is nothing to do) and their arguments.
inline moe_status_t attend_args(moe_kv_t* h, const void* q, int64_t q_stride, void* out, float* lse,
                                const moe_kv_mask_t* mask, const moe_kv_batch_t* batch, KvView* view_out, AttnArgs* args) {
  if (!mask) {
    fail(h, "mask is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  const float scale_log2 = mask->scale * 1.4426950408889634f;
  if (!isfinite(scale_log2)) {
    fail(h, "scale must be finite, in base 2 too");
    return MOE_ERR_INVALID_ARG;
  }
  if (mask->window < 0 || mask->sinks < 0) {
    fail(h, "window and sinks must not be negative (got %d, %d)", mask->window, mask->sinks);
    return MOE_ERR_INVALID_ARG;
  }
  if (!mask->causal && (mask->window || mask->sinks)) {
    fail(h, "window and sinks need causal != 0");
    return MOE_ERR_INVALID_ARG;
  }
  moe_status_t st = view(h, batch, view_out);
  const KvView& c = *view_out;
  if (st != MOE_OK || c.n_seqs == 0) return st;
  if (static_cast<int64_t>(c.n_tokens) * h->cfg.n_q_heads > INT_MAX) {  // the kernels number rows in 32 bits
    fail(h, "%d tokens of %d query heads are more rows than one call takes", c.n_tokens, h->cfg.n_q_heads);
    return MOE_ERR_UNSUPPORTED;
  }
  const int64_t row = static_cast<int64_t>(h->cfg.n_q_heads) * h->cfg.head_dim;
  if ((st = check_stride(h, "q_stride", q_stride, row, 2)) != MOE_OK) return st;
  const void *o = out, *z = lse;
  if ((st = tensor(h, &h->device, "q", &q)) != MOE_OK) return st;
  if ((st = tensor(h, &h->device, "out", &o)) != MOE_OK) return st;
  if (lse && (st = tensor(h, &h->device, "lse", &z)) != MOE_OK) return st;
  AttnArgs& a = *args;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<__nv_bfloat16*>(const_cast<void*>(o));
  a.lse = static_cast<float*>(const_cast<void*>(z));
  a.scale_log2 = scale_log2;
  a.causal = mask->causal != 0;
  // a window that reaches every cached token is none
  a.window = mask->window >= c.max_kv ? 0 : mask->window;
  a.sinks = a.window ? mask->sinks : 0;
  a.hq = h->cfg.n_q_heads;
  a.G = h->cfg.n_q_heads / h->cfg.n_kv_heads;
  a.inv_g = 1.f / static_cast<float>(a.G);
  return MOE_OK;
}

// Makes a device current while a call works on it, and the caller's again.  A
// launch (and the stream NULL) goes to the current device, which need not be the
// one whose memory the call was given.
class OnDevice {
 public:
  explicit OnDevice(int device) {
    error = cudaGetDevice(&back_);
    if (error != cudaSuccess || device < 0 || back_ == device)
      back_ = -1;
    else
      error = cudaSetDevice(device);
  }
  ~OnDevice() {
    if (back_ >= 0) cudaSetDevice(back_);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;
  cudaError_t error;

 private:
  int back_ = -1;
};

inline moe_status_t launched(HandleBase* h, cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  fail(h, "%s: %s", what, cudaGetErrorString(e));
  return MOE_ERR_CUDA;
}

}  // namespace moe
