// C ABI of the attention-side operators (include/moe_attn.h): argument checks,
// workspace, dispatch.
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <new>

#include "attn_internal.cuh"
#include "moe_internal.cuh"

struct moe_rope {
  int rot_dim;
  float amplitude;
  bool interleaved;
  uint64_t inc[128];
};

struct moe_kv {
  moe_kv_config_t cfg;
  moe_kv_store_t st;
  int device, n_sm;
  void* base;  // workspace
  moe::AttnWs ws;
  moe::KvMaps maps;
  size_t count_bytes;
  int* err;  // device error word
  char msg[512];
};

namespace {

void fail(moe_kv_t* h, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  if (h)
    snprintf(h->msg, sizeof(h->msg), "%s", text);
  else
    moe::set_thread_error("%s", text);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A tensor as the kernels address it, or NULL with the reason in *why.  Device
// memory has to lie on *device; -1 becomes the tensor's device.
const void* resolve(const void* p, int* device, const char** why) {
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

const char* check_dtype(moe_dtype_t dt) {
  return dt == MOE_F32 || dt == MOE_BF16 ? nullptr : "dtype must be MOE_F32 or MOE_BF16";
}

// x in [0, 1) as a 64-bit fraction: two 32-bit steps carry every bit down to 2^-64.
uint64_t fixed64(double x) {
  const double hi = floor(x * 4294967296.0);
  const double lo = (x * 4294967296.0 - hi) * 4294967296.0;
  return (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo + 0.5);
}

// |f| / (2 pi) mod 1 as a 64-bit fraction of a turn.  A double of the quotient
// is off by 2^-56 of a turn, which a position of 2^31 makes 2^-25; so 2 pi and the
// quotient have a second double each, and what is left is the fraction's own
// step, for |f| below 2^38.
uint64_t turn_fraction(double f) {
  constexpr double kHi = 6.283185307179586477, kLo = 2.4492935982947064e-16;  // 2 pi
  f = fabs(f);
  const double q1 = f / kHi;
  const double q2 = fma(-q1, kLo, fma(-q1, kHi, f)) / kHi;
  const double a1 = q1 - floor(q1), a2 = fabs(q2) - floor(fabs(q2));
  return q2 < 0 ? fixed64(a1) - fixed64(a2) : fixed64(a1) + fixed64(a2);
}

const char* check_kv_config(const moe_kv_config_t* c) {
  if (!c) return "cfg is NULL";
  if (c->n_kv_heads < 1 || c->n_kv_heads > 256) return "n_kv_heads must be in [1, 256]";
  if (c->n_q_heads < 1 || c->n_q_heads % c->n_kv_heads != 0 || c->n_q_heads > 4096)
    return "n_q_heads must be a multiple of n_kv_heads, at most 4096";
  if (c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 64 or 128";
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return "page_size must be 16, 32, 64 or 128";
  if (c->n_pages < 1) return "n_pages must be at least 1";
  if (c->max_seqs < 1 || c->max_seqs > 65535) return "max_seqs must be in [1, 65535]";
  if (c->max_tokens < 1 || c->max_tokens > (1 << 24)) return "max_tokens must be in [1, 2^24]";
  if (c->max_kv_len < 1 || c->max_kv_len > (1 << 30)) return "max_kv_len must be in [1, 2^30]";
  return nullptr;
}

// Rows of partial results: as many as the largest call within the handle's bounds
// can use, that is every tile of keys of every row tile a split (at most 256, or
// 4096 rows in the kernel for few rows), but at most 2^18 (64 or 128 MB of sums):
// six CTAs of 256 rows a SM.  The splits of a call are limited to what fits.
size_t part_rows(const moe_kv_config_t* c) {
  const int64_t tiles = (static_cast<int64_t>(c->max_kv_len) + 127) / 128;
  const int64_t heads = static_cast<int64_t>(c->n_kv_heads) * c->max_seqs;
  const int64_t rows = static_cast<int64_t>(c->max_tokens) * (c->n_q_heads / c->n_kv_heads);
  const int64_t few = heads * std::min<int64_t>(32 * tiles, 4096);
  const int64_t most = rows > 32 ? (rows + 255) / 256 * 256 * std::min<int64_t>(tiles, 256) : 0;
  constexpr int64_t kEnd = 1 << 18;
  return static_cast<size_t>(std::min(kEnd, std::max(few, most >= kEnd ? kEnd : heads * most)));
}

struct KvLayout {
  size_t rows, o, ml, count, err, total;
};
KvLayout kv_layout(const moe_kv_config_t* c) {
  KvLayout L;
  L.rows = part_rows(c);
  L.o = 0;
  L.ml = L.o + L.rows * c->head_dim * 4;
  L.count = L.ml + L.rows * 8;
  L.err = L.count + L.rows / 16 * 4;
  L.total = L.err + 256;
  return L;
}

// Checks a batch (shapes, bounds, pointers); fills the kernels' view of it.
moe_status_t view(moe_kv_t* h, const moe_kv_batch_t* b, moe::KvView* v) {
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
  *v = moe::KvView{h->st.k, h->st.v, h->st.k_scale, h->st.v_scale,
                   static_cast<const int32_t*>(p[0]), static_cast<const int32_t*>(p[1]),
                   static_cast<const int32_t*>(p[2]), b->table_stride, b->n_seqs, b->n_tokens,
                   b->max_q_len, b->max_kv_len, c.n_pages, c.n_kv_heads, c.head_dim, c.page_size,
                   log2, h->err};
  return MOE_OK;
}

moe_status_t check_stride(moe_kv_t* h, const char* name, int64_t stride, int64_t row, size_t esz) {
  if (stride < row || (stride * static_cast<int64_t>(esz)) % 16 != 0 || stride > (1LL << 40)) {
    fail(h, "%s must be at least %lld elements and a multiple of 16 bytes, got %lld", name,
         static_cast<long long>(row), static_cast<long long>(stride));
    return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

moe_status_t tensor(moe_kv_t* h, int* device, const char* name, const void** p) {
  const char* why = nullptr;
  const void* r = resolve(*p, device, &why);
  if (!r) {
    fail(h, "%s %s", name, why);
    return MOE_ERR_INVALID_ARG;
  }
  *p = r;
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

moe_status_t launched(moe_kv_t* h, cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  fail(h, "%s: %s", what, cudaGetErrorString(e));
  return MOE_ERR_CUDA;
}

}  // namespace

namespace moe {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

bool kv_create_maps(const moe_kv_config_t& cfg, const moe_kv_store_t& st, KvMaps* m) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
          cudaSuccess ||
      q != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return false;
  }
  const EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(p);
  const cuuint64_t D = cfg.head_dim, rows = static_cast<cuuint64_t>(cfg.n_kv_heads) * cfg.page_size;
  const cuuint64_t dims[3] = {D, rows, static_cast<cuuint64_t>(cfg.n_pages)};
  const cuuint64_t strides[2] = {D, rows * D};
  const cuuint32_t es[3] = {1, 1, 1};
  auto make = [&](CUtensorMap* map, uint8_t* base, int box_rows) {
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(box_rows), 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return make(&m->k_tile, st.k, cfg.page_size) && make(&m->v_tile, st.v, cfg.page_size);
}

}  // namespace moe

extern "C" {

moe_status_t moe_rope_create(int rot_dim, const double* inv_freq, float amplitude,
                             int interleaved, moe_rope_t** out) {
  if (!out) {
    fail(nullptr, "out is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  *out = nullptr;
  if (rot_dim < 16 || rot_dim > 256 || rot_dim % 16 != 0) {
    fail(nullptr, "rot_dim must be a multiple of 16 in [16, 256], got %d", rot_dim);
    return MOE_ERR_UNSUPPORTED;
  }
  if (!inv_freq) {
    fail(nullptr, "inv_freq is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  if (!isfinite(amplitude)) {
    fail(nullptr, "amplitude must be finite");
    return MOE_ERR_INVALID_ARG;
  }
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!isfinite(inv_freq[i])) {
      fail(nullptr, "inv_freq[%d] must be finite", i);
      return MOE_ERR_INVALID_ARG;
    }
  moe_rope_t* r = new (std::nothrow) moe_rope();
  if (!r) {
    fail(nullptr, "host allocation failed");
    return MOE_ERR_OOM;
  }
  r->rot_dim = rot_dim;
  r->amplitude = amplitude;
  r->interleaved = interleaved != 0;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const uint64_t turn = turn_fraction(inv_freq[i]);
    r->inc[i] = inv_freq[i] < 0 ? 0 - turn : turn;
  }
  *out = r;
  return MOE_OK;
}

void moe_rope_destroy(moe_rope_t* r) { delete r; }

moe_status_t moe_rope_apply(const moe_rope_t* r, const moe_rope_tensor_t* q,
                            const moe_rope_tensor_t* k, int head_dim, moe_dtype_t dtype,
                            const int32_t* positions, int n_tokens, void* stream) {
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
  moe_rope_tensor_t t[2];
  int device = -1;
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
  if (n_tokens == 0) return MOE_OK;
  const void* pos = positions;
  if (const moe_status_t st = tensor(nullptr, &device, "positions", &pos); st != MOE_OK) return st;
  const OnDevice on(device);
  if (on.error != cudaSuccess) return launched(nullptr, on.error, "moe_rope_apply");
  return launched(nullptr,
                  moe::rope_launch(r->inc, r->rot_dim, r->amplitude, r->interleaved, &t[0],
                                   k ? &t[1] : nullptr, head_dim, dtype,
                                   static_cast<const int32_t*>(pos), n_tokens,
                                   static_cast<cudaStream_t>(stream)),
                  "moe_rope_apply");
}

size_t moe_kv_workspace_bytes(const moe_kv_config_t* cfg) {
  return check_kv_config(cfg) ? 0 : kv_layout(cfg).total;
}

const char* moe_kv_last_error(const moe_kv_t* h) { return h ? h->msg : moe_last_error(nullptr); }

moe_status_t moe_kv_create(const moe_kv_config_t* cfg, const moe_kv_store_t* store,
                           moe_kv_t** out) {
  if (!out) {
    fail(nullptr, "out is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  *out = nullptr;
  if (const char* m = check_kv_config(cfg)) {
    fail(nullptr, "%s", m);
    return MOE_ERR_UNSUPPORTED;
  }
  if (!store) {
    fail(nullptr, "store is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  const size_t blocks = static_cast<size_t>(cfg->n_pages) * cfg->n_kv_heads;
  const size_t codes = blocks * cfg->page_size * cfg->head_dim;
  const struct {
    const char* name;
    const void* p;
    size_t bytes;
  } arrays[4] = {{"k", store->k, codes},
                 {"v", store->v, codes},
                 {"k_scale", store->k_scale, blocks * 4},
                 {"v_scale", store->v_scale, blocks * 4}};
  for (const auto& x : arrays)
    if (!x.p || !aligned16(x.p)) {
      fail(nullptr, "store array %s must be a non-NULL 16-byte aligned pointer", x.name);
      return MOE_ERR_INVALID_ARG;
    }
  moe_kv_t* h = new (std::nothrow) moe_kv();
  if (!h) {
    fail(nullptr, "host allocation failed");
    return MOE_ERR_OOM;
  }
  h->cfg = *cfg;
  h->st = *store;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&h->n_sm, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) {
    fail(nullptr, "no usable CUDA device: %s", cudaGetErrorString(e));
    delete h;
    return MOE_ERR_CUDA;
  }
  const KvLayout L = kv_layout(cfg);
  e = cudaMalloc(&h->base, L.total);
  if (e != cudaSuccess) {
    fail(nullptr, "workspace allocation of %zu bytes failed: %s", L.total, cudaGetErrorString(e));
    cudaGetLastError();
    delete h;
    return MOE_ERR_OOM;
  }
  for (const auto& x : arrays)
    if (const char* m = moe::device_extent_error(x.p, x.bytes, h->device)) {
      fail(nullptr, "store array %s %s", x.name, m);
      cudaFree(h->base);
      delete h;
      return MOE_ERR_INVALID_ARG;
    }
  char* base = static_cast<char*>(h->base);
  h->ws = moe::AttnWs{reinterpret_cast<float*>(base + L.o), reinterpret_cast<float2*>(base + L.ml),
                      reinterpret_cast<unsigned*>(base + L.count), L.rows};
  h->count_bytes = L.err - L.count;
  h->err = reinterpret_cast<int*>(base + L.err);
  e = cudaMemset(base + L.count, 0, L.total - L.count);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    fail(nullptr, "workspace initialisation failed: %s", cudaGetErrorString(e));
    cudaFree(h->base);
    delete h;
    return MOE_ERR_CUDA;
  }
  if (!moe::kv_create_maps(h->cfg, h->st, &h->maps)) {
    fail(nullptr, "the TMA maps of the store could not be made");
    cudaFree(h->base);
    delete h;
    return MOE_ERR_CUDA;
  }
  *out = h;
  return MOE_OK;
}

void moe_kv_destroy(moe_kv_t* h) {
  if (!h) return;
  const OnDevice on(h->device);
  cudaDeviceSynchronize();
  cudaFree(h->base);
  delete h;
}

moe_status_t moe_kv_write(moe_kv_t* h, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, moe_dtype_t dtype, const moe_kv_batch_t* batch,
                          void* stream) {
  if (!h) {
    fail(nullptr, "the cache handle is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  if (const char* m = check_dtype(dtype)) {
    fail(h, "%s", m);
    return MOE_ERR_INVALID_ARG;
  }
  moe::KvView c{};
  moe_status_t st = view(h, batch, &c);
  if (st != MOE_OK || c.n_seqs == 0) return st;
  const size_t esz = dtype == MOE_BF16 ? 2 : 4;
  const int64_t row = static_cast<int64_t>(h->cfg.n_kv_heads) * h->cfg.head_dim;
  if ((st = check_stride(h, "k_stride", k_stride, row, esz)) != MOE_OK) return st;
  if ((st = check_stride(h, "v_stride", v_stride, row, esz)) != MOE_OK) return st;
  if ((st = tensor(h, &h->device, "k", &k)) != MOE_OK) return st;
  if ((st = tensor(h, &h->device, "v", &v)) != MOE_OK) return st;
  const OnDevice on(h->device);
  if (on.error != cudaSuccess) return launched(h, on.error, "moe_kv_write");
  return launched(h, moe::kv_write_launch(c, k, k_stride, v, v_stride, dtype,
                                          static_cast<cudaStream_t>(stream)),
                  "moe_kv_write");
}

moe_status_t moe_kv_read(moe_kv_t* h, void* k_out, void* v_out, moe_dtype_t dtype,
                         const moe_kv_batch_t* batch, void* stream) {
  if (!h) {
    fail(nullptr, "the cache handle is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  if (const char* m = check_dtype(dtype)) {
    fail(h, "%s", m);
    return MOE_ERR_INVALID_ARG;
  }
  moe::KvView c{};
  moe_status_t st = view(h, batch, &c);
  if (st != MOE_OK || c.n_seqs == 0 || (!k_out && !v_out)) return st;
  const void* p[2] = {k_out, v_out};
  if (p[0] && (st = tensor(h, &h->device, "k_out", &p[0])) != MOE_OK) return st;
  if (p[1] && (st = tensor(h, &h->device, "v_out", &p[1])) != MOE_OK) return st;
  const OnDevice on(h->device);
  if (on.error != cudaSuccess) return launched(h, on.error, "moe_kv_read");
  return launched(h, moe::kv_read_launch(c, const_cast<void*>(p[0]), const_cast<void*>(p[1]), dtype,
                                         static_cast<cudaStream_t>(stream)),
                  "moe_kv_read");
}

moe_status_t moe_kv_attend(moe_kv_t* h, const void* q, int64_t q_stride, void* out, float* lse,
                           const moe_kv_mask_t* mask, const moe_kv_batch_t* batch, void* stream) {
  if (!h) {
    fail(nullptr, "the cache handle is NULL");
    return MOE_ERR_INVALID_ARG;
  }
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
  moe::KvView c{};
  moe_status_t st = view(h, batch, &c);
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
  moe::AttnArgs a{};
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
  // Rows of a kv head, up to 32: keys as the products' M dimension; more: rows as
  // M.  At 32 rows the first kernel takes 90 us and the second 101 us (16 x 16384
  // keys, 4 kv heads), at 16 rows 103 and 175 us (8 kv heads), at 8 rows 208 and
  // 350 us (64 sequences).  33 rows would be two passes of the first over keys
  // that the second reads once.
  const bool tiles = static_cast<int64_t>(c.max_q) * a.G > 32;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const OnDevice on(h->device);
  if (on.error != cudaSuccess) return launched(h, on.error, "moe_kv_attend");
  return launched(h, tiles ? moe::attn_tiles_launch(c, a, h->ws, h->maps, h->n_sm, s)
                           : moe::attn_few_launch(c, a, h->ws, h->maps, h->n_sm, s),
                  "moe_kv_attend");
}

moe_status_t moe_kv_device_status(moe_kv_t* h, int32_t* flags) {
  if (!h || !flags) {
    fail(h, "the cache handle or flags is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  int32_t v = 0;
  const OnDevice on(h->device);
  cudaError_t e = on.error;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&v, h->err, 4, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && v) {
    e = cudaMemset(h->err, 0, 4);
    // a call that gave up may leave arrival counters out of step
    if (e == cudaSuccess && (v & 1)) e = cudaMemset(h->ws.count, 0, h->count_bytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) return launched(h, e, "moe_kv_device_status");
  *flags = v;
  if (!v) return MOE_OK;
  fail(h, "device error word %d:%s%s%s", v, v & 1 ? " a bounded wait gave up;" : "",
       v & 2 ? " a batch broke its bounds;" : "", v & 4 ? " NaN or infinity was written, or a scale met that is negative or not finite;" : "");
  return MOE_ERR_CUDA;
}

}  // extern "C"
