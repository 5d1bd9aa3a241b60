// C ABI of the attention-side operators (include/moe_attn.h): argument checks,
// workspace, dispatch.
#include <algorithm>
#include <new>

#include "attn_host.cuh"

namespace {

using namespace moe;

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
  static const int32_t kFirst[128] = {};
  return moe_rope_create_axes(rot_dim, inv_freq, amplitude, interleaved, 1, kFirst, out);
}

moe_status_t moe_rope_create_axes(int rot_dim, const double* inv_freq, float amplitude,
                                  int interleaved, int n_axes, const int32_t* axis,
                                  moe_rope_t** out) {
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
  if (n_axes < 1 || n_axes > 4) {
    fail(nullptr, "n_axes must be in [1, 4], got %d", n_axes);
    return MOE_ERR_UNSUPPORTED;
  }
  if (!axis) {
    fail(nullptr, "axis is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  for (int i = 0; i < rot_dim / 2; ++i)
    if (axis[i] < 0 || axis[i] >= n_axes) {
      fail(nullptr, "axis[%d] must be in [0, %d), got %d", i, n_axes, axis[i]);
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
  r->n_axes = n_axes;
  for (int i = 0; i < rot_dim / 2; ++i) {
    r->axis[i] = static_cast<uint8_t>(axis[i]);
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
  moe_rope_tensor_t t[2];
  int device;
  if (const moe_status_t st = rope_args(r, q, k, head_dim, dtype, n_tokens, t, device); st != MOE_OK) return st;
  if (r->n_axes != 1) {
    fail(nullptr, "the rope handle has %d axes: moe_rope_apply_axes", r->n_axes);
    return MOE_ERR_INVALID_ARG;
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
  KvView c{};
  AttnArgs a{};
  const moe_status_t st = attend_args(h, q, q_stride, out, lse, mask, batch, &c, &a);
  if (st != MOE_OK || c.n_seqs == 0) return st;
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
