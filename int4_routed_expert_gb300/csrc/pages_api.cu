// C ABI of the page pool (include/moe_pages.h) and of copying pages: argument checks,
// workspace.
#include <algorithm>
#include <new>

#include "attn_host.cuh"
#include "pages_internal.cuh"

struct moe_pages : moe::HandleBase {
  moe_pages_config_t cfg;
  moe::PagesView v;
  int n_sm;
  void* base;  // workspace
};

namespace {

using namespace moe;

const char* check_config(const moe_pages_config_t* c) {
  if (!c) return "cfg is NULL";
  if (c->n_pages < 1 || c->n_pages > (1 << 27)) return "n_pages must be in [1, 2^27]";
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return "page_size must be 16, 32, 64 or 128";
  if (c->n_slots < 1 || c->n_slots > 65535) return "n_slots must be in [1, 65535]";
  if (c->table_stride < 1 || c->table_stride > (1 << 24)) return "table_stride must be in [1, 2^24]";
  if (static_cast<int64_t>(c->n_slots) * c->table_stride > (1 << 28)) return "n_slots * table_stride must be at most 2^28";
  return nullptr;
}

struct Layout {
  size_t slot, place, rows, ids, writers, first, err, total;
};
Layout layout(const moe_pages_config_t* c) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t n = c->n_slots, p = c->n_pages;
  Layout L;
  L.slot = 0;
  L.place = L.slot + up(n * 16);
  L.rows = L.place + up(n * 16);
  L.ids = L.rows + up(n * c->table_stride * 4);
  L.writers = L.ids + up(p * 4);
  L.first = L.writers + up(p * 4);
  L.err = L.first + up(p * 4);
  L.total = L.err + 256;
  return L;
}

}  // namespace

extern "C" {

size_t moe_pages_workspace_bytes(const moe_pages_config_t* cfg) { return check_config(cfg) ? 0 : layout(cfg).total; }

const char* moe_pages_last_error(const moe_pages_t* h) { return h ? h->msg : moe_last_error(nullptr); }

moe_status_t moe_pages_create(const moe_pages_config_t* cfg, const moe_pages_store_t* store, moe_pages_t** out) {
  if (!out) {
    fail(nullptr, "out is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  *out = nullptr;
  if (const char* m = check_config(cfg)) {
    fail(nullptr, "%s", m);
    return MOE_ERR_UNSUPPORTED;
  }
  if (!store) {
    fail(nullptr, "store is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  const size_t n = cfg->n_slots, p = cfg->n_pages;
  const struct {
    const char* name;
    const void* p;
    size_t bytes;
  } arrays[5] = {{"table", store->table, n * cfg->table_stride * 4},
                 {"kv_len", store->kv_len, n * 4},
                 {"ref", store->ref, p * 4},
                 {"cu_q", store->cu_q, (n + 1) * 4},
                 {"free_pages", store->free_pages, 4}};
  for (const auto& x : arrays)
    if (!x.p || !aligned16(x.p)) {
      fail(nullptr, "store array %s must be a non-NULL 16-byte aligned pointer", x.name);
      return MOE_ERR_INVALID_ARG;
    }
  moe_pages_t* h = new (std::nothrow) moe_pages();
  if (!h) {
    fail(nullptr, "host allocation failed");
    return MOE_ERR_OOM;
  }
  h->cfg = *cfg;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->n_sm, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) {
    fail(nullptr, "no usable CUDA device: %s", cudaGetErrorString(e));
    delete h;
    return MOE_ERR_CUDA;
  }
  const Layout L = layout(cfg);
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
  int log2 = 0;
  while ((1 << log2) < cfg->page_size) ++log2;
  h->v = PagesView{store->table, store->kv_len, store->ref, store->cu_q, store->free_pages, cfg->n_pages, cfg->n_slots,
                   cfg->table_stride, cfg->page_size, log2, reinterpret_cast<int*>(base + L.err),
                   reinterpret_cast<int*>(base + L.err + 128),
                   reinterpret_cast<int4*>(base + L.slot), reinterpret_cast<int4*>(base + L.place),
                   reinterpret_cast<int32_t*>(base + L.rows), reinterpret_cast<int32_t*>(base + L.ids),
                   reinterpret_cast<int32_t*>(base + L.writers), reinterpret_cast<int32_t*>(base + L.first)};
  e = cudaMemset(base + L.writers, 0, L.first - L.writers);
  if (e == cudaSuccess) e = cudaMemset(base + L.err, 0, L.total - L.err);
  static_assert(kNoSlot == 0x7f7f7f7f, "the byte below, four times");
  if (e == cudaSuccess) e = cudaMemset(base + L.first, 0x7f, L.err - L.first);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    fail(nullptr, "workspace initialisation failed: %s", cudaGetErrorString(e));
    cudaFree(h->base);
    delete h;
    return MOE_ERR_CUDA;
  }
  *out = h;
  return MOE_OK;
}

void moe_pages_destroy(moe_pages_t* h) {
  if (!h) return;
  const OnDevice on(h->device);
  cudaDeviceSynchronize();
  cudaFree(h->base);
  delete h;
}

moe_status_t moe_pages_fork(moe_pages_t* h, const int32_t* parent, const int32_t* added, const int32_t* keep,
                            moe_page_move_t* moves, void* stream) {
  if (!h) {
    fail(nullptr, "the pool's handle is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  const void *pa = parent, *ad = added, *ke = keep, *mo = moves;
  moe_status_t st;
  if ((st = tensor(h, &h->device, "parent", &pa)) != MOE_OK) return st;
  if ((st = tensor(h, &h->device, "added", &ad)) != MOE_OK) return st;
  if (keep && (st = tensor(h, &h->device, "keep", &ke)) != MOE_OK) return st;
  if ((st = tensor(h, &h->device, "moves", &mo)) != MOE_OK) return st;
  const OnDevice on(h->device);
  if (on.error != cudaSuccess) return launched(h, on.error, "moe_pages_fork");
  return launched(h,
                  pages_fork_launch(h->v, static_cast<const int32_t*>(pa), static_cast<const int32_t*>(ad),
                                    static_cast<const int32_t*>(ke),
                                    static_cast<moe_page_move_t*>(const_cast<void*>(mo)), h->n_sm,
                                    static_cast<cudaStream_t>(stream)),
                  "moe_pages_fork");
}

moe_status_t moe_pages_compact(moe_pages_t* h, moe_page_move_t* moves, void* stream) {
  if (!h) {
    fail(nullptr, "the pool's handle is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  const void* mo = moves;
  if (h->cfg.n_pages > 1)  // (a pool of one page has no moves)
    if (const moe_status_t st = tensor(h, &h->device, "moves", &mo); st != MOE_OK) return st;
  const OnDevice on(h->device);
  if (on.error != cudaSuccess) return launched(h, on.error, "moe_pages_compact");
  return launched(h,
                  pages_compact_launch(h->v, static_cast<moe_page_move_t*>(const_cast<void*>(mo)), h->n_sm,
                                       static_cast<cudaStream_t>(stream)),
                  "moe_pages_compact");
}

moe_status_t moe_pages_device_status(moe_pages_t* h, int32_t* flags) {
  if (!h || !flags) {
    fail(h, "the pool's handle or flags is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  int32_t v = 0;
  const OnDevice on(h->device);
  cudaError_t e = on.error;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&v, h->v.err, 4, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && v) {
    e = cudaMemset(h->v.err, 0, 4);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) return launched(h, e, "moe_pages_device_status");
  *flags = v;
  if (!v) return MOE_OK;
  fail(h, "device error word %d:%s%s", v, v & kErrBadBatch ? " a call's arrays broke their bounds;" : "",
       v & kErrNoPages ? " the pool had too few free pages" : "");
  return MOE_ERR_CUDA;
}

moe_status_t moe_kv_copy(moe_kv_t* h, const moe_page_move_t* moves, int n_moves, void* stream) {
  if (!h) {
    fail(nullptr, "the cache handle is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  if (n_moves < 0) {
    fail(h, "n_moves must not be negative");
    return MOE_ERR_INVALID_ARG;
  }
  if (n_moves == 0) return MOE_OK;
  const void* mo = moves;
  if (const moe_status_t st = tensor(h, &h->device, "moves", &mo); st != MOE_OK) return st;
  const moe_kv_config_t& c = h->cfg;
  KvView v{};
  v.k = h->st.k, v.v = h->st.v, v.k_scale = h->st.k_scale, v.v_scale = h->st.v_scale;
  v.n_pages = c.n_pages, v.hkv = c.n_kv_heads, v.D = c.head_dim, v.page = c.page_size;
  v.err = h->err;
  const OnDevice on(h->device);
  if (on.error != cudaSuccess) return launched(h, on.error, "moe_kv_copy");
  return launched(h, kv_copy_launch(v, static_cast<const moe_page_move_t*>(mo), n_moves, h->n_sm,
                                    static_cast<cudaStream_t>(stream)),
                  "moe_kv_copy");
}

}  // extern "C"
