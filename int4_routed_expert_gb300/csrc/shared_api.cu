// C ABI of attention over shared prefixes (include/moe_attn.h): argument checks,
// workspace.
#include <algorithm>

#include "attn_host.cuh"

namespace {

using namespace moe;

// NULL, or what is wrong with the bounds of a prefix.
const char* check_prefix(const moe_kv_config_t& c, const moe_kv_prefix_t* p) {
  if (!p) return "prefix is NULL";
  if (p->n_groups < 0 || p->n_groups > 65535) return "n_groups must be in [0, 65535]";
  if (p->n_groups == 0) return nullptr;
  if (p->max_group_tokens < 1) return "max_group_tokens must be at least 1";
  if (p->max_prefix_len < 1 || p->max_prefix_len > c.max_kv_len)
    return "max_prefix_len must be in [1, max_kv_len of the handle]";
  if (p->table_stride < 1) return "the prefix's table_stride must be at least 1";
  return nullptr;
}

Share share_of(const moe_kv_batch_t* b, const moe_kv_prefix_t* p) {
  return Share{p->cu_seq, p->prefix_len, p->page_table, p->table_stride, p->n_groups,
               std::min(p->max_group_tokens, b->n_tokens), p->max_prefix_len, b->n_seqs};
}

}  // namespace

extern "C" {

size_t moe_kv_shared_workspace_bytes(const moe_kv_t* h, const moe_kv_batch_t* batch, const moe_kv_prefix_t* prefix) {
  if (!h || !batch || batch->n_seqs < 1 || batch->n_tokens < 1 || batch->max_q_len < 1 || batch->max_kv_len < 0 ||
      batch->n_seqs > h->cfg.max_seqs || batch->n_tokens > h->cfg.max_tokens || batch->max_kv_len > h->cfg.max_kv_len ||
      batch->max_q_len > batch->n_tokens || check_prefix(h->cfg, prefix) || prefix->n_groups == 0)
    return 0;
  KvView c{};
  c.n_seqs = batch->n_seqs, c.n_tokens = batch->n_tokens, c.max_q = batch->max_q_len, c.max_kv = batch->max_kv_len;
  c.hkv = h->cfg.n_kv_heads, c.D = h->cfg.head_dim;
  return attn_shared_workspace(c, share_of(batch, prefix), h->cfg.n_q_heads / h->cfg.n_kv_heads, h->n_sm);
}

moe_status_t moe_kv_attend_shared(moe_kv_t* h, const void* q, int64_t q_stride, void* out, float* lse,
                                  const moe_kv_mask_t* mask, const moe_kv_batch_t* batch, const moe_kv_prefix_t* prefix,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!h) {
    fail(nullptr, "the cache handle is NULL");
    return MOE_ERR_INVALID_ARG;
  }
  if (prefix && prefix->n_groups == 0) return moe_kv_attend(h, q, q_stride, out, lse, mask, batch, stream);
  KvView c{};
  AttnArgs a{};
  moe_status_t st = attend_args(h, q, q_stride, out, lse, mask, batch, &c, &a);
  if (st != MOE_OK || c.n_seqs == 0) return st;
  if (const char* m = check_prefix(h->cfg, prefix)) {
    fail(h, "%s", m);
    return MOE_ERR_INVALID_ARG;
  }
  if (a.window) {
    fail(h, "a window of %d tokens does not see a whole prefix", mask->window);
    return MOE_ERR_UNSUPPORTED;
  }
  Share sh = share_of(batch, prefix);
  const void *p[4] = {sh.cu_seq, sh.prefix_len, sh.table, workspace};
  const char* name[4] = {"cu_seq", "prefix_len", "the prefix's page_table", "workspace"};
  for (int i = 0; i < (workspace ? 4 : 3); ++i)
    if ((st = tensor(h, &h->device, name[i], &p[i])) != MOE_OK) return st;
  sh.cu_seq = static_cast<const int32_t*>(p[0]);
  sh.prefix_len = static_cast<const int32_t*>(p[1]);
  sh.table = static_cast<const int32_t*>(p[2]);
  const OnDevice on(h->device);
  if (on.error != cudaSuccess) return launched(h, on.error, "moe_kv_attend_shared");
  size_t need = 0;
  const cudaError_t e = attn_shared_launch(c, a, sh, h->ws, const_cast<void*>(p[3]), workspace ? workspace_bytes : 0, &need,
                                           h->maps, h->n_sm, static_cast<cudaStream_t>(stream));
  if (need && !workspace) {
    fail(h, "workspace is NULL, the call needs %zu bytes", need);
    return MOE_ERR_INVALID_ARG;
  }
  if (workspace_bytes < need) {
    fail(h, "the workspace has %zu bytes, the call needs %zu", workspace_bytes, need);
    return MOE_ERR_CAPACITY;
  }
  return launched(h, e, "moe_kv_attend_shared");
}

}  // extern "C"
