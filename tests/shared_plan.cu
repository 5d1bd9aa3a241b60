// The plans of attention over shared prefixes for host-side tests: attn_shared.cu's own functions, without a launch.
#include "../int4_routed_expert_gb300/csrc/attn_shared.cu"

namespace moe {

cudaError_t attn_few_both_launch(const KvView&, const AttnArgs&, const AttnWs&, const Share&, const KvMaps&, int, cudaStream_t) {
  return cudaErrorNotSupported;
}
cudaError_t attn_tiles_both_launch(const KvView&, const AttnArgs&, const AttnWs&, const Share&, const KvMaps&, int, cudaStream_t) {
  return cudaErrorNotSupported;
}
cudaError_t attn_few_part_launch(const KvView&, const AttnArgs&, const AttnWs&, const Plan&, const Share&, bool, const KvMaps&,
                                 cudaStream_t) {
  return cudaErrorNotSupported;
}
cudaError_t attn_tiles_part_launch(const KvView&, const AttnArgs&, const AttnWs&, const Plan&, const Share&, bool, int,
                                   const KvMaps&, cudaStream_t) {
  return cudaErrorNotSupported;
}

}  // namespace moe

// sizes: sequences, tokens, max_q_len, max_kv_len, kv heads, head_dim, query heads of each, groups, max_group_tokens,
// max_prefix_len; plan: one launch, CTAs of dealt out work, row tiles, splits and parts of the prefixes, splits of own keys
extern "C" unsigned long long shared_plan(const int* sizes, int n_sm, int* plan) {
  moe::KvView c{};
  c.n_seqs = sizes[0], c.n_tokens = sizes[1], c.max_q = sizes[2], c.max_kv = sizes[3], c.hkv = sizes[4], c.D = sizes[5];
  moe::Share sh{};
  sh.n_groups = sizes[7], sh.max_tokens = sizes[8], sh.max_len = sizes[9], sh.n_seqs = c.n_seqs;
  const moe::Sides s = moe::sides_of(c, sh, sizes[6], n_sm);
  plan[0] = s.one, plan[1] = s.shared.ctas, plan[2] = s.shared.pl.row_tiles, plan[3] = s.shared.pl.splits;
  plan[4] = s.shared.parts, plan[5] = s.own.pl.splits;
  return moe::attn_shared_workspace(c, sh, sizes[6], n_sm);
}
