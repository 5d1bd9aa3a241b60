// Copies pages of the cache (moe_kv_copy): whole ones when a pool is compacted, the
// tokens of half-filled ones when sequences are forked.
//
// A page's codes of keys, or of values, are one run of memory, of which a move takes
// the tokens below `tokens` of each head: pieces of 4 KB, a warp each, 16 bytes a lane and
// load, eight loads under way.  A move's pieces go to the warps of one CTA, or of several
// where moves are few.  Bound by memory.
#include <algorithm>

#include "pages_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 8;
constexpr int kPiece = kLoads * 32 * 16;

__global__ void __launch_bounds__(kThreads)
    kv_copy_kernel(const KvView c, const moe_page_move_t* __restrict__ moves, int n, int slices) {
  const int lane = threadIdx.x & 31;
  const int slice = blockIdx.x % slices;
  const int warp = slice * (kThreads / 32) + (threadIdx.x >> 5), warps = slices * (kThreads / 32);
  const uint32_t bytes = static_cast<uint32_t>(c.hkv * c.page) * c.D;
  const int pieces = (bytes + kPiece - 1) / kPiece;
  const int d_log2 = c.D == 128 ? 7 : 6;
  const int step = gridDim.x / slices;
  bool bad = false;
  // the CTA's next 32 moves, a lane each (in 64 bits: the round behind the last one may begin above 2^31)
  for (int64_t m0 = blockIdx.x / slices; m0 < n; m0 += 32LL * step) {
    const int64_t at = m0 + static_cast<int64_t>(lane) * step;
    int src = -1, dst = -1, tokens = 0;
    if (at < n) src = __ldg(&moves[at].src), dst = __ldg(&moves[at].dst), tokens = __ldg(&moves[at].tokens);
    bool good = src >= 0;
    if (good && (src >= c.n_pages || static_cast<unsigned>(dst) >= static_cast<unsigned>(c.n_pages) ||
                 static_cast<unsigned>(tokens) > static_cast<unsigned>(c.page)))
      good = false, bad = true;
    for (uint32_t todo = __ballot_sync(0xffffffffu, good); todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      const size_t from = __shfl_sync(0xffffffffu, src, l), to = __shfl_sync(0xffffffffu, dst, l);
      const int part = __shfl_sync(0xffffffffu, tokens, l);
      if (from == to) continue;
      for (int u = warp; u < 2 * pieces; u += warps) {
        const bool values = u >= pieces;
        const uint32_t off0 = static_cast<uint32_t>(values ? u - pieces : u) * kPiece + lane * 16;
        const uint8_t* s = (values ? c.v : c.k) + from * bytes;
        uint8_t* d = (values ? c.v : c.k) + to * bytes;
        uint4 x[kLoads];
        bool in[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint32_t off = off0 + i * 512;
          in[i] = off < bytes && static_cast<int>((off >> d_log2) & (c.page - 1)) < part;
          if (in[i]) x[i] = __ldcs(reinterpret_cast<const uint4*>(s + off));
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (in[i]) *reinterpret_cast<uint4*>(d + off0 + i * 512) = x[i];
      }
      if (slice == 0) {
        const int t = threadIdx.x;
        if (t < c.hkv) c.k_scale[to * c.hkv + t] = __ldg(c.k_scale + from * c.hkv + t);
        if (t < c.hkv) c.v_scale[to * c.hkv + t] = __ldg(c.v_scale + from * c.hkv + t);
      }
    }
  }
  if (bad && threadIdx.x < 32) atomicOr(c.err, kErrBadBatch);
}

}  // namespace

cudaError_t kv_copy_launch(const KvView& c, const moe_page_move_t* moves, int n, int n_sm, cudaStream_t s) {
  const int64_t bytes = static_cast<int64_t>(c.hkv) * c.page * c.D;
  const int64_t pieces = 2 * ((bytes + kPiece - 1) / kPiece);
  const int64_t room = static_cast<int64_t>(n_sm) * 8;  // CTAs that run together
  const int64_t most = (pieces + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t slices = std::max<int64_t>(1, std::min(most, room / n));
  const int64_t grid = std::min<int64_t>(n, std::max<int64_t>(1, room / slices)) * slices;
  kv_copy_kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(c, moves, n, static_cast<int>(slices));
  return cudaGetLastError();
}

}  // namespace moe
