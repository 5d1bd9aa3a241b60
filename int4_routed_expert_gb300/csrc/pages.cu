// The page pool: the next step's sequences out of the last one's (moe_pages_fork),
// pages in use moved to the front (moe_pages_compact).
//
// Fork.  Slot i keeps the first k_i = min(keep_i, len[parent_i]) tokens of its parent,
// in ceil(k_i / S) pages, and gets pages up to ceil((k_i + added_i) / S).  Uses of a
// page change by +1 for every row that keeps it and -1 for every row that had it;
// rows that go on (parent_i = i) change what they drop alone.  A slot writes into
// the page of its last kept token where k_i is no multiple of S and added_i > 0; it
// copies the page when others use it: ref > 1, and the slot is not the lowest of ref
// writers.  New pages: the d-th page needed, in order of the slots, is the d-th free
// one, by two prefix sums.
//
// Integer work on a few hundred KB, of which each step needs the one before whole: bound
// by latency, so it is one cluster of CTAs whose steps are hardware barriers of the cluster
// apart, and the totals that a step hands on go through distributed shared memory.
//
// Compact.  With u pages in use, those from u on move, in their order, into the free ones
// below u; a page's rank among its kind is the same prefix sum over the pool.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "pages_internal.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostCtas = 8;  // of a cluster

// A value of each CTA, handed to all of the cluster: put, the cluster's barrier, then take.
template <typename T>
struct Box {
  T v[kMostCtas];
  __device__ __forceinline__ void put(cg::cluster_group& cl, const T& x) {
    for (unsigned r = 0; r < cl.num_blocks(); ++r) cl.map_shared_rank(this, r)->v[cl.block_rank()] = x;
  }
  __device__ __forceinline__ T before(unsigned rank) const {
    T s{};
    for (unsigned r = 0; r < rank; ++r) s += v[r];
    return s;
  }
};

// All stores of the CTAs before are seen by __ldcg behind it.
__device__ __forceinline__ void cluster_sync(cg::cluster_group& cl) {
  __threadfence();
  cl.sync();
}

// Sum over the lower threads of the CTA and over all of them.
__device__ __forceinline__ uint64_t scan_cta(uint64_t x, uint64_t (&part)[kWarps], uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) part[warp] = s;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  __syncthreads();
  return before + s - x;
}

// The pool in segments of whole 32s, a warp of the cluster each, in their order.
struct Segment {
  int begin, end;
  __device__ __forceinline__ Segment(int n, int warp, int warps) {
    const int64_t each = (static_cast<int64_t>(n) + 32 * warps - 1) / (32 * warps) * 32;
    begin = static_cast<int>(min(each * warp, static_cast<int64_t>(n)));
    end = static_cast<int>(min(each * (warp + 1), static_cast<int64_t>(n)));
  }
  // Pages with ref == 0 among [begin, stop).
  __device__ __forceinline__ int count_free(const int32_t* ref, int stop) const {
    constexpr int kBatch = 8;
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int a = begin; a < stop; a += 32 * kBatch) {
      int x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) x[k] = a + 32 * k + lane < stop ? __ldcg(ref + a + 32 * k + lane) : 1;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) n += x[k] == 0;
    }
    return __reduce_add_sync(0xffffffffu, n);
  }
};

// Threads of a row: as many as the cluster has, at least a warp, at most a CTA.
__device__ __forceinline__ int threads_of_row(int all, int rows) {
  int t = 32;
  while (t < kThreads && 2 * t <= all / max(rows, 1)) t *= 2;
  return t;
}

// Calls f(j, value) for j = lane, lane + step, ... below n, with several loads under way.
template <typename F>
__device__ __forceinline__ void each_entry(const int32_t* row, int begin, int n, int lane, int step, F f) {
  constexpr int kBatch = 4;
  for (int j = begin + lane; j < n; j += kBatch * step) {
    int x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) x[k] = j + k * step < n ? __ldcg(row + j + k * step) : -1;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (j + k * step < n) f(j + k * step, x[k]);
  }
}

__device__ __forceinline__ void no_moves(moe_page_move_t* moves, int begin, int end, int tid, int all) {
  int32_t* m = reinterpret_cast<int32_t*>(moves);
  for (int64_t j = 3LL * begin + tid; j < 3LL * end; j += all) m[j] = -1;
}

__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(const PagesView p, const int32_t* parent, const int32_t* added, const int32_t* keep,
                moe_page_move_t* moves) {
  __shared__ Box<int> s_bad, s_free;
  __shared__ Box<int> s_bad_page;
  __shared__ Box<uint64_t> s_need, s_added;
  __shared__ uint64_t part[kWarps];
  __shared__ int warp_free[kWarps];
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();  // (that the others run: before their shared memory is written to)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned rank = cl.block_rank(), ctas = cl.num_blocks();
  const int all = static_cast<int>(ctas) * kThreads, tid = static_cast<int>(rank) * kThreads + threadIdx.x;
  const int64_t most = static_cast<int64_t>(p.stride) << p.page_log2;  // tokens of a row
  auto pages = [&](int tokens) { return static_cast<int>((static_cast<int64_t>(tokens) + p.page - 1) >> p.page_log2); };
  auto in_pool = [&](int x) { return static_cast<unsigned>(x) < static_cast<unsigned>(p.n_pages); };
  auto row_of = [&](int i) { return p.table + static_cast<size_t>(i) * p.stride; };

  // what each slot keeps
  int bad = 0;
  for (int i = tid; i < p.n_slots; i += all) {
    const int pa = __ldg(parent + i), ad = __ldg(added + i), kp = keep ? __ldg(keep + i) : INT_MAX;
    const int len = __ldcg(p.kv_len + i);
    bool ok = pa >= -1 && pa < p.n_slots && ad >= 0 && len >= 0 && len <= most;
    const int has = ok && pa >= 0 ? __ldcg(p.kv_len + pa) : 0;
    const int k = max(min(kp, has), 0);
    ok = ok && has >= 0 && has <= most && static_cast<int64_t>(k) + ad <= min(most, static_cast<int64_t>(INT_MAX));
    bad |= !ok;
    p.slot[i] = ok ? make_int4(pa, k, pages(len), ad) : make_int4(-1, 0, 0, 0);
  }
  bad = __syncthreads_or(bad);
  cl.barrier_wait();
  if (threadIdx.x == 0) s_bad.put(cl, bad);
  cluster_sync(cl);
  const bool refused = s_bad.before(ctas) != 0;

  // the pages' uses, and the slots that write into pages that are not full
  const int T = threads_of_row(all, p.n_slots);
  const int row0 = tid / T, row_lane = tid % T, rows_at_once = all / T;
  auto change_uses = [&](int sign, bool note) {
    int wrong = 0;
    for (int i = row0; i < p.n_slots; i += rows_at_once) {
      const int4 s = __ldcg(p.slot + i);
      const int kept = pages(s.y);
      if (s.x != i && s.x >= 0)
        each_entry(row_of(s.x), 0, kept, row_lane, T, [&](int j, int x) {
          if (in_pool(x)) {
            if (note) p.rows[static_cast<size_t>(i) * p.stride + j] = x;
            atomicAdd(p.ref + x, sign);
          } else {
            wrong = 1;
          }
        });
      each_entry(row_of(i), s.x == i ? kept : 0, s.z, row_lane, T, [&](int, int x) {
        if (in_pool(x)) atomicSub(p.ref + x, sign);
      });
      if (note && row_lane == 0 && s.w > 0 && (s.y & (p.page - 1)) != 0) {
        const int x = __ldcg(row_of(s.x) + kept - 1);
        if (in_pool(x)) {
          atomicAdd(p.writers + x, 1);
          atomicMin(p.first + x, i);
        } else {
          wrong = 1;
        }
      }
    }
    return wrong;
  };
  int wrong = refused ? 1 : change_uses(1, true);
  wrong = __syncthreads_or(wrong);
  if (threadIdx.x == 0) s_bad_page.put(cl, wrong);
  cluster_sync(cl);
  const bool bad_page = s_bad_page.before(ctas) != 0;

  // what each slot needs (a thread has neighbouring slots), and what is free
  const int per = (p.n_slots + all - 1) / all;
  const int i0 = min(tid * per, p.n_slots), i1 = min(i0 + per, p.n_slots);
  constexpr int kShift = 20;  // pages in the upper bits, copies in the lower
  uint64_t need = 0, sum = 0;
  for (int i = i0; !bad_page && i < i1; ++i) {
    const int4 s = __ldcg(p.slot + i);
    const int kept = pages(s.y);
    int copy = -1, x = -1;
    if (s.w > 0 && (s.y & (p.page - 1)) != 0) {
      x = __ldcg(row_of(s.x) + kept - 1);
      const int uses = __ldcg(p.ref + x), n = __ldcg(p.writers + x), lowest = __ldcg(p.first + x);
      if (uses > 1 && !(n == uses && lowest == i)) copy = x;
    }
    p.place[i] = make_int4(0, 0, copy, x);  // (this thread's own until it is whole)
    need += (static_cast<uint64_t>(pages(s.y + s.w) - kept + (copy >= 0)) << kShift) + (copy >= 0);
    sum += s.w;
  }
  uint64_t all_need, all_added;
  const uint64_t need0 = scan_cta(need, part, all_need), added0 = scan_cta(sum, part, all_added);
  const Segment seg(p.n_pages, static_cast<int>(rank) * kWarps + warp, static_cast<int>(ctas) * kWarps);
  const int mine = bad_page ? 0 : seg.count_free(p.ref, seg.end);
  if (lane == 0) warp_free[warp] = mine;
  __syncthreads();
  int free_before = 0, free_cta = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) free_before += warp_free[w];
    free_cta += warp_free[w];
  }
  if (threadIdx.x == 0) {
    s_need.put(cl, all_need);
    s_added.put(cl, all_added);
    s_free.put(cl, free_cta);
  }
  cluster_sync(cl);
  const uint64_t total = s_need.before(ctas);
  const int wanted = static_cast<int>(total >> kShift), copies = static_cast<int>(total & ((1 << kShift) - 1));
  const int n_free = s_free.before(ctas);
  const bool too_long = s_added.before(ctas) > INT_MAX;

  if (bad_page || too_long || wanted > n_free) {
    // nothing happens
    if (!refused) change_uses(-1, false);
    no_moves(moves, 0, p.n_slots, tid, all);
    for (int i = tid; i <= p.n_slots; i += all) p.cu_q[i] = 0;
    if (!refused)
      for (int i = tid; i < p.n_slots; i += all) {
        const int4 s = __ldcg(p.slot + i);
        if (s.w == 0 || (s.y & (p.page - 1)) == 0) continue;
        const int x = __ldcg(row_of(s.x) + pages(s.y) - 1);
        if (in_pool(x)) p.writers[x] = 0, p.first[x] = kNoSlot;
      }
    if (tid == 0) atomicOr(p.err, bad_page || too_long ? kErrBadBatch : kErrNoPages);
    return;
  }

  // the free pages that are needed, and where each slot's ones stand among them
  free_before += s_free.before(rank);
  if (free_before < wanted)
    for (int a = seg.begin, at = free_before; a < seg.end && at < wanted; a += 32) {
      const bool is_free = a + lane < seg.end && __ldcg(p.ref + a + lane) == 0;
      const uint32_t m = __ballot_sync(0xffffffffu, is_free);
      const int to = at + __popc(m & ((1u << lane) - 1));
      if (is_free && to < wanted) p.ids[to] = a + lane;
      at += __popc(m);
    }
  uint64_t at = s_need.before(rank) + need0, tokens = s_added.before(rank) + added0;
  for (int i = i0; i < i1; ++i) {
    const int4 s = __ldcg(p.slot + i);
    const int copy = p.place[i].z, x = p.place[i].w;
    p.place[i] = make_int4(static_cast<int>(at >> kShift), static_cast<int>(at & ((1 << kShift) - 1)), copy, x);
    if (x >= 0) p.writers[x] = 0, p.first[x] = kNoSlot;  // (all have seen them)
    at += (static_cast<uint64_t>(pages(s.y + s.w) - pages(s.y) + (copy >= 0)) << kShift) + (copy >= 0);
    tokens += s.w;
    p.cu_q[i + 1] = static_cast<int32_t>(tokens);
  }
  if (tid == 0) {
    p.cu_q[0] = 0;
    *p.free_pages = n_free - wanted;
  }
  no_moves(moves, copies, p.n_slots, tid, all);
  cluster_sync(cl);

  for (int i = row0; i < p.n_slots; i += rows_at_once) {
    const int4 s = __ldcg(p.slot + i), pl = __ldcg(p.place + i);
    const int kept = pages(s.y), have = pages(s.y + s.w), copy = pl.z >= 0;
    const int32_t* fresh = p.ids + pl.x;
    int32_t* row = row_of(i);
    const bool moved = s.x != i;
    if (moved)
      each_entry(p.rows + static_cast<size_t>(i) * p.stride, 0, kept - copy, row_lane, T,
                 [&](int j, int x) { row[j] = x; });
    for (int j = kept - copy + row_lane; j < max(have, s.z); j += T) {
      const int x = j < have ? __ldcg(fresh + (j - kept + copy)) : -1;
      row[j] = x;
      if (x >= 0) p.ref[x] = 1;
    }
    if (row_lane == 0) {
      p.kv_len[i] = s.y + s.w;
      if (copy) {
        moves[pl.y] = moe_page_move_t{pl.z, __ldcg(fresh), s.y & (p.page - 1)};
        atomicSub(p.ref + pl.z, 1);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const PagesView p, moe_page_move_t* moves) {
  __shared__ int s_free[kMostCtas * kWarps];  // free pages of every warp's segment
  __shared__ int s_below;
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();
  const int lane = threadIdx.x & 31;
  const int ctas = static_cast<int>(cl.num_blocks()), all = ctas * kThreads, warps = ctas * kWarps;
  const int tid = static_cast<int>(cl.block_rank()) * kThreads + threadIdx.x, gw = tid >> 5;
  const Segment seg(p.n_pages, gw, warps);
  const int mine = seg.count_free(p.ref, seg.end);
  if (threadIdx.x == 0) s_below = 0;
  cl.barrier_wait();
  if (lane < ctas) cl.map_shared_rank(s_free, lane)[gw] = mine;
  cluster_sync(cl);

  // pages in use, and the free ones among the first so many: whole segments, then a part of one
  int free_before = 0, n_free = 0;
  for (int w = lane; w < warps; w += 32) {
    n_free += s_free[w];
    if (w < gw) free_before += s_free[w];
  }
  n_free = __reduce_add_sync(0xffffffffu, n_free);
  free_before = __reduce_add_sync(0xffffffffu, free_before);
  const int used = p.n_pages - n_free;
  const int each = Segment(p.n_pages, 0, warps).end, w_end = used / max(each, 1);
  int below = 0;
  if (threadIdx.x < w_end) below = s_free[threadIdx.x];
  for (int a = w_end * each + threadIdx.x; a < used; a += kThreads) below += __ldcg(p.ref + a) == 0;
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0 && below) atomicAdd(&s_below, below);
  __syncthreads();
  const int n_moves = s_below;

  // both ends of the moves, in their order
  constexpr int kBatch = 4;
  for (int a = seg.begin, at = free_before; a < seg.end; a += 32 * kBatch) {
    int x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) x[k] = a + 32 * k + lane < seg.end ? __ldcg(p.ref + a + 32 * k + lane) : 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int page = a + 32 * k + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, page < seg.end && x[k] == 0);
      const int free_below = at + __popc(m & ((1u << lane) - 1));
      if (page < seg.end) {
        const bool is_free = x[k] == 0;
        if (page < used) {
          if (is_free) moves[free_below].dst = page;
        } else {
          const int r = is_free ? -1 : page - free_below - (used - n_moves);
          p.ids[page] = r;
          if (!is_free) moves[r].src = page, moves[r].tokens = p.page;
        }
      }
      at += __popc(m);
    }
  }
  no_moves(moves, n_moves, p.n_pages / 2, tid, all);
  if (tid == 0) *p.free_pages = n_free;
  cluster_sync(cl);

  for (int r = tid; r < n_moves; r += all) {
    const int src = __ldcg(&moves[r].src), dst = __ldcg(&moves[r].dst);
    p.ref[dst] = __ldcg(p.ref + src);
    p.ref[src] = 0;
  }
  const int64_t most = static_cast<int64_t>(p.stride) << p.page_log2;
  const int T = threads_of_row(all, p.n_slots);
  bool bad = false;
  for (int i = tid / T; i < p.n_slots; i += all / T) {
    const int len = __ldcg(p.kv_len + i);
    const int n = static_cast<int>((min(max(static_cast<int64_t>(len), static_cast<int64_t>(0)), most) + p.page - 1) >> p.page_log2);
    int32_t* row = p.table + static_cast<size_t>(i) * p.stride;
    each_entry(row, 0, n, tid % T, T, [&](int j, int x) {
      if (static_cast<unsigned>(x) >= static_cast<unsigned>(p.n_pages)) {
        bad = true;
      } else if (x >= used) {
        const int r = __ldcg(p.ids + x);
        if (r >= 0)
          row[j] = __ldcg(&moves[r].dst);
        else
          bad = true;
      }
    });
  }
  if (bad) atomicOr(p.err, kErrBadBatch);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int ctas, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// One CTA while the pool and the slots give its threads a few words each: its barriers
// are the cheaper ones.
int ctas_of(const PagesView& p) {
  const int64_t words = static_cast<int64_t>(p.n_slots) * std::min(p.stride, 64) + p.n_pages;
  return words <= 8 * kThreads ? 1 : kMostCtas;
}

}  // namespace

cudaError_t pages_fork_launch(const PagesView& p, const int32_t* parent, const int32_t* added, const int32_t* keep,
                              moe_page_move_t* moves, cudaStream_t s) {
  return launch(fork_kernel, ctas_of(p), s, p, parent, added, keep, moves);
}

cudaError_t pages_compact_launch(const PagesView& p, moe_page_move_t* moves, cudaStream_t s) {
  return launch(compact_kernel, ctas_of(p), s, p, moves);
}

}  // namespace moe
