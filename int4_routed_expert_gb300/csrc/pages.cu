// The page pool: the next step's sequences out of the last one's (moe_pages_fork),
// pages in use moved to the front (moe_pages_compact).
//
// Fork.  Slot i keeps the first k_i = min(keep_i, len[parent_i]) tokens of its parent,
// in ceil(k_i / S) pages, and gets pages up to ceil((k_i + added_i) / S).  Uses of a
// page change by +1 for every row that keeps it and -1 for every row that had it;
// rows that go on (parent_i = i) change what they drop alone, and what they keep is looked at
// (777 slots: 0.5 us of the call's 14.0).  A slot writes into
// the page of its last kept token where k_i is no multiple of S and added_i > 0; it
// copies the page when others use it: ref > 1, and the slot is not the lowest of ref
// writers.  New pages: the d-th page needed, in order of the slots, is the d-th free
// one, by two prefix sums.
//
// Integer work on a few hundred KB to a few MB, of which each step needs the one before
// whole: bound by latency.  A small pool is one CTA's work.  In a large one the uses and
// the rows are changed by the whole device, in launches before and behind a cluster of CTAs
// that adds up what is needed and what is free, its totals by way of distributed shared
// memory.
// Figures (calls in a replayed graph): 16 slots of up to 1500 tokens 7.9 us; 777 slots of
// up to 40000 tokens in a pool of 460,000 pages, a tenth of them forked, 14.0 us (one
// cluster for all three steps: 35 us); 344,000 pages compacted 11.5 us (all in the cluster:
// 28 us).
//
// Compact.  With u pages in use, those from u on move, in their order, into the free ones
// below u; a page's rank among its kind is the same prefix sum over the pool, kept as words of
// 32 pages and the free ones before them.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "pages_internal.cuh"
#include "smem_opt_in.cuh"
#include "stream_common.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostCtas = 16;  // of a cluster
constexpr int kGridThreads = 256;

// What the slots and the pool's segments add up to.
struct Sums {
  uint64_t need, added;  // pages (upper bits) and copies that slots need, their new tokens
  int free;
  __device__ __forceinline__ Sums& operator+=(const Sums& x) {
    need += x.need, added += x.added, free += x.free;
    return *this;
  }
};
constexpr int kShift = 20;  // of pages in `need`

// Sums over the lower threads of the CTA (free: over the lower warps) and over all of it;
// x.free is a warp's.
__device__ __forceinline__ Sums scan_cta(const Sums& x, Sums (&part)[kWarps + 1], Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](Sums s) {  // of the warp's lanes, inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y{__shfl_up_sync(0xffffffffu, s.need, o), __shfl_up_sync(0xffffffffu, s.added, o),
                   __shfl_up_sync(0xffffffffu, s.free, o)};
      if (lane >= o) s += y;
    }
    return s;
  };
  const Sums s = scan(Sums{x.need, x.added, 0});
  if (lane == 31) part[warp] = Sums{s.need, s.added, x.free};
  __syncthreads();
  if (warp == 0) {
    const Sums mine = part[lane], up = scan(mine);
    if (lane == 31) part[kWarps] = up;
    part[lane] = Sums{up.need - mine.need, up.added - mine.added, up.free - mine.free};
  }
  __syncthreads();
  total = part[kWarps];
  const Sums before = part[warp];
  return Sums{before.need + s.need - x.need, before.added + s.added - x.added, before.free};
}

// The pool in segments of whole 128s, a warp of the cluster each, in their order: a lane
// has four neighbouring pages of each 128.
struct Segment {
  int begin, end;
  __device__ __forceinline__ Segment(int n, int warp, int warps) {
    const int64_t each = size(n, warps);
    begin = static_cast<int>(min(each * warp, static_cast<int64_t>(n)));
    end = static_cast<int>(min(each * (warp + 1), static_cast<int64_t>(n)));
  }
  static __device__ __forceinline__ int64_t size(int n, int warps) {
    return (static_cast<int64_t>(n) + 128 * warps - 1) / (128 * warps) * 128;
  }
  // The uses of pages a + 4 lane .. + 3; `none` behind the segment.
  __device__ __forceinline__ int4 load(const int32_t* ref, int a, int none) const {
    const int x = a + 4 * (threadIdx.x & 31);
    if (x + 4 <= end) return __ldcg(reinterpret_cast<const int4*>(ref + x));
    return make_int4(x < end ? __ldcg(ref + x) : none, x + 1 < end ? __ldcg(ref + x + 1) : none,
                     x + 2 < end ? __ldcg(ref + x + 2) : none, none);
  }
  __device__ __forceinline__ int count_free(const int32_t* ref) const {
    constexpr int kBatch = 4;
    int n = 0;
    for (int a = begin; a < end; a += 128 * kBatch) {
      int4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) x[k] = load(ref, a + 128 * k, 1);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) n += (x[k].x == 0) + (x[k].y == 0) + (x[k].z == 0) + (x[k].w == 0);
    }
    return __reduce_add_sync(0xffffffffu, n);
  }
};

// The same in words of free pages, 1024 pages at once: bits 4 g .. 4 g + 3 of a lane's are pages
// 128 g + 4 lane ... Up to as many a segment (half a million in the pool) stay in registers
// between the count and the list (344,000 pages compacted: 11.5 us, read again 13.3 us).
struct FreeWords : Segment {
  uint32_t kept;
  __device__ __forceinline__ FreeWords(int n, int warp, int warps) : Segment(n, warp, warps), kept(0) {}
  __device__ __forceinline__ uint32_t look(const int32_t* ref, int a) const {
    constexpr int kBatch = 4;
    uint32_t bits = 0;
#pragma unroll
    for (int g0 = 0; g0 < 8; g0 += kBatch) {
      if (a + 128 * g0 >= end) break;
      int4 x[kBatch];
#pragma unroll
      for (int g = 0; g < kBatch; ++g) x[g] = load(ref, a + 128 * (g0 + g), 1);
#pragma unroll
      for (int g = 0; g < kBatch; ++g)
        bits |= ((x[g].x == 0) + 2u * (x[g].y == 0) + 4u * (x[g].z == 0) + 8u * (x[g].w == 0)) << 4 * (g0 + g);
    }
    return bits;
  }
  __device__ __forceinline__ int count(const int32_t* ref) {
    int n = 0;
    for (int a = begin; a < end; a += 1024) {
      kept = look(ref, a);
      n += __popc(kept);
    }
    return __reduce_add_sync(0xffffffffu, n);
  }
  // each(a, four, rank, any) for every 128 pages a ..: which of a lane's four are free, how many
  // free ones are before them (`at` of them before the segment), whether any of the 128 is.
  template <typename F>
  __device__ __forceinline__ void list(const int32_t* ref, int at, F each) const {
    for (int a = begin; a < end; a += 1024) {
      const uint32_t bits = end - begin <= 1024 ? kept : look(ref, a);
      // counts of the eight 128s, a byte each: even ones, odd ones
      uint32_t n = bits - (bits >> 1 & 0x55555555u);
      n = (n & 0x33333333u) + (n >> 2 & 0x33333333u);
      const uint32_t own[2] = {n & 0x0f0f0f0fu, n >> 4 & 0x0f0f0f0fu};
      uint32_t sum[2] = {own[0], own[1]}, all[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, sum[h], o);
          if ((threadIdx.x & 31) >= o) sum[h] += y;
        }
        all[h] = __shfl_sync(0xffffffffu, sum[h], 31);
        sum[h] -= own[h];
      }
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        if (a + 128 * g >= end) break;
        const int shift = 8 * (g >> 1), any = all[g & 1] >> shift & 0xff;
        each(a + 128 * g, bits >> 4 * g & 0xfu, at + static_cast<int>(sum[g & 1] >> shift & 0xff), any != 0);
        at += any;
      }
    }
  }
};

// Sum over the lower lanes; all lanes' into *total.
__device__ __forceinline__ int scan_warp(int x, int& total) {
  const int lane = threadIdx.x & 31;
  int s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  return s - x;
}

// Entries j = first, first + step, ... below n of a row: f(j, value), several loads under way.
template <typename F>
__device__ __forceinline__ void each_entry(const int32_t* row, int first, int n, int step, F f) {
  constexpr int kBatch = 4;
  for (int j = first; j < n; j += kBatch * step) {
    int x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) x[k] = j + k * step < n ? __ldcg(row + j + k * step) : -1;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (j + k * step < n) f(j + k * step, x[k]);
  }
}

// The table's rows are cut into `chunks` parts each (32 entries in every 32 * chunks), dealt
// out to the cluster's warps.  A warp looks at 32 of its parts at once, a lane each:
// look(row, chunk) says what a lane's part needs and whether it needs anything; the parts
// that do are then the whole warp's: work(row, chunk, what).
template <typename What, typename Look, typename Do>
__device__ __forceinline__ void each_part(int rows, int chunks, int warp, int warps, Look look, Do work) {
  const int lane = threadIdx.x & 31;
  const int64_t parts = static_cast<int64_t>(rows) * chunks;
  for (int64_t u0 = warp; u0 < parts; u0 += 32LL * warps) {
    const int64_t u = u0 + static_cast<int64_t>(lane) * warps;
    const int row = static_cast<int>(u / chunks), chunk = static_cast<int>(u - static_cast<int64_t>(row) * chunks);
    What what{};
    const bool any = u < parts && look(row, chunk, what);
    for (uint32_t todo = __ballot_sync(0xffffffffu, any); todo; todo &= todo - 1) {
      const int l = __ffs(todo) - 1;
      What w;
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(What) / 4); ++i)
        reinterpret_cast<int*>(&w)[i] = __shfl_sync(0xffffffffu, reinterpret_cast<const int*>(&what)[i], l);
      work(__shfl_sync(0xffffffffu, row, l), __shfl_sync(0xffffffffu, chunk, l), w);
    }
  }
}

// Entries begin .. end - 1 of the moves: none.
__device__ __forceinline__ void no_moves(moe_page_move_t* moves, int begin, int end, int tid, int all) {
  int32_t* m = reinterpret_cast<int32_t*>(moves);  // (16-byte aligned)
  const int64_t a = 3LL * begin, z = 3LL * end, a4 = min((a + 3) / 4 * 4, z), z4 = max(z / 4 * 4, a4);
  for (int64_t j = a4 / 4 + tid; j < z4 / 4; j += all) reinterpret_cast<int4*>(m)[j] = make_int4(-1, -1, -1, -1);
  if (a + tid < a4) m[a + tid] = -1;
  if (z4 + tid < z) m[z4 + tid] = -1;
}

// What becomes of a slot.
struct Slot {
  int parent, kept, had, added;  // kept tokens, pages that the slot had
};

struct ForkArgs {
  PagesView p;
  const int32_t* parent;
  const int32_t* added;
  const int32_t* keep;
  moe_page_move_t* moves;
  int chunks;

  __device__ __forceinline__ int64_t most() const { return static_cast<int64_t>(p.stride) << p.page_log2; }
  __device__ __forceinline__ int pages(int tokens) const {
    return static_cast<int>((static_cast<int64_t>(tokens) + p.page - 1) >> p.page_log2);
  }
  __device__ __forceinline__ bool in_pool(int x) const { return static_cast<unsigned>(x) < static_cast<unsigned>(p.n_pages); }
  __device__ __forceinline__ int32_t* row(int i) const { return p.table + static_cast<size_t>(i) * p.stride; }
  __device__ __forceinline__ int32_t* note(int i) const { return p.rows + static_cast<size_t>(i) * p.stride; }
  // Until the rows change, that is: the lengths are the last step's, and keep may be them.
  __device__ __forceinline__ bool slot(int i, Slot& s) const {
    const int pa = parent[i], ad = added[i], ke = keep ? keep[i] : INT_MAX, len = p.kv_len[i];
    bool ok = pa >= -1 && pa < p.n_slots && ad >= 0 && len >= 0 && len <= most();
    const int has = ok && pa >= 0 ? p.kv_len[pa] : 0;
    const int k = max(min(ke, has), 0);
    ok = ok && has >= 0 && has <= most() && static_cast<int64_t>(k) + ad <= min(most(), static_cast<int64_t>(INT_MAX));
    s = ok ? Slot{pa, k, pages(len), ad} : Slot{-1, 0, 0, 0};
    return ok;
  }
  // The page that is not full into which the slot writes, or -1.
  __device__ __forceinline__ int landing(const Slot& s) const {
    return s.added > 0 && (s.kept & (p.page - 1)) != 0 ? row(s.parent)[pages(s.kept) - 1] : -1;
  }
};

// The pages' uses, and the slots that write into pages that are not full; with sign -1 all
// of it taken back.  False where the arrays break their bounds.
__device__ __forceinline__ bool change_uses(const ForkArgs& f, int gw, int warps, int sign) {
  const PagesView& p = f.p;
  constexpr int kBatch = 4;
  const int lane = threadIdx.x & 31;
  bool bad = false;
  int late[kBatch] = {};  // what rows that go on keep: looked at when the next entries are on their way
  each_part<Slot>(
      p.n_slots, f.chunks, gw, warps,
      [&](int i, int chunk, Slot& s) {
        bad |= !f.slot(i, s);
        const int kept = f.pages(s.kept);
        int x = -1;
        if (chunk == 0 && s.added > 0 && (s.kept & (p.page - 1)) != 0) {
          x = f.landing(s);
          if (!f.in_pool(x)) {
            bad = true;
          } else if (sign > 0) {
            atomicAdd(p.writers + x, 1);
            atomicMin(p.first + x, i);
          } else {
            p.writers[x] = 0, p.first[x] = kNoSlot;
          }
        }
        if (chunk == 0 && sign > 0) {  // (for the sums)
          p.slot[i] = make_int4(s.parent, s.kept, s.had, s.added);
          p.place[i] = make_int4(0, 0, 0, x);
        }
        return s.parent == i ? kept + 32 * chunk < s.had || (sign > 0 && 32 * chunk < kept) : 32 * chunk < max(kept, s.had);
      },
      [&](int i, int chunk, const Slot& s) {
        const int kept = f.pages(s.kept), step = 32 * f.chunks;
        const bool goes_on = s.parent == i;
        const int32_t *from = f.row(max(s.parent, 0)), *old = f.row(i);
        const int n_from = goes_on || s.parent < 0 ? 0 : kept;
        if (goes_on && sign > 0)
          for (int j = 32 * chunk + lane; j < kept; j += kBatch * step) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              bad |= !f.in_pool(late[k]);
              late[k] = j + k * step < kept ? old[j + k * step] : 0;
            }
          }
        for (int j = (goes_on ? kept : 0) + 32 * chunk + lane; j < max(n_from, s.had); j += kBatch * step) {
          int x[kBatch], y[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            x[k] = j + k * step < n_from ? from[j + k * step] : INT_MIN;
            y[k] = j + k * step < s.had ? old[j + k * step] : INT_MIN;
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const bool in = f.in_pool(x[k]);
            bad |= j + k * step < n_from && !in;
            if (in && sign > 0) f.note(i)[j + k * step] = x[k];
            if (x[k] == y[k]) continue;  // (a page that stays, as in a fork of the same trunk)
            if (in) atomicAdd(p.ref + x[k], sign);
            if (f.in_pool(y[k])) atomicSub(p.ref + y[k], sign);
          }
        }
      });
#pragma unroll
  for (int k = 0; k < kBatch; ++k) bad |= !f.in_pool(late[k]);
  return !bad;
}

// What each slot needs, what is free, and whether it fits; then the free pages that are
// needed and where each slot's ones stand among them.  One cluster; `wait` ends what changes
// the uses, and says whether that went well.
struct Middle {
  Sums box[kMostCtas], sum[2];
  Sums part[kWarps + 1];
  uint32_t free[kWarps][32];  // free pages of the warps' segments
};
template <typename Wait>
__device__ __forceinline__ bool add_up(const ForkArgs& f, cg::cluster_group& cl, Middle& m, int& copies, Wait wait) {
  const PagesView& p = f.p;
  const int lane = threadIdx.x & 31;
  const unsigned rank = cl.block_rank(), ctas = cl.num_blocks();
  const int all = static_cast<int>(ctas) * kThreads, tid = static_cast<int>(rank) * kThreads + threadIdx.x;
  // a thread's slots: neighbours, one for most pools
  const int per = (p.n_slots + all - 1) / all;
  const int i0 = min(tid * per, p.n_slots), i1 = min(i0 + per, p.n_slots);
  const bool good = wait();
  auto slot = [&](int i, Slot& s, int& x) {  // as change_uses has left them
    const int4 y = __ldcg(p.slot + i);
    s = Slot{y.x, y.y, y.z, y.w};
    x = __ldcg(&p.place[i].w);
  };
  Slot s0{-1, 0, 0, 0};
  int x0 = -1, copy0 = -1;
  if (good && i0 < i1) slot(i0, s0, x0);
  auto count = [&](const Slot& s, int copy) {
    return (static_cast<uint64_t>(f.pages(s.kept + s.added) - f.pages(s.kept) + (copy >= 0)) << kShift) + (copy >= 0);
  };
  Sums mine{0, 0, 0};
  for (int i = i0; good && i < i1; ++i) {
    Slot s = s0;
    int x = x0, copy = -1;
    if (i > i0) slot(i, s, x);
    if (x >= 0) {
      const int uses = __ldcg(p.ref + x), n = __ldcg(p.writers + x), lowest = __ldcg(p.first + x);
      if (uses > 1 && !(n == uses && lowest == i)) copy = x;
    }
    mine += Sums{count(s, copy), static_cast<uint64_t>(s.added), 0};
    if (i == i0) copy0 = copy;
    if (i > i0) p.place[i] = make_int4(0, 0, copy, x);  // (this thread's own until it is whole)
  }
  const int warp = threadIdx.x >> 5;
  FreeWords seg(p.n_pages, tid >> 5, all >> 5);
  const int64_t each = Segment::size(p.n_pages, all >> 5);
  const bool spread = each > 256 && each <= 1024;
  if (good && spread) {
    mine.free = seg.count(p.ref);
    m.free[warp][lane] = seg.kept;
  } else if (good) {
    mine.free = seg.count_free(p.ref);
  }
  Sums total;
  Sums before = scan_cta(mine, m.part, total);
  if (ctas > 1) {
    if (threadIdx.x < ctas) cl.map_shared_rank(m.box, threadIdx.x)[rank] = total;
    cl.sync();
    if (threadIdx.x < 2) {  // (by all threads 0.5 us more)
      Sums s{0, 0, 0};
      for (unsigned r = 0; r < (threadIdx.x ? ctas : rank); ++r) s += m.box[r];
      m.sum[threadIdx.x] = s;
    }
    __syncthreads();
    before += m.sum[0];
    total = m.sum[1];
  }
  const int64_t wanted = static_cast<int64_t>(total.need >> kShift);
  copies = static_cast<int>(total.need & ((1 << kShift) - 1));
  const bool bounds = good && total.added <= INT_MAX;
  if (!bounds || wanted > total.free) {
    if (tid == 0) atomicOr(p.err, bounds ? kErrNoPages : kErrBadBatch);
    return false;
  }
  // The pages that are needed are in few segments: a warp lists a 128 of each fourth one of the
  // CTA's (each its own: 15.8 us instead of 14.6).
  if (spread) {
    const int base = before.free - m.part[warp].free, g = warp & 7;
    for (int v = warp >> 3; v < kWarps; v += 4) {
      int to = base + m.part[v].free;
      if (to >= wanted) break;
      const uint32_t bits = m.free[v][lane], four = bits >> 4 * g & 0xfu;
      to += __reduce_add_sync(0xffffffffu, __popc(bits & ((1u << 4 * g) - 1)));
#pragma unroll
      for (int i = 0; i < 4; ++i) to += __popc(__ballot_sync(0xffffffffu, four & (1u << i)) & ((1u << lane) - 1));
      const int page = static_cast<int>(each * (static_cast<int>(rank) * kWarps + v)) + 128 * g + 4 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (four & (1u << i)) {
          if (to < wanted) p.ids[to] = page + i;
          ++to;
        }
    }
  }
  constexpr int kBatch = 2;
  for (int a = spread ? seg.end : seg.begin, at = before.free; a < seg.end && at < wanted; a += 128 * kBatch) {
    int4 x[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) x[k] = seg.load(p.ref, a + 128 * k, 1);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int u[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      int n;
      int to = at + scan_warp((u[0] == 0) + (u[1] == 0) + (u[2] == 0) + (u[3] == 0), n);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (u[i] == 0 && to < wanted) p.ids[to] = a + 128 * k + 4 * lane + i;
        to += u[i] == 0;
      }
      at += n;
    }
  }
  for (int i = i0; i < i1; ++i) {
    Slot s = s0;
    int x = x0, copy = copy0;
    if (i > i0) {
      slot(i, s, x);
      copy = p.place[i].z;
    }
    if (x >= 0) p.writers[x] = 0, p.first[x] = kNoSlot;  // (all have seen them)
    p.place[i] = make_int4(static_cast<int>(before.need >> kShift), static_cast<int>(before.need & ((1 << kShift) - 1)), copy, 0);
    before.need += count(s, copy);
    before.added += s.added;
    p.cu_q[i + 1] = static_cast<int32_t>(before.added);
  }
  if (tid == 0) {
    p.cu_q[0] = 0;
    *p.free_pages = total.free - static_cast<int>(wanted);
  }
  return true;
}

// The rows, lengths and moves; or what change_uses did, taken back.
__device__ __forceinline__ void change_rows(const ForkArgs& f, bool good, int copies, int tid, int all) {
  const PagesView& p = f.p;
  const int lane = threadIdx.x & 31;
  if (!good) {
    change_uses(f, tid >> 5, all >> 5, -1);
    no_moves(f.moves, 0, p.n_slots, tid, all);
    for (int i = tid; i <= p.n_slots; i += all) p.cu_q[i] = 0;
    return;
  }
  no_moves(f.moves, copies, p.n_slots, tid, all);
  struct Row {
    Slot s;
    int fresh, copy;
  };
  each_part<Row>(
      p.n_slots, f.chunks, tid >> 5, all >> 5,
      [&](int i, int chunk, Row& r) {
        const int4 s = __ldcg(p.slot + i), pl = __ldcg(p.place + i);
        r = Row{{s.x, s.y, s.z, s.w}, pl.x, pl.z};
        const int copies = pl.z >= 0;
        if (chunk == 0) {
          p.kv_len[i] = s.y + s.w;
          if (copies) {
            f.moves[pl.y] = moe_page_move_t{pl.z, __ldcg(p.ids + pl.x), s.y & (p.page - 1)};
            atomicSub(p.ref + pl.z, 1);
          }
        }
        return (s.x != i ? 0 : f.pages(s.y) - copies) + 32 * chunk < max(f.pages(s.y + s.w), s.z);
      },
      [&](int i, int chunk, const Row& r) {
        const int kept = f.pages(r.s.kept), have = f.pages(r.s.kept + r.s.added), copies = r.copy >= 0;
        const int j = 32 * chunk + lane, step = 32 * f.chunks;
        int32_t* row = f.row(i);
        if (r.s.parent != i) each_entry(f.note(i), j, kept - copies, step, [&](int at, int x) { row[at] = x; });
        for (int at = kept - copies + j; at < max(have, r.s.had); at += step) {
          const int x = at < have ? __ldcg(p.ids + r.fresh + (at - kept + copies)) : -1;
          row[at] = x;
          if (x >= 0) p.ref[x] = 1;
        }
      });
}

// A small pool: one CTA.
__global__ void __launch_bounds__(kThreads, 1) fork_kernel(const __grid_constant__ ForkArgs f) {
  __shared__ Middle m;
  cg::cluster_group cl = cg::this_cluster();
  const bool bad = !change_uses(f, threadIdx.x >> 5, kWarps, 1);
  int copies;
  const bool good = add_up(f, cl, m, copies, [&]() { return !__syncthreads_or(bad); });
  __syncthreads();
  change_rows(f, good, copies, threadIdx.x, kThreads);
}

// A large one: uses, sums, rows.  State between them: whether bounds were broken, then
// whether the rows change and the number of copies.
__global__ void __launch_bounds__(kGridThreads) fork_uses_kernel(const __grid_constant__ ForkArgs f) {
  pdl_launch_dependents();
  const int tid = blockIdx.x * kGridThreads + threadIdx.x;
  if (!change_uses(f, tid >> 5, gridDim.x * (kGridThreads / 32), 1)) atomicOr(f.p.state, 1);
}

__global__ void __launch_bounds__(kThreads, 1) fork_sums_kernel(const __grid_constant__ ForkArgs f) {
  __shared__ Middle m;
  pdl_launch_dependents();
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();  // (that the others run: before their shared memory is written to)
  int copies;
  const bool good = add_up(f, cl, m, copies, [&]() {
    pdl_wait();
    cl.barrier_wait();
    return __ldcg(f.p.state) == 0;
  });
  if (cl.block_rank() == 0 && threadIdx.x == 0) f.p.state[1] = good ? copies : -1;
}

__global__ void __launch_bounds__(kGridThreads) fork_rows_kernel(const __grid_constant__ ForkArgs f) {
  pdl_wait();
  const int copies = __ldcg(f.p.state + 1), tid = blockIdx.x * kGridThreads + threadIdx.x;
  change_rows(f, copies >= 0, copies, tid, gridDim.x * kGridThreads);
  if (tid == 0) f.p.state[0] = 0;
}

// The free pages' ranks, and both ends of the moves.  One cluster.
struct Ranks {
  int free[kMostCtas * kWarps];  // free pages of every warp's segment
  int below;
};
__device__ __forceinline__ void rank_pages(const PagesView& p, moe_page_move_t* moves, cg::cluster_group& cl, Ranks& m,
                                           int& used, int& n_moves) {
  const int lane = threadIdx.x & 31;
  const int ctas = static_cast<int>(cl.num_blocks()), warps = ctas * kWarps;
  const int tid = static_cast<int>(cl.block_rank()) * kThreads + threadIdx.x, gw = tid >> 5;
  FreeWords seg(p.n_pages, gw, warps);
  const int mine = seg.count(p.ref);
  if (threadIdx.x == 0) m.below = 0;
  if (ctas > 1) {
    cl.barrier_wait();
    if (lane < ctas) cl.map_shared_rank(&m, lane)->free[gw] = mine;
    cl.sync();
  } else {
    if (lane == 0) m.free[gw] = mine;
    __syncthreads();
  }
  // pages in use, and the free ones among the first so many: whole segments, then a part of one
  int free_before = 0, n_free = 0;
  for (int w = lane; w < warps; w += 32) {
    n_free += m.free[w];
    if (w < gw) free_before += m.free[w];
  }
  n_free = __reduce_add_sync(0xffffffffu, n_free);
  free_before = __reduce_add_sync(0xffffffffu, free_before);
  used = p.n_pages - n_free;
  const int64_t each = Segment::size(p.n_pages, warps);
  const int w_end = static_cast<int>(used / each);
  int below = 0;
  if (threadIdx.x < w_end) below = m.free[threadIdx.x];
  for (int a = static_cast<int>(w_end * each) + threadIdx.x; a < used; a += kThreads) below += __ldcg(p.ref + a) == 0;
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0 && below) atomicAdd(&m.below, below);
  __syncthreads();
  n_moves = m.below;
  if (tid == 0) *p.free_pages = n_free;

  // what tells a page's rank, and the free pages below `used`
  int2* words = reinterpret_cast<int2*>(p.ids);
  seg.list(p.ref, free_before, [&](int a, uint32_t four, int to, bool any) {
    uint32_t word = four << 4 * (lane & 7);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    const int page = a + 4 * lane;
    if ((lane & 7) == 0 && page < seg.end) words[page / 32] = make_int2(static_cast<int>(word), to);
    if (!any || a >= used) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (four & (1u << i)) {
        if (page + i < used) moves[to].dst = page + i;
        ++to;
      }
  });
}

// The uses and the table's entries of pages that move.
__device__ __forceinline__ void move_pages(const PagesView& p, moe_page_move_t* moves, int used, int n_moves, int chunks,
                                           int tid, int all) {
  const int lane = threadIdx.x & 31;
  const int2* words = reinterpret_cast<const int2*>(p.ids);
  const int stay = used - n_moves;  // pages in use that do
  auto rank = [&](int page, int2 w) {  // of a page from `used` on, -1 of a free one
    const uint32_t free = static_cast<uint32_t>(w.x), bit = 1u << (page & 31);
    return free & bit ? -1 : page - (w.y + __popc(free & (bit - 1))) - stay;
  };
  for (int page = used + tid; page < p.n_pages; page += all) {
    const int r = rank(page, __ldcg(words + (page >> 5)));
    if (r < 0) continue;
    const int dst = __ldcg(&moves[r].dst);
    moves[r].src = page, moves[r].tokens = p.page;
    p.ref[dst] = __ldcg(p.ref + page);
    p.ref[page] = 0;
  }
  no_moves(moves, n_moves, p.n_pages / 2, tid, all);
  const int64_t most = static_cast<int64_t>(p.stride) << p.page_log2;
  bool bad = false;
  each_part<int>(
      p.n_slots, chunks, tid >> 5, all >> 5,
      [&](int i, int chunk, int& n) {
        const int64_t len = min(max(static_cast<int64_t>(p.kv_len[i]), static_cast<int64_t>(0)), most);
        n = static_cast<int>((len + p.page - 1) >> p.page_log2);
        return 32 * chunk < n;
      },
      [&](int i, int chunk, int n) {
        int32_t* row = p.table + static_cast<size_t>(i) * p.stride;
        const int step = 32 * chunks;
        constexpr int kBatch = 4;
        for (int j = 32 * chunk + lane; j < n; j += kBatch * step) {
          int x[kBatch], r[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) x[k] = j + k * step < n ? row[j + k * step] : 0;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const bool in = static_cast<unsigned>(x[k]) < static_cast<unsigned>(p.n_pages);
            r[k] = in && x[k] >= used ? rank(x[k], __ldcg(words + (x[k] >> 5))) : in ? INT_MIN : -1;
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            bad |= r[k] == -1;
            r[k] = r[k] >= 0 ? __ldcg(&moves[r[k]].dst) : -1;
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
            if (r[k] >= 0) row[j + k * step] = r[k];
        }
      });
  if (bad) atomicOr(p.err, kErrBadBatch);
}

__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const PagesView p, moe_page_move_t* moves, int chunks) {
  __shared__ Ranks m;
  cg::cluster_group cl = cg::this_cluster();
  int used, n_moves;
  rank_pages(p, moves, cl, m, used, n_moves);
  __syncthreads();
  move_pages(p, moves, used, n_moves, chunks, threadIdx.x, kThreads);
}

__global__ void __launch_bounds__(kThreads, 1) compact_ranks_kernel(const PagesView p, moe_page_move_t* moves) {
  __shared__ Ranks m;
  pdl_launch_dependents();
  cg::cluster_group cl = cg::this_cluster();
  cl.barrier_arrive();
  int used, n_moves;
  rank_pages(p, moves, cl, m, used, n_moves);
  if (cl.block_rank() == 0 && threadIdx.x == 0) p.state[1] = used, p.state[2] = n_moves;
}

__global__ void __launch_bounds__(kGridThreads) compact_rows_kernel(const PagesView p, moe_page_move_t* moves, int chunks) {
  pdl_wait();
  move_pages(p, moves, __ldcg(p.state + 1), __ldcg(p.state + 2), chunks, blockIdx.x * kGridThreads + threadIdx.x,
             gridDim.x * kGridThreads);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int grid, int threads, int cluster, bool early, cudaStream_t s,
                   const Args&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A pool that gives a CTA's threads a few words each, and its warps a few rows, is one CTA's
// work (20 slots of up to 425 pages, most of them forked: 20.2 us in one CTA, 11.3 us in three
// launches; 683 slots of one page compacted: 17.2 and 7.2 us; 13 slots of 2 pages forked: 6.4
// and 8.5 us; 3 slots compacted: 5.5 and 6.8 us).
bool is_small(const PagesView& p) {
  return p.n_slots <= 128 && static_cast<int64_t>(p.n_slots) * std::min(p.stride, 64) + p.n_pages <= 4 * kThreads;
}

// Parts of a row, where `warps` warps share the rows: about as many as there are warps, of
// 32 entries at least.
int chunks_of(const PagesView& p, int warps) {
  return std::min((p.stride + 31) / 32, std::max(1, warps / p.n_slots));
}

// CTAs of a cluster: 16 where the device runs so many together (8 are what every one does;
// 344,000 pages compacted, pages read twice: 13.3 us, with 8 16.5 us).
int cluster_of(const void* kernel, std::atomic<int> (&known)[kMaxDevices]) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device >= kMaxDevices) return 8;
  int n = known[device].load(std::memory_order_relaxed);
  if (n) return n;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMostCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kMostCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int fit = 0;
  const bool ok = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                  cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) == cudaSuccess && fit > 0;
  if (!ok) cudaGetLastError();
  n = ok ? kMostCtas : 8;
  known[device].store(n, std::memory_order_relaxed);
  return n;
}

int grid_of(const PagesView& p, int n_sm) {
  const int64_t parts = static_cast<int64_t>(p.n_slots) * ((p.stride + 31) / 32);
  return static_cast<int>(std::min<int64_t>((parts + kGridThreads / 32 - 1) / (kGridThreads / 32), 4LL * n_sm));
}

}  // namespace

cudaError_t pages_fork_launch(const PagesView& p, const int32_t* parent, const int32_t* added, const int32_t* keep,
                              moe_page_move_t* moves, int n_sm, cudaStream_t s) {
  ForkArgs f{p, parent, added, keep, moves, 1};
  if (is_small(p)) {
    f.chunks = chunks_of(p, kThreads);  // (a lane looks at a part)
    return launch(fork_kernel, 1, kThreads, 1, false, s, f);
  }
  const int grid = grid_of(p, n_sm);
  f.chunks = chunks_of(p, 2 * grid * (kGridThreads / 32));
  cudaError_t e = launch(fork_uses_kernel, grid, kGridThreads, 1, false, s, f);
  static std::atomic<int> known[kMaxDevices];
  const int ctas = cluster_of(reinterpret_cast<const void*>(fork_sums_kernel), known);
  if (e == cudaSuccess) e = launch(fork_sums_kernel, ctas, kThreads, ctas, true, s, f);
  if (e == cudaSuccess) e = launch(fork_rows_kernel, grid, kGridThreads, 1, true, s, f);
  return e;
}

cudaError_t pages_compact_launch(const PagesView& p, moe_page_move_t* moves, int n_sm, cudaStream_t s) {
  if (is_small(p)) return launch(compact_kernel, 1, kThreads, 1, false, s, p, moves, chunks_of(p, kThreads));
  const int grid = std::max(grid_of(p, n_sm), n_sm);
  static std::atomic<int> known[kMaxDevices];
  const int ctas = cluster_of(reinterpret_cast<const void*>(compact_ranks_kernel), known);
  const cudaError_t e = launch(compact_ranks_kernel, ctas, kThreads, ctas, false, s, p, moves);
  if (e != cudaSuccess) return e;
  return launch(compact_rows_kernel, grid, kGridThreads, 1, true, s, p, moves, chunks_of(p, 2 * grid * (kGridThreads / 32)));
}

}  // namespace moe
