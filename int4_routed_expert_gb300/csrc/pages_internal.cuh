// Internal declarations of the page pool (include/moe_pages.h).
#pragma once

#include "../../include/moe_pages.h"
#include "attn_internal.cuh"

namespace moe {

constexpr int kErrNoPages = 8;  // device error bit of a pool: too few free pages
constexpr int kNoSlot = 0x7f7f7f7f;  // above every slot, a byte repeated

// What the kernels know of a pool (by value).
struct PagesView {
  int32_t* table;
  int32_t* kv_len;
  int32_t* ref;
  int32_t* cu_q;
  int32_t* free_pages;
  int n_pages, n_slots, stride, page, page_log2;
  int* err;
  // workspace
  int* state;          // [3] between the launches of a call: broken bounds (0 between calls), and sizes
  int4* slot;          // [n_slots] parent, kept tokens, pages that it had, added tokens
  int4* place;         // [n_slots] first of its new pages, rank of its copy, page that it copies or -1
  int32_t* rows;       // [n_slots][stride] kept pages of slots whose parent is another
  int32_t* ids;        // [n_pages] free pages, or {free ones, free ones before} of every 32 pages
  int32_t* writers;    // [n_pages] slots that write into a page that is not full; 0 between calls
  int32_t* first;      // [n_pages] the lowest of them; kNoSlot between calls
};

cudaError_t pages_fork_launch(const PagesView& p, const int32_t* parent, const int32_t* added, const int32_t* keep,
                              moe_page_move_t* moves, int n_sm, cudaStream_t s);
cudaError_t pages_compact_launch(const PagesView& p, moe_page_move_t* moves, int n_sm, cudaStream_t s);
cudaError_t kv_copy_launch(const KvView& c, const moe_page_move_t* moves, int n, int n_sm, cudaStream_t s);

}  // namespace moe
