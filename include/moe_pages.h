/*
 * moe_pages.h - C ABI of the page pool of a key/value cache: which sequence has which
 * pages.  Sequences are forked (for several answers, beams, drafts at different points),
 * extended, cut back and freed on the device, with no word from the host, so that a
 * captured graph can hold a whole step; their pages are shared until one of them is
 * written to.  The pool knows page numbers only: a model has one pool and a cache
 * (moe_attn.h) for each layer, in which the pool's moves are then copied.
 * Part of libmoe.so; conventions are those of moe_attn.h.  Calls work on the device that
 * was current when the handle was made.
 *
 * A pool's state is the caller's memory, borrowed for the handle's lifetime, and the
 * caller may look at it and set it between calls:
 *   table  [n_slots][table_stride] page ids of the sequences' tokens, in their order;
 *          entries from ceil(kv_len / page_size) on are -1
 *   kv_len [n_slots] tokens of each slot's sequence, 0 for none
 *   ref    [n_pages] how often a page stands in the table; a caller who adds to an entry
 *          keeps the page (for sequences to come).  Pages with 0 are free.
 *   cu_q   [n_slots + 1] offsets of the new tokens: with table and kv_len a batch of
 *          moe_attn.h
 *   free_pages [1] number of free pages after the call
 * Whatever the arrays hold, nothing outside of them is read or written.
 */
#ifndef MOE_PAGES_H_
#define MOE_PAGES_H_

#include "moe_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_pages moe_pages_t;
typedef struct {
  int n_pages;      /* 1 .. 2^27 */
  int page_size;    /* 16, 32, 64 or 128 tokens */
  int n_slots;      /* 1 .. 65535 */
  int table_stride; /* 1 .. 2^24, n_slots * table_stride at most 2^28 */
} moe_pages_config_t;
typedef struct {
  int32_t* table;
  int32_t* kv_len;
  int32_t* ref;
  int32_t* cu_q;
  int32_t* free_pages;
} moe_pages_store_t;

/* Checks cfg (MOE_ERR_UNSUPPORTED) and that the store's arrays lie in device memory and
 * hold what cfg implies; allocates the workspace. */
moe_status_t moe_pages_create(const moe_pages_config_t* cfg, const moe_pages_store_t* store,
                              moe_pages_t** out);
size_t moe_pages_workspace_bytes(const moe_pages_config_t* cfg); /* 0 if cfg is invalid */
const char* moe_pages_last_error(const moe_pages_t* h);          /* NULL: moe_last_error(NULL) */
void moe_pages_destroy(moe_pages_t* h); /* device synchronise, then free; NULL is ignored */

/* The next step's sequences out of the last one's, all at once.  parent, added and keep:
 * [n_slots] on the device.  Slot i becomes the first min(keep[i], kv_len[parent[i]]) tokens
 * (all where keep is NULL; none for a negative one) of what slot parent[i] held, and none where
 * parent[i] is -1, with room for added[i] tokens behind them.  So parent[i] == i goes on, with
 * rejected drafts cut off; another parent is a fork; sequences that no slot names end, and pages
 * that no slot needs any more are free at once.  Kept pages are shared, except that a slot with
 * new tokens in a page that is not full, and that others use or the caller keeps, gets a copy of
 * it: all such slots but the lowest where they are the page's only users, else all.  New pages
 * are the free pages of the lowest numbers, in order of the slots; in a slot the copy comes first.
 * cu_q becomes the sums of added, kv_len the new lengths.  moves: [n_slots]; the copies in order
 * of their slots (moe_kv_copy in every layer, before the step's tokens are written), then
 * entries of -1.
 * A call that needs more pages than are free (bit 3 of moe_pages_device_status), or whose
 * arrays break their bounds (parent outside [-1, n_slots), added below 0, lengths above
 * table_stride pages, kept page ids outside [0, n_pages): bit 1), changes nothing but cu_q,
 * which becomes all 0, and moves, all -1: the rest of a step then has no tokens. */
moe_status_t moe_pages_fork(moe_pages_t* h, const int32_t* parent, const int32_t* added,
                            const int32_t* keep, moe_page_move_t* moves, void* stream);

/* Moves the pages in use (ref not 0) to the front of the pool: the k-th of those behind it
 * takes the k-th free page there, both by their numbers.  Updates table and ref; moves:
 * [n_pages / 2], the pages that move in that order (all of their tokens), then entries of -1.
 * Table entries outside [0, n_pages) stay and, within a sequence's length, set bit 1. */
moe_status_t moe_pages_compact(moe_pages_t* h, moe_page_move_t* moves, void* stream);

/* Copies the handle's device error word to *flags (synchronous) and clears it;
 * MOE_ERR_CUDA when it was not 0.  Bit 1: a call's arrays broke their bounds; bit 3: the
 * pool had too few free pages. */
moe_status_t moe_pages_device_status(moe_pages_t* h, int32_t* flags);

#ifdef __cplusplus
}
#endif

#endif /* MOE_PAGES_H_ */
