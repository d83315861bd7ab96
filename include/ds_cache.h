/*
 * ds_cache.h -- C ABI of the paged key/value cache of the verify cycle: the
 * pages' bookkeeping, the new tokens' keys and values, and the attention that
 * reads them (one GPU, NVIDIA GB300 / sm_103a).
 *
 * Method sources (cited by page and section, as in ds_draft.h):
 *   [DSpark]  배경: the target scores K drafted tokens and the next one in a
 *             single pass over a cached context, then the sequence falls back
 *             to the accepted prefix.
 *   [DFlash]  1 + K query tokens per request and cycle, and the draft backbone's
 *             non-causal attention of a block over the injected context.
 *   [vLLM-V4] pages of up to 256 tokens, sliding windows.
 *
 * The conventions of ds_draft.h hold: the caller owns every buffer, calls
 * enqueue on `stream` and return, host-checkable arguments are refused before
 * anything is launched, conditions only the device can see go to `status`
 * (first error wins), no call synchronises, allocates or keeps a pointer, and
 * every call can be captured into a CUDA graph. Pointers are 16-byte aligned
 * unless a field says otherwise. Strides are in elements. Calls launch on the
 * current device, where the buffers have to be.
 *
 * One cycle with a cache:
 *   ds_cache_update  (new_len = kv_len + n)      pages for the n new tokens
 *   ds_cache_append, ds_paged_attention          per layer
 *   ... logits ..., ds_verify
 *   ds_cache_update  (new_len = accepted prefix) back to what was accepted
 */
#ifndef DS_CACHE_H
#define DS_CACHE_H

#include "ds_draft.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A pool of pages for all layers: K and V [n_layers][n_pages][page_size]
 * [n_kv_heads][head_dim], the last index contiguous, the others at the given
 * strides (the same for K and V), so tokens or heads may be outermost in a
 * page and K and V may be interleaved.
 *   page_size   16, 32, 64, 128 or 256 tokens
 *   n_pages     1..2^28, n_layers 1..2^28
 *   head_dim    a multiple of 8, at most 256 (ds_paged_attention: 64 or 128)
 *   n_kv_heads  1..256
 *   strides     multiples of 16 bytes, >= head_dim (layer_stride is not read
 *               if n_layers = 1)
 */
typedef struct {
  int32_t dtype;              /* ds_dtype of k and v */
  int32_t n_layers, n_pages, page_size, n_kv_heads, head_dim;
  void* k;
  void* v;
  int64_t layer_stride, page_stride, token_stride, head_stride;
} ds_kv_pool;

/*
 * New tokens of B requests come as ragged rows: request b has rows
 * q_start[b] .. q_start[b+1] - 1 of T; its row i stands at position
 * kv_len[b] - n_b + i, n_b = q_start[b+1] - q_start[b]: kv_len counts the new
 * tokens. Position p lives in page block_table[b][p / page_size], entry
 * p % page_size. Positions below zero (n_b > kv_len[b]) belong to no token.
 * Rows outside [0, T), a kv_len outside [0, max_pages * page_size] or a page
 * outside [0, n_pages) that a call needs: DS_ERR_BOUNDS in `status`; nothing
 * outside the buffers is read or written. max_pages * page_size <= 2^30,
 * T <= 2^23.
 */

/* ---- new keys and values into their pages --------------------------------- */

typedef struct {
  ds_kv_pool pool;
  int32_t layer;
  int32_t B, T, max_pages;      /* 1 <= B <= 65535, T >= 0, max_pages >= 1 */
  const void* k_new;            /* [T][n_kv_heads][head_dim] of the pool's dtype */
  const void* v_new;
  int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride; /* multiples of 16 bytes */
  const int32_t* q_start;       /* [B+1] */
  const int32_t* block_table;   /* [B][max_pages] */
  const int32_t* kv_len;        /* [B], the new tokens counted */
  int32_t* status;
} ds_append_args;

/* Copies row i of request b to its position's place in K and V of `layer`.
 * A request's tokens go to distinct places; pages shared between requests must
 * not be written (ds_cache_update sees to that). */
ds_status ds_cache_append(const ds_append_args* args, ds_stream_t stream);

/* ---- attention of ragged new tokens over the cache ------------------------- */

/*
 * Query head h of n_heads = G * n_kv_heads reads KV head h / G. A row at
 * position p sees the cached tokens
 *     j in [lo, hi),  hi = causal ? min(p + 1, kv_len) : kv_len,
 *                     lo = window > 0 ? max(0, p - window + 1) : 0,
 * and gets, with s_j = scale * (q . k_j),
 *     lse = ln sum_j exp(s_j),   out = sum_j exp(s_j - lse) v_j.
 * A row that sees nothing gets out = 0 and lse = -inf. What lies in the pages
 * outside a row's view (past kv_len, before the window, later tokens) has no
 * effect on it, whatever its bits; pages that no row sees need no table entry.
 * (Values that are not finite, seen by some rows of a request and not by others,
 * cost those others a second, slow computation: bfloat16 58 to 217 rows x keys a
 * us and SM, float32 2 to 4. In bfloat16 calls of up to 16 rows a KV head it is done
 * for the rows that see the value, too.)
 * bfloat16: products and sums in float32, the weights exp(s_j - r) of the
 * value product rounded to bfloat16. float32: all in float32; 256 KV heads over a
 * table of more than 2^30 - 128 tokens are DS_ERR_UNSUPPORTED.
 * `out` must not overlap q or the pool.
 */
typedef struct {
  ds_kv_pool pool;              /* head_dim 64 or 128 */
  int32_t layer;
  int32_t B, T, max_pages;
  int32_t max_q;                /* upper bound of n_b, >= 1 (a longer request: DS_ERR_BOUNDS) */
  int32_t n_heads;              /* multiple of n_kv_heads, at most 128 per KV head */
  int32_t causal;               /* 0 or 1 */
  int32_t window;               /* 0: none */
  float scale;                  /* finite, > 0 */
  const void* q;                /* [T][n_heads][head_dim] */
  int64_t q_token_stride, q_head_stride;     /* multiples of 16 bytes */
  const int32_t* q_start;       /* [B+1] */
  const int32_t* block_table;   /* [B][max_pages] */
  const int32_t* kv_len;        /* [B] */
  void* out;                    /* out [T][n_heads][head_dim], the pool's dtype */
  int64_t out_token_stride, out_head_stride; /* multiples of 16 bytes */
  float* lse;                   /* optional out [T][n_heads], or NULL (4-byte aligned) */
  void* workspace;              /* ds_paged_attention_workspace_bytes(...) bytes */
  size_t workspace_bytes;
  int32_t* status;
} ds_attention_args;

/* Does not depend on the batch, the lengths or max_q. 0: not supported. */
size_t ds_paged_attention_workspace_bytes(int32_t dtype, int32_t head_dim);
ds_status ds_paged_attention(const ds_attention_args* args, ds_stream_t stream);

/* ---- the pages' bookkeeping -------------------------------------------------- */

/*
 * Every request's next state in one call. Request b continues request
 * parent[b] (parent NULL: itself; -1: nothing), keeps
 *     keep = min(kv_len[parent[b]], new_len[b])   (0 without a parent)
 * tokens of it and has pages for new_len[b] tokens afterwards: growing, falling
 * back, ending (new_len 0), forking and reordering of beams are one operation.
 *   - The ceil(keep / page_size) kept pages are shared with the parent.
 *     ref[p] counts the rows of the table that hold page p, plus whatever the
 *     caller adds for holders of its own (a prefix cache); 0 is free.
 *   - Copy on write: a request that will write into a partly filled kept page
 *     (keep % page_size != 0 and new_len > keep) which has other holders after
 *     the call gets a page of its own with the keep % page_size tokens copied,
 *     K and V of all layers. If all holders are such writers, the lowest
 *     request keeps the page.
 *   - New pages are the lowest pages without a holder after the call, given
 *     out in the order of the requests and of their positions.
 * State comes in through (block_table, kv_len, ref) and goes out through
 * (table_out, len_out, ref_out), which must not overlap it; table_out is -1
 * past a request's pages. Too few free pages (DS_ERR_PAGES), or a length,
 * parent, count or page out of range (DS_ERR_BOUNDS): the state out is the
 * state in, and no page is written.
 */
typedef struct {
  ds_kv_pool pool;
  int32_t B, max_pages;         /* 1 <= B <= 65535, 1 <= max_pages */
  const int32_t* block_table;   /* [B][max_pages] */
  const int32_t* kv_len;        /* [B] */
  const int32_t* ref;           /* [n_pages] */
  const int32_t* parent;        /* [B] or NULL */
  const int32_t* new_len;       /* [B] */
  int32_t* table_out;           /* out [B][max_pages] */
  int32_t* len_out;             /* out [B] */
  int32_t* ref_out;             /* out [n_pages] */
  void* workspace;              /* ds_cache_update_workspace_bytes(B, n_pages) bytes */
  size_t workspace_bytes;
  int32_t* status;
} ds_update_args;

size_t ds_cache_update_workspace_bytes(int32_t B, int32_t n_pages);
ds_status ds_cache_update(const ds_update_args* args, ds_stream_t stream);

/*
 * Moves the held pages to the front: with U = #{p : ref[p] > 0}, the i-th held
 * page at or above U goes to the i-th free page below U, K and V of all
 * layers. Table and counts are rewritten (out of place, as above); page_map[p]
 * is where held page p is afterwards, -1 for a free one, for holders outside
 * the table; n_used = U. A table entry outside [0, n_pages) becomes -1. A
 * negative count: DS_ERR_BOUNDS, state out = state in, nothing moved.
 */
typedef struct {
  ds_kv_pool pool;
  int32_t B, max_pages;
  const int32_t* block_table;   /* [B][max_pages], -1 past a request's pages */
  const int32_t* ref;           /* [n_pages] */
  int32_t* table_out;           /* out [B][max_pages] */
  int32_t* ref_out;             /* out [n_pages] */
  int32_t* page_map;            /* out [n_pages] */
  int32_t* n_used;              /* out [1] (4-byte aligned) */
  void* workspace;              /* ds_cache_compact_workspace_bytes(n_pages) bytes */
  size_t workspace_bytes;
  int32_t* status;
} ds_compact_args;

size_t ds_cache_compact_workspace_bytes(int32_t n_pages);
ds_status ds_cache_compact(const ds_compact_args* args, ds_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DS_CACHE_H */
