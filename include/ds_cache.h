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
 * With a tree of drafted tokens a request (below), ds_tree_masks once a cycle,
 * ds_paged_attention_tree in place of ds_paged_attention, and ds_cache_keep, which
 * gives the lengths for the last ds_cache_update. A quantised pool (below) takes the
 * calls that have `scales`.
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

/* ---- quantised pools ----------------------------------------------------------- */

/*
 * dtype DS_E4M3: K and V hold 8-bit floats (OCP FP8 E4M3, no infinities), and every
 * token's row of a head has a power of two for all of its head_dim values:
 *     x = code * 2^(scale - 127),
 * scale a byte (OCP E8M0) of `scales` [n_layers][n_pages][2][n_kv_heads][page_size],
 * contiguous, K's of a page first, then V's; 255 (not a number): the row is NaN. Such
 * a row of a pool has head_dim a multiple of 16 (strides count 8-bit elements); rows
 * outside the cache (k_new, v_new, q, out) are bfloat16.
 *   ds_cache_append_scaled   a row gets the smallest 2^e, e >= -100, with
 *       max |x| <= 448 * 2^e, and its values x / 2^e rounded to the nearest (ties to
 *       even): off by at most 2^-4 |x| or 2^(e - 10), whichever is more. A row with a
 *       value that is not finite gets scale 255 and zeros for codes. (Scales are 27 to 247. With 247,
 *       a row whose largest |x| is above 1.75 * 2^127, values from 248 * 2^120 on get the code of
 *       256, which stands for 2^128: past bfloat16 and float32, and infinite where it is restored.)
 *   ds_paged_attention_tree  reads code * 2^(scale - 127). With more than 16 rows a KV head
 *       these are rounded to bfloat16, which holds them exactly for scales from 27 (the least that
 *       append writes) to 246 (with 247 all but 2^128, see above), and to its smallest subnormal below 27; all else is as
 *       for bfloat16 pools. With up to 16 rows the products take codes as they are and q
 *       as float16 relative to its row's largest value (bfloat16's 8 bits down to 2^-31 of
 *       that, multiples of 2^-39 of it below), and weights are rounded to float16 (11 bits;
 *       fewer from 2^-29 of a row's largest weight times its value's power of two on,
 *       none below 2^-37). The codes 0x7F and 0xFF, which append does not write,
 *       must not stand in rows that a row of the call sees.
 *   ds_cache_update_scaled, ds_cache_compact_scaled   move the scales with the pages.
 * With scales = NULL the calls are those without the suffix.
 */
enum { DS_E4M3 = 2 };

ds_status ds_cache_append_scaled(const ds_append_args* args, uint8_t* scales, ds_stream_t stream);
ds_status ds_cache_update_scaled(const ds_update_args* args, uint8_t* scales, ds_stream_t stream);
ds_status ds_cache_compact_scaled(const ds_compact_args* args, uint8_t* scales, ds_stream_t stream);

/* ---- trees of drafted tokens ------------------------------------------------------ */

/*
 * The new tokens of a request may be the nodes of a tree (or several trees) that
 * hang on its cached context: its first kv_len - n_b tokens. Bit j % 32 of word
 * j / 32 of a row's mask: the row sees new token j of its request. So row i sees
 *   the context's tokens (window > 0: those at p - window + 1 and after,
 *                          p = kv_len - n_b + depth[i], depth 0 without `depth`),
 *   the new tokens of its mask, itself among them only if its bit is set.
 * Bits of tokens past n_b count for nothing. A negative depth counts as 0, one past 2^29
 * as that. `causal` of the arguments has to be 1. A request with rows but kv_len < n_b has no context, and
 * its first n_b - kv_len tokens have no place: their bits count for nothing. Table
 * entries are needed for all pages from the first that a row of depth 0 would see.
 */
typedef struct {
  const uint32_t* mask;     /* [T][mask_words] */
  int32_t mask_words;       /* >= ceil(min(max_q, T) / 32), <= 2^18 */
  const int32_t* depth;     /* [T] or NULL; looked at only if window > 0 */
} ds_tree;

/* ds_paged_attention over a pool with or without `scales`, of a tree or (NULL) not. */
ds_status ds_paged_attention_tree(const ds_attention_args* args, const uint8_t* scales, const ds_tree* tree,
                                  ds_stream_t stream);

/*
 * Masks and depths of trees given by their nodes' parents: rows as in ds_append_args,
 * parent[t] the place within the request of row t's parent, -1 for a root. A
 * parent comes before its children; any other value: DS_ERR_BOUNDS, and the node
 * counts as a root. depth = number of ancestors; mask: the node and its ancestors
 * (window > 0: those less than `window` above it). A request outside the limits
 * (longer than max_q, rows outside [0, T)): DS_ERR_BOUNDS, its rows are left alone.
 */
typedef struct {
  int32_t B, T;                 /* 1 <= B <= 65535, 0 <= T <= 2^23 */
  int32_t max_q;                /* upper bound of n_b, 1..4096 */
  int32_t mask_words;           /* >= ceil(min(max_q, T) / 32), <= 2^18 */
  int32_t window;               /* 0: none */
  const int32_t* parent;        /* [T] */
  const int32_t* q_start;       /* [B+1] */
  uint32_t* mask;               /* out [T][mask_words] */
  int32_t* depth;               /* out [T], or NULL */
  int32_t* status;
} ds_tree_args;

ds_status ds_tree_masks(const ds_tree_args* args, ds_stream_t stream);

/*
 * Keeps a path of each request's new tokens: for i < m_b, the number of entries of
 * path[b] before its first negative one, the row at position first + path[b][i]
 * goes to position first + i, first = kv_len[b] - n_b, K and V of all layers; and
 * new_len[b] = first + m_b, the length to go on with (ds_cache_update). The path's
 * entries ascend, below n_b. Rows move in place: what stood at the places that are
 * written and is not of the path is lost. Pages that other requests hold must not be written
 * (as by ds_cache_append). A request whose rows, length (below n_b, too) or path is out of these
 * limits, or which needs a page outside [0, n_pages): DS_ERR_BOUNDS, its rows stay, new_len[b] = kv_len[b].
 */
typedef struct {
  ds_kv_pool pool;
  int32_t B, T, max_pages;
  int32_t path_len;             /* 1..4096 */
  const int32_t* path;          /* [B][path_len] */
  const int32_t* q_start;       /* [B+1] */
  const int32_t* block_table;   /* [B][max_pages] */
  const int32_t* kv_len;        /* [B], the new tokens counted */
  int32_t* new_len;             /* out [B], not overlapping the inputs */
  uint8_t* scales;              /* of a quantised pool, else NULL */
  int32_t* status;
} ds_keep_args;

ds_status ds_cache_keep(const ds_keep_args* args, ds_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DS_CACHE_H */
