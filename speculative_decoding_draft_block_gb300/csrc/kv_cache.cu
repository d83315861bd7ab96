// C ABI of the paged cache: argument checks and launches, and the kernel that
// writes new keys and values into their pages. The contract of every entry
// point is in include/ds_cache.h.
#include <math.h>
#include <string.h>

#include <initializer_list>

#include "common.cuh"
#include "internal.h"
#include "kv_internal.h"
#include "sm100.cuh"

namespace ds {
namespace {

// ---- append -------------------------------------------------------------------
//
// pool[table[b][p / S]][p % S] = new[q_start[b] + i], p = kv_len[b] - n_b + i:
// a gather of ragged rows into pages, 4 * T * Hk * D * e bytes moved and
// nothing computed. A block takes kTokens consecutive rows; all its
// threads find the rows' requests together by counting the requests that end
// at or before each row (one coalesced pass over q_start, no chain of
// dependent loads as in a bisection per row). Where q_start decreases somewhere, that
// may find a request which ends before the row: no place, and the first block
// reports every malformed request. Bound by memory: prompts of 16 requests
// (462 MB) 71.7 us, 6.4 TB/s; below a few MB by the launch, 6 to 7 us.
constexpr int kAppendThreads = 256;

// kTokens rows a block: see launch_append.
template <int kTokens>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  static_assert(kTokens <= 32, "a lane a row");
  __shared__ int ends[kTokens];
  __shared__ int64_t at[kTokens];  // byte offset of the row's place in the pool, -1: none
  const int t0 = blockIdx.x * kTokens;
  const int tid = threadIdx.x;
  if (tid < kTokens) ends[tid] = 0;
  int before = 0;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  __syncthreads();
  for (int i = tid; i < p.B; i += kAppendThreads) {
    const int e = __ldcg(p.q_start + i + 1);
    if (blockIdx.x == 0) {
      const int s = __ldcg(p.q_start + i);
      if (s < 0 || e < s || e > p.T) report(p.status, kErrBounds);
    }
    if (e <= t0)
      ++before;
    else if (e < t0 + kTokens)
      atomicAdd(&ends[e - t0], 1);
  }
  // requests that end at or before t0, over the block
  before = __reduce_add_sync(0xffffffffu, before);
  __shared__ int warp_before[kAppendThreads / 32];
  if ((tid & 31) == 0) warp_before[tid >> 5] = before;
  __syncthreads();
  if (tid < kTokens) {
    int b = 0;
    for (int w = 0; w < kAppendThreads / 32; ++w) b += warp_before[w];
    int here = tid > 0 ? ends[tid] : 0;  // requests that end at the block's rows 1 .. tid
    constexpr uint32_t kLanes = kTokens == 32 ? 0xffffffffu : (1u << kTokens) - 1;
#pragma unroll
    for (int d = 1; d < kTokens; d <<= 1) {
      const int v = __shfl_up_sync(kLanes, here, d);
      if (tid >= d) here += v;
    }
    b += here;
    const int t = t0 + tid;
    int64_t off = -1;
    if (t < p.T && b < p.B) {
      const int64_t cap = (int64_t)p.max_pages << p.pool.page_shift;
      const Request r = load_request(p.q_start, p.kv_len, b, p.T, p.T, cap);
      const int i = t - r.q0, pos = r.kv - r.n + i;
      if (!r.ok) {
        report(p.status, kErrBounds);
      } else if (i >= 0 && i < r.n && pos >= 0) {
        const int page = __ldcg(p.block_table + (int64_t)b * p.max_pages + (pos >> p.pool.page_shift));
        if (page < 0 || page >= p.pool.n_pages)
          report(p.status, kErrBounds);
        else
          off = (int64_t)page * p.pool.page_stride +
                (int64_t)(pos & ((1 << p.pool.page_shift) - 1)) * p.pool.token_stride;
      }
    }
    at[tid] = off;
  }
  __syncthreads();
  const int chunks = p.pool.row_bytes >> 4;        // 16-byte pieces of a head's row
  const int per_token = chunks * p.pool.n_kv_heads;
  for (int x = tid; x < kTokens * per_token; x += kAppendThreads) {
    const int i = x / per_token, y = x - i * per_token;
    const int h = y / chunks, c = y - h * chunks;
    const int64_t off = at[i];
    if (off < 0) continue;
    const int64_t t = t0 + i;
    const uint4 kk = __ldcg(reinterpret_cast<const uint4*>(p.k_new + t * p.k_token + h * p.k_head) + c);
    const uint4 vv = __ldcg(reinterpret_cast<const uint4*>(p.v_new + t * p.v_token + h * p.v_head) + c);
    const int64_t o = off + h * p.pool.head_stride;
    reinterpret_cast<uint4*>(p.pool.k + o)[c] = kk;
    reinterpret_cast<uint4*>(p.pool.v + o)[c] = vv;
  }
}

// ---- argument checks --------------------------------------------------------------

bool aligned(const void* p, unsigned a) { return p != nullptr && ((uintptr_t)p & (a - 1)) == 0; }

int esize(int32_t dtype) { return dtype == DS_BF16 ? 2 : 4; }

bool strides16(std::initializer_list<int64_t> strides, int32_t dtype) {
  for (int64_t s : strides)
    if (s <= 0 || (s * esize(dtype)) % 16 != 0) return false;
  return true;
}

// The pool's fields, and its view with `layer` as base (all layers: layer 0).
ds_status check_pool(const ds_kv_pool& a, int32_t layer, PoolView* v) {
  if (a.dtype != DS_F32 && a.dtype != DS_BF16) return DS_ERR_INVALID_ARG;
  if (a.n_layers < 1 || a.n_layers > (1 << 28) || a.n_pages < 1 || a.n_pages > (1 << 28) || layer < 0 ||
      layer >= a.n_layers)
    return DS_ERR_INVALID_ARG;
  if (a.page_size < 16 || a.page_size > 256 || (a.page_size & (a.page_size - 1)) != 0) return DS_ERR_INVALID_ARG;
  if (a.n_kv_heads < 1 || a.n_kv_heads > 256) return DS_ERR_INVALID_ARG;
  if (a.head_dim < 8 || a.head_dim > 256 || a.head_dim % 8 != 0) return DS_ERR_INVALID_ARG;
  if (!aligned(a.k, 16) || !aligned(a.v, 16)) return DS_ERR_INVALID_ARG;
  if (!strides16({a.page_stride, a.token_stride, a.head_stride}, a.dtype)) return DS_ERR_INVALID_ARG;
  if (a.page_stride < a.head_dim || a.token_stride < a.head_dim || a.head_stride < a.head_dim)
    return DS_ERR_INVALID_ARG;
  if (a.n_layers > 1 && (!strides16({a.layer_stride}, a.dtype) || a.layer_stride < a.head_dim))
    return DS_ERR_INVALID_ARG;
  const int64_t e = esize(a.dtype);
  v->layer_stride = a.n_layers > 1 ? a.layer_stride * e : 0;
  v->page_stride = a.page_stride * e;
  v->token_stride = a.token_stride * e;
  v->head_stride = a.head_stride * e;
  v->k = static_cast<char*>(a.k) + layer * v->layer_stride;
  v->v = static_cast<char*>(a.v) + layer * v->layer_stride;
  v->n_layers = a.n_layers;
  v->n_pages = a.n_pages;
  v->page_shift = 31 - __builtin_clz((unsigned)a.page_size);
  v->n_kv_heads = a.n_kv_heads;
  v->row_bytes = a.head_dim * (int32_t)e;
  return DS_OK;
}

// Requests, rows and table of a call over ragged rows. Positions are 32-bit.
bool rows_ok(int32_t B, int32_t T, int32_t max_pages, int32_t page_size) {
  return B >= 1 && B <= 65535 && T >= 0 && T <= (1 << 23) && max_pages >= 1 && (int64_t)max_pages * page_size <= (1 << 30);
}

bool overlap(const void* a, const void* b, size_t na, size_t nb) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
  const int pieces = p.pool.n_kv_heads * (p.pool.row_bytes >> 4);  // 16-byte pieces of a row
  // Eight rows of 1 KB and more keep a block's threads busy, of smaller rows it takes
  // more: 16 prompts (56 k rows) of 128 bytes 6.2 us by 32 rows a block, 12.3 by 8;
  // of 512 bytes 22.0 and 23.1; of 1 KB 39.3 and 38.4; of 2 KB 74.4 and 71.8.
  const int tokens = pieces >= 64 ? 8 : 32;
  const dim3 blocks((p.T + tokens - 1) / tokens);
  return launch_early(tokens == 8 ? append_kernel<8> : append_kernel<32>, blocks, dim3(kAppendThreads), 0, s, p);
}

}  // namespace ds

using namespace ds;

extern "C" {

ds_status ds_cache_append(const ds_append_args* a, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  AppendParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, a->layer, &p.pool);
  if (ps != DS_OK) return ps;
  if (!rows_ok(a->B, a->T, a->max_pages, a->pool.page_size)) return DS_ERR_INVALID_ARG;
  const void* ptrs[] = {a->q_start, a->block_table, a->kv_len, a->status};
  for (const void* q : ptrs)
    if (!aligned(q, 16)) return DS_ERR_INVALID_ARG;
  if (a->T == 0) return DS_OK;
  if (!aligned(a->k_new, 16) || !aligned(a->v_new, 16)) return DS_ERR_INVALID_ARG;
  if (!strides16({a->k_token_stride, a->k_head_stride, a->v_token_stride, a->v_head_stride}, a->pool.dtype))
    return DS_ERR_INVALID_ARG;
  const ds_status st = device_supported();
  if (st != DS_OK) return st;
  const int64_t e = esize(a->pool.dtype);
  p.B = a->B;
  p.T = a->T;
  p.max_pages = a->max_pages;
  p.k_new = static_cast<const char*>(a->k_new);
  p.v_new = static_cast<const char*>(a->v_new);
  p.k_token = a->k_token_stride * e;
  p.k_head = a->k_head_stride * e;
  p.v_token = a->v_token_stride * e;
  p.v_head = a->v_head_stride * e;
  p.q_start = a->q_start;
  p.block_table = a->block_table;
  p.kv_len = a->kv_len;
  p.status = a->status;
  return launch_append(p, (cudaStream_t)stream) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

size_t ds_paged_attention_workspace_bytes(int32_t dtype, int32_t head_dim) {
  if ((dtype != DS_F32 && dtype != DS_BF16) || (head_dim != 64 && head_dim != 128)) return 0;
  return attention_ws_bytes(head_dim);
}

ds_status ds_paged_attention(const ds_attention_args* a, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, a->layer, &p.pool);
  if (ps != DS_OK) return ps;
  if (a->pool.head_dim != 64 && a->pool.head_dim != 128) return DS_ERR_UNSUPPORTED;
  if (!rows_ok(a->B, a->T, a->max_pages, a->pool.page_size)) return DS_ERR_INVALID_ARG;
  if (a->max_q < 1 || a->n_heads < 1 || a->n_heads % a->pool.n_kv_heads != 0 ||
      a->n_heads / a->pool.n_kv_heads > 128)
    return DS_ERR_INVALID_ARG;
  if (!work_fits(a->pool.dtype, (int64_t)a->max_pages * a->pool.page_size, a->pool.n_kv_heads)) return DS_ERR_UNSUPPORTED;
  if ((a->causal != 0 && a->causal != 1) || a->window < 0 || !isfinite(a->scale) ||
      !(a->scale > 0.f))
    return DS_ERR_INVALID_ARG;
  const void* ptrs[] = {a->q_start, a->block_table, a->kv_len, a->status};
  for (const void* q : ptrs)
    if (!aligned(q, 16)) return DS_ERR_INVALID_ARG;
  if (a->lse != nullptr && !aligned(a->lse, 4)) return DS_ERR_INVALID_ARG;
  if (!aligned(a->workspace, 16) || a->workspace_bytes < attention_ws_bytes(a->pool.head_dim))
    return DS_ERR_WORKSPACE;
  if (a->T == 0) return DS_OK;
  if (!aligned(a->q, 16) || !aligned(a->out, 16)) return DS_ERR_INVALID_ARG;
  if (!strides16({a->q_token_stride, a->q_head_stride, a->out_token_stride, a->out_head_stride}, a->pool.dtype))
    return DS_ERR_INVALID_ARG;
  const ds_status st = device_supported();
  if (st != DS_OK) return st;
  const int64_t e = esize(a->pool.dtype);
  p.dtype = a->pool.dtype;
  p.D = a->pool.head_dim;
  p.B = a->B;
  p.T = a->T;
  p.max_pages = a->max_pages;
  p.max_q = a->max_q < a->T ? a->max_q : a->T;
  p.n_heads = a->n_heads;
  p.group = a->n_heads / a->pool.n_kv_heads;
  p.by_group.set((uint32_t)p.group);
  p.causal = a->causal;
  // a window as long as the table hides nothing
  p.window = (int64_t)a->window >= (int64_t)a->max_pages * a->pool.page_size ? 0 : a->window;
  p.scale = a->scale;
  p.q = static_cast<const char*>(a->q);
  p.out = static_cast<char*>(a->out);
  p.q_token = a->q_token_stride * e;
  p.q_head = a->q_head_stride * e;
  p.o_token = a->out_token_stride * e;
  p.o_head = a->out_head_stride * e;
  p.q_start = a->q_start;
  p.block_table = a->block_table;
  p.kv_len = a->kv_len;
  p.lse = a->lse;
  p.workspace = static_cast<char*>(a->workspace);
  p.status = a->status;
  const cudaError_t err = p.dtype == DS_BF16 ? launch_attention_tc(p, (cudaStream_t)stream)
                                             : launch_attention_f32(p, (cudaStream_t)stream);
  return err == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

size_t ds_cache_update_workspace_bytes(int32_t B, int32_t n_pages) {
  if (B < 1 || B > 65535 || n_pages < 1) return 0;
  return update_ws_bytes(B, n_pages);
}

ds_status ds_cache_update(const ds_update_args* a, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  UpdateParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, 0, &p.pool);
  if (ps != DS_OK) return ps;
  if (!rows_ok(a->B, 0, a->max_pages, a->pool.page_size)) return DS_ERR_INVALID_ARG;
  const void* ptrs[] = {a->block_table, a->kv_len, a->ref, a->new_len, a->table_out, a->len_out, a->ref_out,
                        a->status};
  for (const void* q : ptrs)
    if (!aligned(q, 16)) return DS_ERR_INVALID_ARG;
  if (a->parent != nullptr && !aligned(a->parent, 16)) return DS_ERR_INVALID_ARG;
  const size_t nb = (size_t)a->B * 4, nt = nb * (size_t)a->max_pages, np = (size_t)a->pool.n_pages * 4;
  const struct { const void* p; size_t n; } in[] = {{a->block_table, nt}, {a->kv_len, nb}, {a->ref, np},
                                                    {a->new_len, nb}, {a->parent, a->parent ? nb : 0}},
                                            out[] = {{a->table_out, nt}, {a->len_out, nb}, {a->ref_out, np}};
  for (int i = 0; i < 3; ++i) {
    for (const auto& x : in)
      if (x.n && overlap(out[i].p, x.p, out[i].n, x.n)) return DS_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[j].p, out[i].n, out[j].n)) return DS_ERR_INVALID_ARG;
  }
  if (!aligned(a->workspace, 16) || a->workspace_bytes < update_ws_bytes(a->B, a->pool.n_pages))
    return DS_ERR_WORKSPACE;
  const ds_status st = device_supported();
  if (st != DS_OK) return st;
  p.B = a->B;
  p.max_pages = a->max_pages;
  p.table = a->block_table;
  p.kv_len = a->kv_len;
  p.ref = a->ref;
  p.parent = a->parent;
  p.new_len = a->new_len;
  p.table_out = a->table_out;
  p.len_out = a->len_out;
  p.ref_out = a->ref_out;
  p.ws = static_cast<int32_t*>(a->workspace);
  p.status = a->status;
  return launch_update(p, (cudaStream_t)stream) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

size_t ds_cache_compact_workspace_bytes(int32_t n_pages) { return n_pages < 1 ? 0 : compact_ws_bytes(n_pages); }

ds_status ds_cache_compact(const ds_compact_args* a, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  CompactParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, 0, &p.pool);
  if (ps != DS_OK) return ps;
  if (!rows_ok(a->B, 0, a->max_pages, a->pool.page_size)) return DS_ERR_INVALID_ARG;
  const void* ptrs[] = {a->block_table, a->ref, a->table_out, a->ref_out, a->page_map, a->status};
  for (const void* q : ptrs)
    if (!aligned(q, 16)) return DS_ERR_INVALID_ARG;
  if (!aligned(a->n_used, 4)) return DS_ERR_INVALID_ARG;
  const size_t nt = (size_t)a->B * a->max_pages * 4, np = (size_t)a->pool.n_pages * 4;
  const struct { const void* p; size_t n; } in[] = {{a->block_table, nt}, {a->ref, np}},
                                            out[] = {{a->table_out, nt}, {a->ref_out, np}, {a->page_map, np},
                                                     {a->n_used, 4}};
  for (int i = 0; i < 4; ++i) {
    for (const auto& x : in)
      if (overlap(out[i].p, x.p, out[i].n, x.n)) return DS_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[j].p, out[i].n, out[j].n)) return DS_ERR_INVALID_ARG;
  }
  if (!aligned(a->workspace, 16) || a->workspace_bytes < compact_ws_bytes(a->pool.n_pages)) return DS_ERR_WORKSPACE;
  const ds_status st = device_supported();
  if (st != DS_OK) return st;
  p.B = a->B;
  p.max_pages = a->max_pages;
  p.table = a->block_table;
  p.ref = a->ref;
  p.table_out = a->table_out;
  p.ref_out = a->ref_out;
  p.page_map = a->page_map;
  p.n_used = a->n_used;
  p.ws = static_cast<int32_t*>(a->workspace);
  p.status = a->status;
  return launch_compact(p, (cudaStream_t)stream) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

}  // extern "C"
