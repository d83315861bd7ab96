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

// The places of rows t0 .. t0 + kTokens - 1, by the whole block: `put(i, page, token)` is
// called by thread i < kTokens, with page -1 for a row that has none.
template <int kTokens, class Put>
__device__ __forceinline__ void find_rows(const AppendParams& p, int t0, Put put) {
  static_assert(kTokens <= 32, "a lane a row");
  __shared__ int ends[kTokens];
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
    int page = -1, token = 0;
    if (t < p.T && b < p.B) {
      const int64_t cap = (int64_t)p.max_pages << p.pool.page_shift;
      const Request r = load_request(p.q_start, p.kv_len, b, p.T, p.T, cap);
      const int i = t - r.q0, pos = r.kv - r.n + i;
      if (!r.ok) {
        report(p.status, kErrBounds);
      } else if (i >= 0 && i < r.n && pos >= 0) {
        page = __ldcg(p.block_table + (int64_t)b * p.max_pages + (pos >> p.pool.page_shift));
        token = pos & ((1 << p.pool.page_shift) - 1);
        if (page < 0 || page >= p.pool.n_pages) {
          report(p.status, kErrBounds);
          page = -1;
        }
      }
    }
    put(tid, page, token);
  }
  __syncthreads();
}

// kTokens rows a block: see launch_append.
template <int kTokens>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  __shared__ int64_t at[kTokens];  // byte offset of the row's place in the pool, -1: none
  const int t0 = blockIdx.x * kTokens;
  const int tid = threadIdx.x;
  find_rows<kTokens>(p, t0, [&](int i, int page, int token) {
    at[i] = page < 0 ? -1 : (int64_t)page * p.pool.page_stride + (int64_t)token * p.pool.token_stride;
  });
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

// ---- append to a quantised pool ------------------------------------------------------
//
// A head's row x (bfloat16) becomes codes e4m3(x / 2^e) and the byte e + 127, with
// the smallest e >= -100 such that max |x| <= 448 * 2^e. 448 = 1.75 * 2^8: with max |x| =
// 2^E (1 + m / 128), 0 <= m < 128, that is e = E - 8, one more if m > 96: the largest
// value's bits decide, and their order is that of the values'. x / 2^e is exact in
// float32 (or below half of the smallest code), so the conversion's rounding is
// the only one. Powers of two cost the format at most one of its 17 binades and no
// precision, and let the attention restore a row exactly in bfloat16.
//
// 2 T Hk D (2 + 1) bytes are moved: bound by memory (16 prompts of 8 heads of 128 values, 347 MB,
// 56 us: 6.2 TB/s; with the loop over lanes not unrolled, 60), of few rows by the launch (64: 3.5 us of
// their own). A lane takes 16 values of K and of V, the power of two of lanes that D / 16 asks
// for a row's maximum.
constexpr int kLowestScale = 27, kNoScale = 255;  // bytes: e = -100; a row that is not finite

// The scale byte of a row whose largest |x| has these bits.
__device__ __forceinline__ int scale_of(uint32_t top) {
  if (top >= 0x7f80u) return kNoScale;
  return max(kLowestScale, (int)(top >> 7) - 8 + ((top & 0x7fu) > 96u ? 1 : 0));
}

// Four codes of the values (two pairs of bfloat16) times f.
__device__ __forceinline__ uint32_t codes_of(uint32_t a, uint32_t b, float f) {
  uint16_t lo, hi;
  const float a0 = __uint_as_float(a << 16) * f, a1 = __uint_as_float(a & 0xffff0000u) * f;
  const float b0 = __uint_as_float(b << 16) * f, b1 = __uint_as_float(b & 0xffff0000u) * f;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a1), "f"(a0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b1), "f"(b0));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

__device__ __forceinline__ uint32_t top_of(uint4 a, uint4 b) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t m = __vmaxu2(__vmaxu2(a.x & kAbs, a.y & kAbs), __vmaxu2(a.z & kAbs, a.w & kAbs));
  m = __vmaxu2(m, __vmaxu2(__vmaxu2(b.x & kAbs, b.y & kAbs), __vmaxu2(b.z & kAbs, b.w & kAbs)));
  return max(m & 0xffffu, m >> 16);
}

__device__ __forceinline__ uint4 quantise(uint4 a, uint4 b, int scale) {
  if (scale == kNoScale) return make_uint4(0, 0, 0, 0);
  const float f = __uint_as_float((uint32_t)(254 - scale) << 23);  // 2^-e
  return make_uint4(codes_of(a.x, a.y, f), codes_of(a.z, a.w, f), codes_of(b.x, b.y, f), codes_of(b.z, b.w, f));
}

template <int kTokens>
__global__ void __launch_bounds__(kAppendThreads) append_e4m3_kernel(const AppendParams p) {
  __shared__ int2 at[kTokens];  // a row's page (-1: none) and place in it
  const int t0 = blockIdx.x * kTokens;
  find_rows<kTokens>(p, t0, [&](int i, int page, int token) { at[i] = make_int2(page, token); });
  const int pieces = p.pool.row_bytes >> 4;  // of 16 values, 1..16
  const int shift = pieces == 1 ? 0 : 32 - __clz(pieces - 1), lanes = 1 << shift;
  const int lane = threadIdx.x & 31, c = lane & (lanes - 1);
  const int total = kTokens * p.pool.n_kv_heads << shift;
#pragma unroll 1
  for (int x0 = threadIdx.x - lane; x0 < total; x0 += kAppendThreads) {
    const int y = (x0 + lane) >> shift, i = y / p.pool.n_kv_heads, h = y - i * p.pool.n_kv_heads;
    const int2 place = i < kTokens ? at[i] : make_int2(-1, 0);
    const bool here = place.x >= 0 && c < pieces;
    uint4 k[2], v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      k[j] = v[j] = make_uint4(0, 0, 0, 0);
      if (here) {
        const int64_t t = t0 + i;
        k[j] = __ldcg(reinterpret_cast<const uint4*>(p.k_new + t * p.k_token + h * p.k_head) + 2 * c + j);
        v[j] = __ldcg(reinterpret_cast<const uint4*>(p.v_new + t * p.v_token + h * p.v_head) + 2 * c + j);
      }
    }
    uint32_t top = top_of(k[0], k[1]) | top_of(v[0], v[1]) << 16;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1)
      if (d < lanes) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (!here) continue;
    const int sk = scale_of(top & 0xffffu), sv = scale_of(top >> 16);
    const int64_t o = (int64_t)place.x * p.pool.page_stride + (int64_t)place.y * p.pool.token_stride + h * p.pool.head_stride;
    reinterpret_cast<uint4*>(p.pool.k + o)[c] = quantise(k[0], k[1], sk);
    reinterpret_cast<uint4*>(p.pool.v + o)[c] = quantise(v[0], v[1], sv);
    if (c == 0) {
      uint8_t* to = p.pool.scales + 2 * p.pool.scale_part() * place.x + ((int64_t)h << p.pool.page_shift) + place.y;
      to[0] = (uint8_t)sk;
      to[p.pool.scale_part()] = (uint8_t)sv;
    }
  }
}

// ---- argument checks --------------------------------------------------------------

bool aligned(const void* p, unsigned a) { return p != nullptr && ((uintptr_t)p & (a - 1)) == 0; }

int esize(int32_t dtype) { return dtype == DS_E4M3 ? 1 : dtype == DS_BF16 ? 2 : 4; }

// Type of the rows outside the cache.
int32_t rows_dtype(int32_t dtype) { return dtype == DS_E4M3 ? (int32_t)DS_BF16 : dtype; }

bool strides16(std::initializer_list<int64_t> strides, int32_t dtype) {
  for (int64_t s : strides)
    if (s <= 0 || (s * esize(dtype)) % 16 != 0) return false;
  return true;
}

// The pool's fields, and its view with `layer` as base (all layers: layer 0). A quantised
// pool has scales, the others none.
ds_status check_pool(const ds_kv_pool& a, int32_t layer, const uint8_t* scales, PoolView* v) {
  if (scales == nullptr ? a.dtype != DS_F32 && a.dtype != DS_BF16 : a.dtype != DS_E4M3 || !aligned(scales, 16))
    return DS_ERR_INVALID_ARG;
  if (a.n_layers < 1 || a.n_layers > (1 << 28) || a.n_pages < 1 || a.n_pages > (1 << 28) || layer < 0 ||
      layer >= a.n_layers)
    return DS_ERR_INVALID_ARG;
  if (a.page_size < 16 || a.page_size > 256 || (a.page_size & (a.page_size - 1)) != 0) return DS_ERR_INVALID_ARG;
  if (a.n_kv_heads < 1 || a.n_kv_heads > kMaxKvHeads) return DS_ERR_INVALID_ARG;
  if (a.head_dim < 8 || a.head_dim > 256 || a.head_dim % (scales != nullptr ? 16 : 8) != 0) return DS_ERR_INVALID_ARG;
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
  v->scales = scales == nullptr ? nullptr : const_cast<uint8_t*>(scales) + layer * v->scale_layer();
  return DS_OK;
}

// Requests, rows and table of a call over ragged rows. Positions are 32-bit.
bool rows_ok(int32_t B, int32_t T, int32_t max_pages, int32_t page_size) {
  return B >= 1 && B <= 65535 && T >= 0 && T <= (1 << 23) && max_pages >= 1 && (int64_t)max_pages * page_size <= kMaxTableTokens;
}

// Words of a tree's masks for requests of up to max_q tokens.
bool mask_words_ok(int32_t words, int32_t max_q) { return words >= 1 && words <= (1 << 18) && words >= (max_q + 31) / 32; }

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
  // of 512 bytes 22.0 and 23.1; of 1 KB 39.3 and 38.4; of 2 KB 74.4 and 71.8. Codes, whose
  // pieces take two loads and a conversion, of 128 bytes 9.8 by 32, 18.0 by 8; of 512 29.4 and
  // 33.1; of 1 KB 56.8 and 56.0, and 64 rows of them 7.7 and 7.1; of 2 KB 115 and 105.
  const int tokens = pieces >= 64 ? 8 : 32;
  const dim3 blocks((p.T + tokens - 1) / tokens);
  if (p.pool.scales != nullptr)
    return launch_early(tokens == 8 ? append_e4m3_kernel<8> : append_e4m3_kernel<32>, blocks, dim3(kAppendThreads), 0, s, p);
  return launch_early(tokens == 8 ? append_kernel<8> : append_kernel<32>, blocks, dim3(kAppendThreads), 0, s, p);
}

}  // namespace ds

using namespace ds;

extern "C" {

ds_status ds_cache_append(const ds_append_args* a, ds_stream_t stream) { return ds_cache_append_scaled(a, nullptr, stream); }

ds_status ds_cache_append_scaled(const ds_append_args* a, uint8_t* scales, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  AppendParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, a->layer, scales, &p.pool);
  if (ps != DS_OK) return ps;
  if (!rows_ok(a->B, a->T, a->max_pages, a->pool.page_size)) return DS_ERR_INVALID_ARG;
  const void* ptrs[] = {a->q_start, a->block_table, a->kv_len, a->status};
  for (const void* q : ptrs)
    if (!aligned(q, 16)) return DS_ERR_INVALID_ARG;
  if (a->T == 0) return DS_OK;
  if (!aligned(a->k_new, 16) || !aligned(a->v_new, 16)) return DS_ERR_INVALID_ARG;
  const int32_t rows = rows_dtype(a->pool.dtype);
  if (!strides16({a->k_token_stride, a->k_head_stride, a->v_token_stride, a->v_head_stride}, rows))
    return DS_ERR_INVALID_ARG;
  const ds_status st = device_supported();
  if (st != DS_OK) return st;
  const int64_t e = esize(rows);
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
  if ((dtype != DS_F32 && dtype != DS_BF16 && dtype != DS_E4M3) || (head_dim != 64 && head_dim != 128)) return 0;
  return attention_ws_bytes(head_dim);
}

ds_status ds_paged_attention(const ds_attention_args* a, ds_stream_t stream) {
  return ds_paged_attention_tree(a, nullptr, nullptr, stream);
}

ds_status ds_paged_attention_tree(const ds_attention_args* a, const uint8_t* scales, const ds_tree* tree,
                                  ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, a->layer, scales, &p.pool);
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
  const int32_t max_q = a->max_q < a->T ? a->max_q : a->T;
  if (tree != nullptr && (a->causal != 1 || !mask_words_ok(tree->mask_words, max_q))) return DS_ERR_INVALID_ARG;
  if (a->T == 0) return DS_OK;
  if (!aligned(a->q, 16) || !aligned(a->out, 16)) return DS_ERR_INVALID_ARG;
  if (tree != nullptr && (!aligned(tree->mask, 4) || (tree->depth != nullptr && !aligned(tree->depth, 4))))
    return DS_ERR_INVALID_ARG;
  const int32_t rows = rows_dtype(a->pool.dtype);
  if (!strides16({a->q_token_stride, a->q_head_stride, a->out_token_stride, a->out_head_stride}, rows))
    return DS_ERR_INVALID_ARG;
  const ds_status st = device_supported();
  if (st != DS_OK) return st;
  const int64_t e = esize(rows);
  p.dtype = a->pool.dtype;
  p.D = a->pool.head_dim;
  p.B = a->B;
  p.T = a->T;
  p.max_pages = a->max_pages;
  p.max_q = max_q;
  p.n_heads = a->n_heads;
  p.group = a->n_heads / a->pool.n_kv_heads;
  p.by_group.set((uint32_t)p.group);
  p.causal = a->causal;
  // a window as long as the table hides nothing (but of a tree's depths, which may be larger)
  const bool deep = tree != nullptr && tree->depth != nullptr;
  constexpr int32_t kLongest = INT32_MAX - (1 << 24);  // past any position and depth (2^30, 2^29), without overflow
  p.window = !deep && (int64_t)a->window >= (int64_t)a->max_pages * a->pool.page_size ? 0
             : a->window < kLongest                                                   ? a->window
                                                                                      : kLongest;
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
  if (tree != nullptr) {
    p.mask = tree->mask;
    p.mask_words = tree->mask_words;
    p.depth = p.window > 0 ? tree->depth : nullptr;
  }
  const cudaStream_t to = (cudaStream_t)stream;
  const cudaError_t err = p.dtype == DS_F32        ? launch_attention_f32(p, to)
                          : p.dtype == DS_E4M3     ? launch_attention_tc_e4m3(p, to)
                          : tree != nullptr        ? launch_attention_tc_tree(p, to)
                                                   : launch_attention_tc(p, to);
  return err == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

size_t ds_cache_update_workspace_bytes(int32_t B, int32_t n_pages) {
  if (B < 1 || B > 65535 || n_pages < 1) return 0;
  return update_ws_bytes(B, n_pages);
}

ds_status ds_cache_update(const ds_update_args* a, ds_stream_t stream) { return ds_cache_update_scaled(a, nullptr, stream); }

ds_status ds_cache_update_scaled(const ds_update_args* a, uint8_t* scales, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  UpdateParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, 0, scales, &p.pool);
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

ds_status ds_cache_compact(const ds_compact_args* a, ds_stream_t stream) { return ds_cache_compact_scaled(a, nullptr, stream); }

ds_status ds_cache_compact_scaled(const ds_compact_args* a, uint8_t* scales, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  CompactParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, 0, scales, &p.pool);
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

ds_status ds_tree_masks(const ds_tree_args* a, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  if (a->B < 1 || a->B > 65535 || a->T < 0 || a->T > (1 << 23) || a->max_q < 1 || a->max_q > kMaxTree || a->window < 0)
    return DS_ERR_INVALID_ARG;
  const int32_t max_q = a->max_q < a->T ? a->max_q : a->T;
  if (!mask_words_ok(a->mask_words, max_q)) return DS_ERR_INVALID_ARG;
  if (!aligned(a->q_start, 16) || !aligned(a->status, 16)) return DS_ERR_INVALID_ARG;
  if (a->T == 0) return DS_OK;
  if (!aligned(a->parent, 4) || !aligned(a->mask, 4) || (a->depth != nullptr && !aligned(a->depth, 4)))
    return DS_ERR_INVALID_ARG;
  const size_t nt = (size_t)a->T * 4, nm = nt * a->mask_words, nb = ((size_t)a->B + 1) * 4;
  const struct { const void* p; size_t n; } in[] = {{a->parent, nt}, {a->q_start, nb}};
  for (const auto& x : in)
    if (overlap(a->mask, x.p, nm, x.n) || (a->depth != nullptr && overlap(a->depth, x.p, nt, x.n))) return DS_ERR_INVALID_ARG;
  if (a->depth != nullptr && overlap(a->mask, a->depth, nm, nt)) return DS_ERR_INVALID_ARG;
  const ds_status st = device_supported();
  if (st != DS_OK) return st;
  TreeParams p;
  p.B = a->B;
  p.T = a->T;
  p.max_q = max_q;
  p.mask_words = a->mask_words;
  p.window = a->window;
  p.parent = a->parent;
  p.q_start = a->q_start;
  p.mask = a->mask;
  p.depth = a->depth;
  p.status = a->status;
  return launch_tree_masks(p, (cudaStream_t)stream) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

ds_status ds_cache_keep(const ds_keep_args* a, ds_stream_t stream) {
  if (a == nullptr) return DS_ERR_INVALID_ARG;
  KeepParams p;
  memset(&p, 0, sizeof(p));
  const ds_status ps = check_pool(a->pool, 0, a->scales, &p.pool);
  if (ps != DS_OK) return ps;
  if (!rows_ok(a->B, a->T, a->max_pages, a->pool.page_size) || a->path_len < 1 || a->path_len > kMaxTree)
    return DS_ERR_INVALID_ARG;
  const void* ptrs[] = {a->path, a->q_start, a->block_table, a->kv_len, a->new_len, a->status};
  for (const void* q : ptrs)
    if (!aligned(q, 16)) return DS_ERR_INVALID_ARG;
  const size_t nb = (size_t)a->B * 4;
  const struct { const void* p; size_t n; } in[] = {{a->path, nb * a->path_len}, {a->q_start, nb + 4},
                                                    {a->block_table, nb * a->max_pages}, {a->kv_len, nb}};
  for (const auto& x : in)
    if (overlap(a->new_len, x.p, nb, x.n)) return DS_ERR_INVALID_ARG;
  const ds_status st = device_supported();
  if (st != DS_OK) return st;
  p.B = a->B;
  p.T = a->T;
  p.max_pages = a->max_pages;
  p.path_len = a->path_len;
  p.path = a->path;
  p.q_start = a->q_start;
  p.table = a->block_table;
  p.kv_len = a->kv_len;
  p.new_len = a->new_len;
  p.status = a->status;
  return launch_keep(p, (cudaStream_t)stream) == cudaSuccess ? DS_OK : DS_ERR_CUDA;
}

}  // extern "C"
