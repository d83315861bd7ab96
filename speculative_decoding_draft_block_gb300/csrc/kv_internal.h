// Internal types of the paged cache's kernels (kv_cache.cu, kv_pages.cu,
// attn_*.cu); the contract of the entry points is in include/ds_cache.h.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/ds_cache.h"

namespace ds {

// A pool as the kernels see it: byte strides, one layer's base or all layers'.
struct PoolView {
  char* k;
  char* v;
  int64_t layer_stride, page_stride, token_stride, head_stride;  // bytes
  int32_t n_layers, n_pages, page_shift, n_kv_heads, row_bytes;  // row: head_dim elements
};

struct AppendParams {
  PoolView pool;  // k, v of the layer
  int32_t B, T, max_pages;
  const char* k_new;
  const char* v_new;
  int64_t k_token, k_head, v_token, v_head;  // byte strides
  const int32_t* q_start;
  const int32_t* block_table;
  const int32_t* kv_len;
  int32_t* status;
};

// Quotients of 0 <= n < 2^31 by a divisor d fixed on the host, 1 <= d <= 128: with
// l = ceil(log2 d) and m = ceil(2^(31 + l) / d) <= 2^32 - 1 (or 2^31 for d = 1),
// floor(n / d) = floor(n m / 2^(31 + l)) (Granlund and Montgomery, 1994).
struct Divisor {
  uint32_t m, shift;
  void set(uint32_t d) {
    uint32_t l = 0;
    while ((1u << l) < d) ++l;
    shift = 31 + l;
    m = (uint32_t)(((1ull << shift) + d - 1) / d);
  }
  __device__ __forceinline__ int quotient(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> shift); }
};

struct AttnParams {
  PoolView pool;  // k, v of the layer
  int32_t dtype, D;
  int32_t B, T, max_pages, max_q, n_heads, group;
  Divisor by_group;
  int32_t causal, window;
  float scale;
  const char* q;
  char* out;
  int64_t q_token, q_head, o_token, o_head;  // byte strides
  const int32_t* q_start;
  const int32_t* block_table;
  const int32_t* kv_len;
  float* lse;
  char* workspace;
  int32_t* status;
};

struct UpdateParams {
  PoolView pool;
  int32_t B, max_pages;
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* ref;
  const int32_t* parent;
  const int32_t* new_len;
  int32_t* table_out;
  int32_t* len_out;
  int32_t* ref_out;
  int32_t* ws;
  int32_t* status;
};

struct CompactParams {
  PoolView pool;
  int32_t B, max_pages;
  const int32_t* table;
  const int32_t* ref;
  int32_t* table_out;
  int32_t* ref_out;
  int32_t* page_map;
  int32_t* n_used;
  int32_t* ws;
  int32_t* status;
};

// A request's new rows as every kernel reads them: rows q0 .. q0 + n - 1 of T,
// row i at position kv - n + i. A malformed request has n = 0 and ok = false.
struct Request {
  int32_t q0, n, kv;
  bool ok;
};

__device__ __forceinline__ Request load_request(const int32_t* q_start, const int32_t* kv_len, int32_t b,
                                                int32_t T, int32_t max_q, int64_t cap) {
  // (past the first-level cache: a kernel may have started before the one that wrote these ended)
  Request r;
  r.q0 = __ldcg(q_start + b);
  const int32_t q1 = __ldcg(q_start + b + 1);
  r.kv = __ldcg(kv_len + b);
  r.n = q1 - r.q0;
  r.ok = r.q0 >= 0 && q1 >= r.q0 && q1 <= T && r.n <= max_q && r.kv >= 0 && (int64_t)r.kv <= cap;
  if (!r.ok) r.n = 0;
  return r;
}

// A launch that is set up while the kernel before it on the stream finishes; the
// kernel waits for that one (griddepcontrol.wait) before it touches any memory
// that another kernel may write, and only then lets its successor start: what stands
// before it on the stream is then complete. Kernels that read their inputs
// before they wait (the draft's logits and states, the confidence head's) may follow.
// So the last kernel of the attention, whose output may be such an input, lets them
// start at its end only. What earlier kernels wrote is read past the first-level cache.
template <class... A, class... B>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const B&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What a kernel needs once on each device before its first launch there (a function's
// attributes hold for the device that was current when they were set). Two threads
// may both do it.
struct Readiness {
  static constexpr int kDevices = 64;
  std::atomic<int> state[kDevices];  // 0: not yet, else 1 + the preparation's result
  template <class F>
  cudaError_t get(F prepare) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    int s = state[dev].load(std::memory_order_acquire);
    if (s == 0) {
      s = 1 + (int)prepare();
      state[dev].store(s, std::memory_order_release);
    }
    return (cudaError_t)(s - 1);
  }
};

// The attention's key tiles, and the set-up of a unit of its work in tiles (0, 2 and 3
// are slower where units of a few tiles stand beside longer ones).
constexpr int kAttnTileTc = 128, kAttnTileF32 = 64, kAttnUnitCost = 1;

// Whether the work of one block of rows, over all KV heads, can be counted in 32 bits: with
// tiles of 128 keys always (2^23 + 1 tiles, 256 heads), with tiles of 64 except for 256
// heads over 2^30 tokens.
inline bool work_fits(int32_t dtype, int64_t tokens, int32_t n_kv_heads) {
  const int64_t tile = dtype == DS_BF16 ? kAttnTileTc : kAttnTileF32;
  return ((tokens + tile - 1) / tile + kAttnUnitCost) * n_kv_heads <= (int64_t)UINT32_MAX;
}

constexpr int kMaxAttnCtas = 152;  // one per SM of the device the kernels are built for

size_t update_ws_bytes(int32_t B, int32_t n_pages);
size_t compact_ws_bytes(int32_t n_pages);
size_t attention_ws_bytes(int32_t D);

cudaError_t launch_append(const AppendParams& p, cudaStream_t s);
cudaError_t launch_update(const UpdateParams& p, cudaStream_t s);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t s);
cudaError_t launch_attention_f32(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t s);

}  // namespace ds
