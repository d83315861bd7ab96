// Trees of drafted tokens over the paged cache: the nodes' masks and depths from
// their parents, and the rows of an accepted path moved together. The contract of
// the entry points is in include/ds_cache.h.
#include "common.cuh"
#include "kv_internal.h"
#include "sm100.cuh"

namespace ds {
namespace {

// ---- masks ------------------------------------------------------------------------
//
// A node's mask is its own bit and those on the way up. A thread takes a node and
// walks up through shared memory; parents come before their children, so the
// bits fall and each word leaves once, when the walk has passed it. T (mask_words + 2)
// words are moved: bound by the launch and the chain of the walk (25 nodes 1.7 us of their
// own; 256 trees of 40 to 256, 1.2 MB, 4.0).
constexpr int kMaskThreads = 128;

__global__ void __launch_bounds__(kMaskThreads) tree_masks_kernel(const TreeParams p) {
  __shared__ int up[kMaxTree];
  const int b = blockIdx.y, tid = threadIdx.x, first = blockIdx.x * kMaskThreads;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int q0 = __ldcg(p.q_start + b), q1 = __ldcg(p.q_start + b + 1), n = q1 - q0;
  if (q0 < 0 || q1 < q0 || q1 > p.T || n > p.max_q) {
    if (first == 0 && tid == 0) report(p.status, kErrBounds);
    return;
  }
  if (first >= n) return;
  const int last = min(n, first + kMaskThreads);
  for (int i = tid; i < last; i += kMaskThreads) {
    int x = __ldcg(p.parent + q0 + i);
    if (x < -1 || x >= i) {
      report(p.status, kErrBounds);
      x = -1;
    }
    up[i] = x;
  }
  __syncthreads();
  const int i = first + tid;
  if (i >= n) return;
  uint32_t* to = p.mask + (int64_t)(q0 + i) * p.mask_words;
  int w = p.mask_words - 1, depth = 0;
  uint32_t bits = 0;
  for (int x = i; x >= 0; x = up[x], ++depth) {
    for (; w > x >> 5; --w) {
      to[w] = bits;
      bits = 0;
    }
    if (p.window == 0 || depth < p.window) bits |= 1u << (x & 31);
  }
  for (; w >= 0; --w) {
    to[w] = bits;
    bits = 0;
  }
  if (p.depth != nullptr) p.depth[q0 + i] = depth - 1;
}

// ---- an accepted path -------------------------------------------------------------
//
// Row first + path[i] goes to first + i, i = 0, 1, ...: path[i] >= i, so a row's place
// is written only after what stood there was read, as long as the rows are taken in
// order. A thread takes 16 bytes of a head's row of K or V of one layer (or its scale) and
// all rows of the path, kFlight at a time: no two threads share bytes. 2 * 2 * moved rows'
// bytes; rows that stand in their place already are left there. Bound by memory, in pieces of
// a head's row (128 trees of 8 to 60 nodes, 32 layers of 8 heads, 138 MB: 23.7 to 26.3 us, 5.2 to 5.8 TB/s),
// of few rows by the launch and the chain path, table, row (3.0 us of their own).
constexpr int kKeepThreads = 256;
constexpr int kFlight = 8;

struct Step {
  int64_t from, to;              // byte offsets in a layer
  int64_t scale_from, scale_to;  // the same of the scales
};

template <typename W, int64_t Step::*kFrom, int64_t Step::*kTo>
__device__ __forceinline__ void move_rows(char* base, const Step* step, int n) {
#pragma unroll 1
  for (int i = 0; i < n; i += kFlight) {
    W y[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (i + f < n) y[f] = __ldcg(reinterpret_cast<const W*>(base + step[i + f].*kFrom));
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (i + f < n) *reinterpret_cast<W*>(base + step[i + f].*kTo) = y[f];
  }
}

__global__ void __launch_bounds__(kKeepThreads, 4) keep_kernel(const KeepParams p) {
  __shared__ Step step[kKeepThreads];
  const int tid = threadIdx.x;
  const PoolView& v = p.pool;
  const int mask = (1 << v.page_shift) - 1, chunks = v.row_bytes >> 4;
  const int64_t rows = (int64_t)2 * v.n_layers * v.n_kv_heads, all = rows * chunks, items = all + (v.scales != nullptr ? rows : 0);
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int b = blockIdx.y;
  const int32_t* path = p.path + (int64_t)b * p.path_len;
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  const Request r = load_request(p.q_start, p.kv_len, b, p.T, p.T, (int64_t)p.max_pages << v.page_shift);
  const int first = r.kv - r.n;
  // its length, whether it can be followed, and its first row that has to move
  int m = p.path_len, stay = p.path_len;
  for (int i = tid; i < p.path_len; i += kKeepThreads) {
    const int at = __ldcg(path + i);
    if (at < 0) m = min(m, i);
    if (at != i) stay = min(stay, i);
  }
  __shared__ int least[2];
  if (tid == 0) least[0] = least[1] = p.path_len;
  __syncthreads();
  m = __reduce_min_sync(0xffffffffu, m);
  stay = __reduce_min_sync(0xffffffffu, stay);
  if ((tid & 31) == 0) {
    atomicMin(&least[0], m);
    atomicMin(&least[1], stay);
  }
  __syncthreads();
  m = least[0];
  stay = min(least[1], m);
  bool bad = !r.ok || first < 0;
  if (!bad)
    for (int i = tid; i < m; i += kKeepThreads) {
      const int at = __ldcg(path + i);
      bool wrong = at >= r.n || (i > 0 && at <= __ldcg(path + i - 1));
      if (!wrong && i >= stay) {
        const int from = __ldcg(table + ((first + at) >> v.page_shift)), to = __ldcg(table + ((first + i) >> v.page_shift));
        wrong = from < 0 || from >= v.n_pages || to < 0 || to >= v.n_pages;
      }
      bad |= wrong;
    }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0) {
    if (bad) report(p.status, kErrBounds);
    p.new_len[b] = bad ? __ldcg(p.kv_len + b) : first + m;
  }
  if (bad) return;
  for (int i0 = stay; i0 < m; i0 += kKeepThreads) {
    const int n = min(kKeepThreads, m - i0);
    if (tid < n) {
      const int src = first + __ldcg(path + i0 + tid), dst = first + i0 + tid;
      const int from = __ldcg(table + (src >> v.page_shift)), to = __ldcg(table + (dst >> v.page_shift));
      Step s;
      s.from = from * v.page_stride + (src & mask) * v.token_stride;
      s.to = to * v.page_stride + (dst & mask) * v.token_stride;
      s.scale_from = 2 * v.scale_part() * from + (src & mask);
      s.scale_to = 2 * v.scale_part() * to + (dst & mask);
      step[tid] = s;
    }
    __syncthreads();
    // a thread's bytes: those of a chunk, head, K or V and layer, or a scale's
    for (int64_t x = (int64_t)blockIdx.x * kKeepThreads + tid; x < items; x += (int64_t)gridDim.x * kKeepThreads) {
      const bool is_chunk = x < all;
      int64_t y = is_chunk ? x / chunks : x - all;
      const int c = is_chunk ? (int)(x - y * chunks) : 0;
      const int h = (int)(y % v.n_kv_heads);
      y /= v.n_kv_heads;
      const int kv = (int)(y & 1);
      const int64_t layer = y >> 1;
      if (is_chunk)
        move_rows<uint4, &Step::from, &Step::to>((kv ? v.v : v.k) + layer * v.layer_stride + h * v.head_stride + c * 16, step, n);
      else
        move_rows<uint8_t, &Step::scale_from, &Step::scale_to>(
            reinterpret_cast<char*>(v.scales) + layer * v.scale_layer() + kv * v.scale_part() + ((int64_t)h << v.page_shift),
            step, n);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_tree_masks(const TreeParams& p, cudaStream_t s) {
  return launch_early(tree_masks_kernel, dim3((p.max_q + kMaskThreads - 1) / kMaskThreads, p.B), dim3(kMaskThreads), 0, s, p);
}

cudaError_t launch_keep(const KeepParams& p, cudaStream_t s) {
  const int64_t rows = (int64_t)2 * p.pool.n_layers * p.pool.n_kv_heads;
  const int64_t items = rows * (p.pool.row_bytes >> 4) + (p.pool.scales != nullptr ? rows : 0);
  // Two waves of four blocks an SM at most, since a block begins with a chain of five loads: 23.7 us, one
  // wave 25.1, a thread for each piece of a row 28.1 in one run; bfloat16 rows 43.6, 47.8 and 49.1.
  const int64_t most = (items + kKeepThreads - 1) / kKeepThreads, waves = (8 * kMaxAttnCtas + p.B - 1) / p.B;
  const int64_t blocks = most < waves ? most : waves;
  return launch_early(keep_kernel, dim3((unsigned)blocks, p.B), dim3(kKeepThreads), 0, s, p);
}

}  // namespace ds
