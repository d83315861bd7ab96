// The pages' bookkeeping: the next state of every request (grow, fall back,
// free, fork, copy on write) and the compaction of the pool.
//
// Both calls are two launches. The plan runs in one thread-block cluster: the
// counts and prefix sums over the pool's pages and the requests need a few
// barriers over all of the work, and a cluster's hardware barrier gives them
// without a grid-wide wait. The second launch spreads what is left (tables and
// page contents) over the whole GPU, reading the plan from the workspace.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kv_internal.h"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace ds {
namespace {

constexpr int kCluster = 8;  // portable size
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// ---- scans ------------------------------------------------------------------------

__device__ __forceinline__ int warp_inclusive(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// Exclusive prefix of v over the block; `total` the block's sum.
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int inc = warp_inclusive(v);
  __syncthreads();  // warp_sums may still be read from the call before
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  const int ws = lane < kPlanWarps ? warp_sums[lane] : 0;
  const int wi = warp_inclusive(ws);
  total = __shfl_sync(0xffffffffu, wi, 31);
  const int base = __shfl_sync(0xffffffffu, wi - ws, warp);
  return base + inc - v;
}

__device__ __forceinline__ int block_sum(int v, int* warp_sums) {
  int total;
  block_exclusive(v, warp_sums, total);
  return total;
}

// What the CTAs of the cluster count, published and summed with one barrier: the
// sums over the CTAs before this one in `before`, over all in the result.
struct Counts {
  long long a;
  int b, c;
};

__device__ __forceinline__ Counts cluster_exchange(cg::cluster_group& cl, Counts* slot, Counts mine, Counts& before) {
  if (threadIdx.x == 0) *slot = mine;
  cl.sync();
  before = Counts{0, 0, 0};
  Counts all = {0, 0, 0};
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    const Counts u = *cl.map_shared_rank(slot, r);
    if (r < (int)cl.block_rank()) {
      before.a += u.a;
      before.b += u.b;
      before.c += u.c;
    }
    all.a += u.a;
    all.b += u.b;
    all.c += u.c;
  }
  return all;
}

// Range of n items that CTA `rank` of the cluster takes, a multiple of 4 at its start.
__device__ __forceinline__ void share(int n, int rank, int& first, int& last) {
  const int per = ((n + kCluster - 1) / kCluster + 3) & ~3;
  first = min(n, rank * per);
  last = min(n, first + per);
}

// ---- update: plan ----------------------------------------------------------------------

// What the plan leaves for the second launch, and works with.
struct UpdateWs {
  int32_t* fail;       // [4]: 1 if the state does not change
  int32_t* count;      // [N] holders
  int32_t* writers;    // [N] requests that will write into the page (entries of touched pages only)
  int32_t* first;      // [N] lowest of them
  int32_t* free_list;  // [N] free pages in ascending order, as many as are given out
  int32_t* start;      // [B] place of the request's first new page in free_list
  int32_t* copy_of;    // [B] page whose tokens the request copies into its first new page, or -1
};

__host__ __device__ inline UpdateWs update_ws(int32_t* ws, int32_t B, int32_t N) {
  const int64_t n = (N + 3) & ~3, b = (B + 3) & ~3;
  UpdateWs w;
  w.fail = ws;
  w.count = ws + 4;
  w.writers = w.count + n;
  w.first = w.writers + n;
  w.free_list = w.first + n;
  w.start = w.free_list + n;
  w.copy_of = w.start + b;
  return w;
}

// One request's move, from device memory.
struct Move {
  int32_t parent, keep, kept, want, old;  // old: pages it holds now
  bool ok;
};

__device__ __forceinline__ int pages_of(int tokens, int shift) {
  return (int)(((int64_t)tokens + (1 << shift) - 1) >> shift);
}

__device__ __forceinline__ Move load_move(const UpdateParams& p, int b) {
  const int64_t cap = (int64_t)p.max_pages << p.pool.page_shift;
  Move m;
  m.parent = p.parent != nullptr ? __ldg(p.parent + b) : b;
  const int now = __ldg(p.kv_len + b), next = __ldg(p.new_len + b);
  m.ok = m.parent >= -1 && m.parent < p.B && now >= 0 && now <= cap && next >= 0 && next <= cap;
  m.keep = 0;
  if (m.ok && m.parent >= 0) {
    const int from = m.parent == b ? now : __ldg(p.kv_len + m.parent);
    m.ok = from >= 0 && from <= cap;
    m.keep = min(from, next);
  }
  m.kept = m.ok ? pages_of(m.keep, p.pool.page_shift) : 0;
  m.want = m.ok ? pages_of(next, p.pool.page_shift) : 0;
  m.old = m.ok ? pages_of(now, p.pool.page_shift) : 0;
  return m;
}

// The partly filled page that request b will write into, or -1.
__device__ __forceinline__ int written_page(const UpdateParams& p, const Move& m, int next) {
  const int mask = (1 << p.pool.page_shift) - 1;
  if ((m.keep & mask) == 0 || next <= m.keep) return -1;
  const int page = __ldg(p.table + (int64_t)m.parent * p.max_pages + m.kept - 1);
  return page >= 0 && page < p.pool.n_pages ? page : -2;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    update_plan_kernel(const UpdateParams p) {
  cg::cluster_group cl = cg::this_cluster();
  sm100::pdl_launch_dependents();
  __shared__ int sums[kPlanWarps];
  __shared__ Counts slot;
  // what the requests ask for may pass 32 bits (a length's limit is the table's,
  // not the pool's), and has to be compared with the free pages all the same
  __shared__ unsigned long long need_sum;
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = (int)cl.block_rank();
  const int N = p.pool.n_pages, B = p.B;
  const UpdateWs w = update_ws(p.ws, B, N);
  int p0, p1, b0, b1;
  share(N, rank, p0, p1);
  share(B, rank, b0, b1);

  // holders as they are; the entries of `writers` and `first` that will be used
  int bad = 0;
  for (int i = p0 + tid; i < p1; i += kPlanThreads) {
    const int r = __ldg(p.ref + i);
    bad |= r < 0;
    w.count[i] = r;
  }
  for (int b = b0 + tid; b < b1; b += kPlanThreads) {
    const Move m = load_move(p, b);
    const int page = m.ok ? written_page(p, m, __ldg(p.new_len + b)) : -1;
    bad |= !m.ok || page == -2;
    if (page >= 0) {
      w.writers[page] = 0;
      w.first[page] = INT32_MAX;
    }
  }
  cl.sync();

  // holders afterwards: a warp a request, only the entries that change
  for (int b = b0 + (tid >> 5); b < b1; b += kPlanWarps) {
    const Move m = load_move(p, b);
    if (!m.ok) continue;
    const int32_t* now = p.table + (int64_t)b * p.max_pages;
    const int32_t* past = p.table + (int64_t)max(m.parent, 0) * p.max_pages;
    const int from = m.parent == b ? m.kept : 0;
    for (int j = from + lane; j < max(m.old, m.kept); j += 32) {
      const int o = j < m.old ? __ldg(now + j) : -1;
      const int h = j < m.kept ? __ldg(past + j) : -1;
      if ((j < m.old && (o < 0 || o >= N)) || (j < m.kept && (h < 0 || h >= N))) {
        bad = 1;
      } else if (o != h) {
        if (o >= 0) atomicSub(w.count + o, 1);
        if (h >= 0) atomicAdd(w.count + h, 1);
      }
    }
    if (lane == 0) {
      const int page = written_page(p, m, __ldg(p.new_len + b));
      if (page >= 0) {
        atomicAdd(w.writers + page, 1);
        atomicMin(w.first + page, b);
      }
    }
  }
  cl.sync();

  // new pages per request and free pages, summed over the cluster
  long long need = 0;
  int free = 0;
  if (tid == 0) need_sum = 0;
  __syncthreads();
  for (int b = b0 + tid; b < b1; b += kPlanThreads) {
    const Move m = load_move(p, b);
    int copy = -1;
    if (m.ok) {
      const int page = written_page(p, m, __ldg(p.new_len + b));
      if (page >= 0) {
        const int holders = __ldcg(w.count + page);
        if (holders > 1 && !(holders == __ldcg(w.writers + page) && b == __ldcg(w.first + page))) copy = page;
      }
      need += m.want - m.kept + (copy >= 0);
    }
    w.copy_of[b] = copy;
  }
  for (int i = p0 + tid; i < p1; i += kPlanThreads) {
    const int c = __ldcg(w.count + i);
    bad |= c < 0;
    free += c == 0;
  }
  if (need > 0) atomicAdd(&need_sum, (unsigned long long)need);
  const int free_sum = block_sum(free, sums);
  const int bad_any = __syncthreads_or(bad);
  Counts before;
  const Counts all = cluster_exchange(cl, &slot, Counts{(long long)need_sum, free_sum, bad_any}, before);
  const long long need_all = all.a;
  const bool bad_all = all.c > 0, fail = bad_all || need_all > all.b;
  if (fail && rank == 0 && tid == 0) report(p.status, bad_all ? kErrBounds : kErrPages);
  if (rank == 0 && tid == 0) w.fail[0] = fail;

  // places of the requests' new pages, and the pages that are given out
  int at = fail ? 0 : (int)before.a;
  for (int base = b0; base < b1; base += kPlanThreads) {
    const int b = base + tid;
    int n = 0;
    if (b < b1) {
      const Move m = load_move(p, b);
      n = m.want - m.kept + (w.copy_of[b] >= 0);
    }
    int total;
    const int ex = block_exclusive(n, sums, total);
    if (b < b1) w.start[b] = at + ex;
    at += total;
  }
  at = before.b;
  for (int base = p0; base < p1; base += kPlanThreads) {
    const int i = base + tid;
    const int c = i < p1 ? __ldcg(w.count + i) : 1;
    int total;
    const int r = at + block_exclusive(c == 0, sums, total);
    if (i < p1) {
      if (!fail && c == 0 && r < need_all) w.free_list[r] = i;
      p.ref_out[i] = fail ? __ldg(p.ref + i) : c == 0 ? (r < need_all ? 1 : 0) : c;
    }
    at += total;
  }
  cl.sync();  // no CTA leaves while another may read its shared memory
}

// ---- update: tables and copies ------------------------------------------------------------

// Copies the first `tokens` tokens of a page of one layer of K or V. The index
// runs along memory (heads inside tokens, or tokens inside heads) over runs of
// contiguous bytes, as long as the strides allow: a whole page as a rule. A thread
// has kFlight loads in flight before it stores.
constexpr int kFlight = 4;
__device__ __forceinline__ void copy_tokens(const PoolView& v, char* base, int src, int dst, int tokens, int tid,
                                            int threads) {
  const char* from = base + (int64_t)src * v.page_stride;
  char* to = base + (int64_t)dst * v.page_stride;
  const bool heads_inside = v.head_stride <= v.token_stride;
  const int64_t s1 = heads_inside ? v.head_stride : v.token_stride, s2 = heads_inside ? v.token_stride : v.head_stride;
  int run = v.row_bytes, n1 = heads_inside ? v.n_kv_heads : tokens, n2 = heads_inside ? tokens : v.n_kv_heads;
  if (s1 == run) {
    run *= n1;
    n1 = 1;
    if (s2 == run) {
      run *= n2;
      n2 = 1;
    }
  }
  run >>= 4;
  const int n = run * n1 * n2;
  for (int x0 = tid; x0 < n; x0 += kFlight * threads) {
    uint4 y[kFlight];
    int64_t off[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int x = x0 + f * threads;
      int64_t o = (int64_t)x * 16;
      if (n1 * n2 > 1) {
        const int q = x / run, i2 = q / n1;
        o = i2 * s2 + (q - i2 * n1) * s1 + (x - q * run) * 16;
      }
      off[f] = o;
      if (x < n) y[f] = __ldcs(reinterpret_cast<const uint4*>(from + o));
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (x0 + f * threads < n) *reinterpret_cast<uint4*>(to + off[f]) = y[f];
  }
}

__global__ void __launch_bounds__(256) update_apply_kernel(const UpdateParams p) {
  sm100::pdl_wait();
  const int b = blockIdx.x, part = blockIdx.y;  // part: 2 * layer + (0: K, 1: V)
  const UpdateWs w = update_ws(p.ws, p.B, p.pool.n_pages);
  if (__ldcg(w.fail)) {
    if (part == 0) {
      for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x)
        p.table_out[(int64_t)b * p.max_pages + j] = __ldg(p.table + (int64_t)b * p.max_pages + j);
      if (threadIdx.x == 0) p.len_out[b] = __ldg(p.kv_len + b);
    }
    return;
  }
  const int copy = __ldcg(w.copy_of + b);
  if (part > 0 && copy < 0) return;
  const Move m = load_move(p, b);
  const int start = __ldcg(w.start + b), shared = m.kept - (copy >= 0);
  if (part == 0) {
    const int32_t* past = p.table + (int64_t)max(m.parent, 0) * p.max_pages;
    for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x)
      p.table_out[(int64_t)b * p.max_pages + j] =
          j < shared ? __ldg(past + j) : j < m.want ? __ldcg(w.free_list + start + j - shared) : -1;
    if (threadIdx.x == 0) {
      p.len_out[b] = __ldg(p.new_len + b);
      if (copy >= 0) atomicSub(p.ref_out + copy, 1);
    }
    if (copy < 0) return;
  }
  const int dst = __ldcg(w.free_list + start);
  char* base = (part & 1 ? p.pool.v : p.pool.k) + (int64_t)(part >> 1) * p.pool.layer_stride;
  copy_tokens(p.pool, base, copy, dst, m.keep & ((1 << p.pool.page_shift) - 1), threadIdx.x, blockDim.x);
}

// ---- compact -------------------------------------------------------------------------------

struct CompactWs {
  int32_t* moves;  // [4]: number of moves, 1 if the state does not change
  int32_t* src;    // [N / 2]
  int32_t* dst;    // [N / 2]
};

__host__ __device__ inline CompactWs compact_ws(int32_t* ws, int32_t N) {
  CompactWs w;
  w.moves = ws;
  w.src = ws + 4;
  w.dst = w.src + ((N / 2 + 4) & ~3);
  return w;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const CompactParams p) {
  cg::cluster_group cl = cg::this_cluster();
  sm100::pdl_launch_dependents();
  __shared__ int sums[kPlanWarps];
  __shared__ Counts slot[2];
  const int tid = threadIdx.x, rank = (int)cl.block_rank();
  const int N = p.pool.n_pages;
  const CompactWs w = compact_ws(p.ws, N);
  int p0, p1;
  share(N, rank, p0, p1);
  int held = 0, bad = 0;
  for (int i = p0 + tid; i < p1; i += kPlanThreads) {
    const int r = __ldg(p.ref + i);
    bad |= r < 0;
    held += r > 0;
  }
  const int held_sum = block_sum(held, sums), bad_any = __syncthreads_or(bad);
  Counts before, none;
  const Counts all = cluster_exchange(cl, &slot[0], Counts{0, held_sum, bad_any}, before);
  const int used = all.b;
  const bool fail = all.c > 0;
  int below = 0;  // held pages below `used`
  for (int i = p0 + tid; i < min(p1, used); i += kPlanThreads) below += __ldg(p.ref + i) > 0;
  const int held_below = cluster_exchange(cl, &slot[1], Counts{0, block_sum(below, sums), 0}, none).b;

  int at = before.b;
  for (int base = p0; base < p1; base += kPlanThreads) {
    const int i = base + tid;
    const int r = i < p1 ? __ldg(p.ref + i) : 0;
    int total;
    const int before = at + block_exclusive(r > 0, sums, total);  // held pages before page i
    at += total;
    if (i >= p1) continue;
    const bool moves = !fail && r > 0 && i >= used, hole = !fail && r == 0 && i < used;
    if (moves) w.src[before - held_below] = i;
    if (hole) w.dst[i - before] = i;
    p.page_map[i] = r > 0 ? i : -1;
    p.ref_out[i] = moves ? 0 : r;
  }
  cl.sync();
  const int n = fail ? 0 : used - held_below;
  for (int i = rank * kPlanThreads + tid; i < n; i += kCluster * kPlanThreads) {
    const int s = __ldcg(w.src + i), d = __ldcg(w.dst + i);
    p.page_map[s] = d;
    p.ref_out[d] = __ldg(p.ref + s);
  }
  if (rank == 0 && tid == 0) {
    w.moves[0] = n;
    w.moves[1] = fail;
    p.n_used[0] = used;
    if (fail) report(p.status, kErrBounds);
  }
  cl.sync();
}

// One block a table row or a (move, layer, K or V); the number of moves is
// known on the device only, so a fixed grid walks over them.
__global__ void __launch_bounds__(256) compact_apply_kernel(const CompactParams p) {
  sm100::pdl_wait();
  const CompactWs w = compact_ws(p.ws, p.pool.n_pages);
  const int64_t entries = (int64_t)p.B * p.max_pages;
  const bool fail = __ldcg(w.moves + 1) != 0;
  for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < entries; x += (int64_t)gridDim.x * blockDim.x) {
    const int e = __ldg(p.table + x);
    p.table_out[x] = fail ? e : e >= 0 && e < p.pool.n_pages ? __ldcg(p.page_map + e) : -1;
  }
  const int n = __ldcg(w.moves), parts = 2 * p.pool.n_layers;
  const int tokens = 1 << p.pool.page_shift;
  for (int64_t x = blockIdx.x; x < (int64_t)n * parts; x += gridDim.x) {
    const int i = (int)(x / parts), part = (int)(x - (int64_t)i * parts);
    char* base = (part & 1 ? p.pool.v : p.pool.k) + (int64_t)(part >> 1) * p.pool.layer_stride;
    copy_tokens(p.pool, base, __ldcg(w.src + i), __ldcg(w.dst + i), tokens, threadIdx.x, blockDim.x);
  }
}

}  // namespace

size_t update_ws_bytes(int32_t B, int32_t n_pages) {
  const size_t n = ((size_t)n_pages + 3) & ~(size_t)3, b = ((size_t)B + 3) & ~(size_t)3;
  return (4 + 4 * n + 2 * b) * sizeof(int32_t);
}

size_t compact_ws_bytes(int32_t n_pages) {
  return (4 + 2 * (((size_t)n_pages / 2 + 4) & ~(size_t)3)) * sizeof(int32_t);
}

// The second launch is set up while the plan runs and waits for it (what the plan
// writes is read past the first-level cache, __ldcg).
template <class P>
cudaError_t launch_apply(void (*kernel)(P), const P& p, dim3 grid, cudaStream_t s) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_update(const UpdateParams& p, cudaStream_t s) {
  update_plan_kernel<<<kCluster, kPlanThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_apply(update_apply_kernel, p, dim3(p.B, 2 * p.pool.n_layers), s);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t s) {
  compact_plan_kernel<<<kCluster, kPlanThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_apply(compact_apply_kernel, p, dim3(152 * 8), s);
}

}  // namespace ds
