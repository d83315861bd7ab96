// The pages' bookkeeping: the next state of every request (grow, fall back,
// free, fork, copy on write) and the compaction of the pool.
//
// Both calls are two launches. The plan runs in one thread-block cluster: the
// counts and prefix sums over the pool's pages and the requests need a few
// barriers over all of the work, and a cluster's hardware barrier gives them
// without a grid-wide wait. The second launch spreads what is left (tables and
// page contents) over the whole GPU, reading the plan from the workspace (past the
// first-level cache: it is set up, and may be resident, while the plan runs).
// Update of 128 requests and 16384 pages: 11.0 us (the plan alone 9.9). Compaction of
// 4 GB, half of it held (2.06 GB read and written): 320 to 328 us, 6.3 to 6.4 TB/s.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kv_internal.h"
#include "sm100.cuh"

namespace cg = cooperative_groups;

namespace ds {
namespace {

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

struct Exchange {
  Counts mine, before, all;
};

template <int kCluster>
__device__ __forceinline__ Counts cluster_exchange(cg::cluster_group& cl, Exchange* x, Counts mine, Counts& before) {
  if (threadIdx.x == 0) x->mine = mine;
  cl.sync();
  if (threadIdx.x < 32) {  // a lane a CTA (the other lanes' words are zero)
    const int r = threadIdx.x;
    Counts u = {0, 0, 0};
    if (r < kCluster) u = *cl.map_shared_rank(&x->mine, r);
    const bool lower = r < (int)cl.block_rank();
    Counts v = lower ? u : Counts{0, 0, 0};
#pragma unroll
    for (int d = kCluster / 2; d > 0; d >>= 1) {
      u.a += __shfl_xor_sync(0xffffffffu, u.a, d);
      v.a += __shfl_xor_sync(0xffffffffu, v.a, d);
    }
    u.b = __reduce_add_sync(0xffffffffu, u.b);
    u.c = __reduce_add_sync(0xffffffffu, u.c);
    v.b = __reduce_add_sync(0xffffffffu, v.b);
    v.c = __reduce_add_sync(0xffffffffu, v.c);
    if (r == 0) {
      x->all = u;
      x->before = v;
    }
  }
  __syncthreads();
  before = x->before;
  return x->all;
}

// Range of n items that CTA `rank` of the cluster takes, a multiple of 4 at its start.
template <int kCluster>
__device__ __forceinline__ void share(int n, int rank, int& first, int& last) {
  const int per = ((n + kCluster - 1) / kCluster + 3) & ~3;
  first = min(n, rank * per);
  last = min(n, first + per);
}

// ---- update: plan ----------------------------------------------------------------------

// What the plan leaves for the second launch, and works with.
struct UpdateWs {
  int32_t* fail;       // [4]: 1 if the state does not change
  int4* row;           // [B] parent, pages shared with it, pages wanted, place of the first new one in free_list
  int2* copy;          // [B] page to copy into the first new one (or -1), its tokens
  int32_t* count;      // [N] holders
  int32_t* writers;    // [N] requests that will write into the page (entries of touched pages only)
  int32_t* first;      // [N] lowest of them
  int32_t* free_list;  // [N] free pages in ascending order, as many as are given out
};

__host__ __device__ inline UpdateWs update_ws(int32_t* ws, int32_t B, int32_t N) {
  const int64_t n = (N + 3) & ~3, b = (B + 3) & ~3;
  UpdateWs w;
  w.fail = ws;
  w.row = reinterpret_cast<int4*>(ws + 4);
  w.copy = reinterpret_cast<int2*>(w.row + b);
  w.count = reinterpret_cast<int32_t*>(w.copy + b);
  w.writers = w.count + n;
  w.first = w.writers + n;
  w.free_list = w.first + n;
  return w;
}

// One request's move.
struct Move {
  int32_t parent, keep, kept, want, old;  // old: pages it holds now
  int32_t page;                           // partly filled page that it will write into, -1: none
  bool ok;
};

__device__ __forceinline__ int pages_of(int tokens, int shift) {
  return (int)(((int64_t)tokens + (1 << shift) - 1) >> shift);
}

__device__ __forceinline__ Move load_move(const UpdateParams& p, int b) {
  const int64_t cap = (int64_t)p.max_pages << p.pool.page_shift;
  Move m;
  m.parent = p.parent != nullptr ? __ldcg(p.parent + b) : b;
  const int now = __ldcg(p.kv_len + b), next = __ldcg(p.new_len + b);
  m.ok = m.parent >= -1 && m.parent < p.B && now >= 0 && now <= cap && next >= 0 && next <= cap;
  m.keep = 0;
  if (m.ok && m.parent >= 0) {
    const int from = m.parent == b ? now : __ldcg(p.kv_len + m.parent);
    m.ok = from >= 0 && from <= cap;
    m.keep = min(from, next);
  }
  m.kept = m.ok ? pages_of(m.keep, p.pool.page_shift) : 0;
  m.want = m.ok ? pages_of(next, p.pool.page_shift) : 0;
  m.old = m.ok ? pages_of(now, p.pool.page_shift) : 0;
  m.page = -1;
  if (m.ok && (m.keep & ((1 << p.pool.page_shift) - 1)) != 0 && next > m.keep) {
    m.page = __ldcg(p.table + (int64_t)m.parent * p.max_pages + m.kept - 1);
    if (m.page < 0 || m.page >= p.pool.n_pages) m.ok = false;
  }
  return m;
}

// A CTA's requests beyond the first kPlanThreads are looked up anew in each phase.
struct PlanShared {
  int sums[kPlanWarps];
  Exchange exchange;
  // what the requests ask for may pass 32 bits (a length's limit is the table's,
  // not the pool's), and has to be compared with the free pages all the same
  unsigned long long need;
  Move move[kPlanThreads];
};

// Four pages' words at once (the arrays are 16-byte aligned, i a multiple of 4).
__device__ __forceinline__ int4 load_four(const int32_t* from, int i, int end, int none) {
  if (i + 4 <= end) return __ldcg(reinterpret_cast<const int4*>(from + i));
  int4 v = make_int4(none, none, none, none);
  if (i < end) v.x = __ldcg(from + i);
  if (i + 1 < end) v.y = __ldcg(from + i + 1);
  if (i + 2 < end) v.z = __ldcg(from + i + 2);
  return v;
}
__device__ __forceinline__ void store_four(int32_t* to, int i, int end, int4 v) {
  if (i + 4 <= end) {
    *reinterpret_cast<int4*>(to + i) = v;
    return;
  }
  if (i < end) to[i] = v.x;
  if (i + 1 < end) to[i + 1] = v.y;
  if (i + 2 < end) to[i + 2] = v.z;
}

// Three phases between cluster barriers: holders as they are, holders afterwards,
// pages given out. What bounds it is the chain of dependent reads (a length, the
// parent's length, its table entry, that page's holders) at the latency of the L2,
// so a request's move is looked up once and kept in shared memory, and four pages
// go to a thread, so that a pool of 32768 pages takes one scan.
template <int kCluster>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    update_plan_kernel(const UpdateParams p) {
  cg::cluster_group cl = cg::this_cluster();
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  __shared__ PlanShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = (int)cl.block_rank();
  const int N = p.pool.n_pages, B = p.B;
  const UpdateWs w = update_ws(p.ws, B, N);
  int p0, p1, b0, b1;
  share<kCluster>(N, rank, p0, p1);
  share<kCluster>(B, rank, b0, b1);
  constexpr int kRowAhead = 16;  // entries of a row in flight a lane: 512 pages are one round trip
  auto move_of = [&](int b) { return b - b0 < kPlanThreads ? sh.move[b - b0] : load_move(p, b); };

  // holders as they are; the entries of `writers` and `first` that will be used
  int bad = 0;
  if (tid == 0) sh.need = 0;
  for (int b = b0 + tid; b < b1; b += kPlanThreads) {
    const Move m = load_move(p, b);
    if (b - b0 < kPlanThreads) sh.move[b - b0] = m;
    bad |= !m.ok;
    if (m.ok && m.page >= 0) {
      w.writers[m.page] = 0;
      w.first[m.page] = INT32_MAX;
    }
  }
  for (int i = p0 + 4 * tid; i < p1; i += 4 * kPlanThreads) {
    const int4 r = load_four(p.ref, i, p1, 0);
    bad |= (r.x | r.y | r.z | r.w) < 0;
    store_four(w.count, i, p1, r);
  }
  cl.sync();

  // holders afterwards: a warp a request, only the entries that change
  for (int b = b0 + (tid >> 5); b < b1; b += kPlanWarps) {
    const Move m = move_of(b);
    if (!m.ok) continue;
    const int32_t* now = p.table + (int64_t)b * p.max_pages;
    const int32_t* past = p.table + (int64_t)max(m.parent, 0) * p.max_pages;
    const bool same = m.parent == b;
    for (int j0 = m.kept + lane; same && j0 < m.old; j0 += 32 * kRowAhead) {
      int o[kRowAhead];
#pragma unroll
      for (int i = 0; i < kRowAhead; ++i) o[i] = j0 + 32 * i < m.old ? __ldcg(now + j0 + 32 * i) : 0;
#pragma unroll
      for (int i = 0; i < kRowAhead; ++i) {
        if (o[i] < 0 || o[i] >= N)
          bad = 1;
        else if (j0 + 32 * i < m.old)
          atomicSub(w.count + o[i], 1);
      }
    }
    const int to = same ? 0 : max(m.old, m.kept);
    constexpr int kAhead = 8;
    for (int j0 = lane; j0 < to; j0 += 32 * kAhead) {
      int o[kAhead], h[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + 32 * i;
        o[i] = j < m.old ? __ldcg(now + j) : -1;
        h[i] = j < m.kept ? __ldcg(past + j) : -1;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + 32 * i;
        if ((j < m.old && (o[i] < 0 || o[i] >= N)) || (j < m.kept && (h[i] < 0 || h[i] >= N))) {
          bad = 1;
        } else if (o[i] != h[i]) {
          if (o[i] >= 0) atomicSub(w.count + o[i], 1);
          if (h[i] >= 0) atomicAdd(w.count + h[i], 1);
        }
      }
    }
    if (lane == 0 && m.page >= 0) {
      atomicAdd(w.writers + m.page, 1);
      atomicMin(w.first + m.page, b);
    }
  }
  cl.sync();

  // Pages that a request keeps from itself: no count of theirs changes, but they have to
  // be pages. A warp a request, from the last one down, since the first ones have reads
  // of their own below. 22 requests 8.45 us without this, 8.62 with it, 9.40 with these
  // reads in the phase before; 512 beams 26.05, 26.9 and 26.5.
  for (int b = b0 + kPlanWarps - 1 - (tid >> 5); b < b1; b += kPlanWarps) {
    const Move m = move_of(b);
    const int32_t* row = p.table + (int64_t)b * p.max_pages;
    for (int j0 = lane; m.ok && m.parent == b && j0 < m.kept; j0 += 32 * kRowAhead) {
      int o[kRowAhead];
#pragma unroll
      for (int i = 0; i < kRowAhead; ++i) o[i] = j0 + 32 * i < m.kept ? __ldcg(row + j0 + 32 * i) : 0;
#pragma unroll
      for (int i = 0; i < kRowAhead; ++i) bad |= o[i] < 0 || o[i] >= N;
    }
  }

  // new pages per request and free pages, summed over the cluster
  long long need = 0;
  int free = 0;
  for (int b = b0 + tid; b < b1; b += kPlanThreads) {
    const Move m = move_of(b);
    int copy = -1;
    if (m.ok && m.page >= 0) {
      const int holders = __ldcg(w.count + m.page), writers = __ldcg(w.writers + m.page), first = __ldcg(w.first + m.page);
      if (holders > 1 && !(holders == writers && b == first)) copy = m.page;
    }
    need += m.want - m.kept + (copy >= 0);
    w.copy[b] = make_int2(copy, m.keep & ((1 << p.pool.page_shift) - 1));
    if (b - b0 < kPlanThreads) sh.move[b - b0].page = copy;
  }
  int4 counts = make_int4(1, 1, 1, 1);  // of this thread's first four pages
  for (int i = p0 + 4 * tid; i < p1; i += 4 * kPlanThreads) {
    const int4 c = load_four(w.count, i, p1, 1);
    if (i == p0 + 4 * tid) counts = c;
    bad |= (c.x | c.y | c.z | c.w) < 0;
    free += (c.x == 0) + (c.y == 0) + (c.z == 0) + (c.w == 0);
  }
  if (need > 0) atomicAdd(&sh.need, (unsigned long long)need);
  const int free_sum = block_sum(free, sh.sums);
  const int bad_any = __syncthreads_or(bad);
  Counts before;
  const Counts all = cluster_exchange<kCluster>(cl, &sh.exchange, Counts{(long long)sh.need, free_sum, bad_any}, before);
  const long long need_all = all.a;
  const bool bad_all = all.c > 0, fail = bad_all || need_all > all.b;
  if (fail && rank == 0 && tid == 0) report(p.status, bad_all ? kErrBounds : kErrPages);
  if (rank == 0 && tid == 0) w.fail[0] = fail;

  // places of the requests' new pages, and the pages that are given out
  int at = fail ? 0 : (int)before.a;
  for (int base = b0; base < b1; base += kPlanThreads) {
    const int b = base + tid;
    int shared = 0, want = 0, parent = 0;
    if (b < b1) {
      Move m = move_of(b);
      if (b - b0 >= kPlanThreads) m.page = w.copy[b].x;  // (this thread's own)
      shared = m.kept - (m.page >= 0);
      want = m.want;
      parent = m.parent;
    }
    int total;
    const int ex = block_exclusive(want - shared, sh.sums, total);
    if (b < b1) w.row[b] = make_int4(parent, shared, want, at + ex);
    at += total;
  }
  at = before.b;
  for (int base = p0; base < p1; base += 4 * kPlanThreads) {
    const int i = base + 4 * tid;
    const int4 c = base == p0 ? counts : load_four(w.count, i, p1, 1);
    int total;
    int r = at + block_exclusive((c.x == 0) + (c.y == 0) + (c.z == 0) + (c.w == 0), sh.sums, total);
    auto give = [&](int count, int page) {
      if (count != 0) return count;
      const bool given = r < need_all;
      if (!fail && given) w.free_list[r] = page;
      ++r;
      return given ? 1 : 0;
    };
    int4 out;
    out.x = give(c.x, i);
    out.y = give(c.y, i + 1);
    out.z = give(c.z, i + 2);
    out.w = give(c.w, i + 3);
    store_four(p.ref_out, i, p1, fail ? load_four(p.ref, i, p1, 0) : out);
    at += total;
  }
  cl.sync();  // no CTA leaves while another may read its shared memory
}

// ---- update: tables and copies ------------------------------------------------------------

// Copies the first `tokens` tokens of a page of one layer of K or V. The index
// runs along memory (heads inside tokens, or tokens inside heads) over runs of
// contiguous bytes, as long as the strides allow: a whole page as a rule. A thread
// has kFlight loads in flight before it stores.
constexpr int kFlight = 8;
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
  const uint4* src4 = reinterpret_cast<const uint4*>(from);
  uint4* dst4 = reinterpret_cast<uint4*>(to);
  if (n == run) {
    for (int x = tid; x < n; x += kFlight * threads) {
      uint4 y[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f)
        if (x + f * threads < n) y[f] = __ldcs(src4 + x + f * threads);
#pragma unroll
      for (int f = 0; f < kFlight; ++f)
        if (x + f * threads < n) dst4[x + f * threads] = y[f];
    }
    return;
  }
#pragma unroll 2
  for (int x = tid; x < n; x += threads) {
    const int q = x / run, i2 = q / n1;
    const int64_t o = (i2 * s2 + (q - i2 * n1) * s1) / 16 + (x - q * run);
    dst4[o] = __ldcs(src4 + o);
  }
}

// The same for the scales of a quantised pool: a head's tokens are contiguous, 16
// at a time; of the last ones of a copied page only those that are copied change.
__device__ __forceinline__ void copy_scales(const PoolView& v, int layer, int kv, int src, int dst, int tokens, int tid,
                                            int threads) {
  uint8_t* base = v.scales + layer * v.scale_layer() + kv * v.scale_part();
  const uint4* from = reinterpret_cast<const uint4*>(base + 2 * v.scale_part() * src);
  uint4* to = reinterpret_cast<uint4*>(base + 2 * v.scale_part() * dst);
  const int n = (int)(v.scale_part() >> 4), in_head = (1 << v.page_shift >> 4) - 1;
  for (int x = tid; x < n; x += threads) {
    const int left = tokens - 16 * (x & in_head);
    if (left <= 0) continue;
    uint4 y = __ldcg(from + x);
    if (left < 16) {
      const uint4 old = __ldcg(to + x);
      auto mix = [&](uint32_t a, uint32_t b, int m) { return m >= 4 ? a : m <= 0 ? b : (a & ((1u << 8 * m) - 1)) | (b & ~((1u << 8 * m) - 1)); };
      y = make_uint4(mix(y.x, old.x, left), mix(y.y, old.y, left - 4), mix(y.z, old.z, left - 8), mix(y.w, old.w, left - 12));
    }
    to[x] = y;
  }
}

__global__ void __launch_bounds__(256) update_apply_kernel(const UpdateParams p) {
  const int b = blockIdx.x;
  const UpdateWs w = update_ws(p.ws, p.B, p.pool.n_pages);
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int fail = __ldcg(w.fail);
  const int2 copy = __ldcg(w.copy + b);
  const int4 row = __ldcg(w.row + b);
  const int parent = row.x, shared = row.y, want = row.z, start = row.w;
  if (fail) {
    if (blockIdx.y == 0) {
      for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x)
        p.table_out[(int64_t)b * p.max_pages + j] = __ldcg(p.table + (int64_t)b * p.max_pages + j);
      if (threadIdx.x == 0) p.len_out[b] = __ldcg(p.kv_len + b);
    }
    return;
  }
  if (blockIdx.y == 0) {
    const int32_t* past = p.table + (int64_t)max(parent, 0) * p.max_pages;
    for (int j = threadIdx.x; j < p.max_pages; j += blockDim.x)
      p.table_out[(int64_t)b * p.max_pages + j] =
          j < shared ? __ldcg(past + j) : j < want ? __ldcg(w.free_list + start + j - shared) : -1;
    if (threadIdx.x == 0) {
      p.len_out[b] = __ldcg(p.new_len + b);
      if (copy.x >= 0) atomicSub(p.ref_out + copy.x, 1);
    }
  }
  if (copy.x < 0) return;
  const int dst = __ldcg(w.free_list + start);
  for (int part = blockIdx.y; part < 2 * p.pool.n_layers; part += gridDim.y) {  // 2 * layer + (0: K, 1: V)
    char* base = (part & 1 ? p.pool.v : p.pool.k) + (int64_t)(part >> 1) * p.pool.layer_stride;
    copy_tokens(p.pool, base, copy.x, dst, copy.y, threadIdx.x, blockDim.x);
    if (p.pool.scales != nullptr) copy_scales(p.pool, part >> 1, part & 1, copy.x, dst, copy.y, threadIdx.x, blockDim.x);
  }
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

template <int kCluster>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const CompactParams p) {
  cg::cluster_group cl = cg::this_cluster();
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  __shared__ int sums[kPlanWarps];
  __shared__ Exchange exchange[2];
  const int tid = threadIdx.x, rank = (int)cl.block_rank();
  const int N = p.pool.n_pages;
  const CompactWs w = compact_ws(p.ws, N);
  int p0, p1;
  share<kCluster>(N, rank, p0, p1);
  int held = 0, bad = 0;
  for (int i = p0 + 4 * tid; i < p1; i += 4 * kPlanThreads) {
    const int4 r = load_four(p.ref, i, p1, 0);
    bad |= (r.x | r.y | r.z | r.w) < 0;
    held += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  const int held_sum = block_sum(held, sums), bad_any = __syncthreads_or(bad);
  Counts before, none;
  const Counts all = cluster_exchange<kCluster>(cl, &exchange[0], Counts{0, held_sum, bad_any}, before);
  const int used = all.b;
  const bool fail = all.c > 0;
  int below = 0;  // held pages below `used`
  for (int i = p0 + 4 * tid; i < min(p1, used); i += 4 * kPlanThreads) {
    const int4 r = load_four(p.ref, i, min(p1, used), 0);
    below += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  const int held_below = cluster_exchange<kCluster>(cl, &exchange[1], Counts{0, block_sum(below, sums), 0}, none).b;

  int at = before.b;
  for (int base = p0; base < p1; base += 4 * kPlanThreads) {
    const int i = base + 4 * tid;
    const int4 r = load_four(p.ref, i, p1, 0);
    int total;
    // held pages before the next page
    int held_before = at + block_exclusive((r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0), sums, total);
    at += total;
    auto place = [&](int count, int page, int& map) {
      const bool moves = !fail && count > 0 && page >= used;
      if (moves) w.src[held_before - held_below] = page;
      if (!fail && count == 0 && page < used) w.dst[page - held_before] = page;
      map = count > 0 ? page : -1;
      held_before += count > 0;
      return moves ? 0 : count;
    };
    int4 map, out;
    out.x = i < p1 ? place(r.x, i, map.x) : 0;
    out.y = i + 1 < p1 ? place(r.y, i + 1, map.y) : 0;
    out.z = i + 2 < p1 ? place(r.z, i + 2, map.z) : 0;
    out.w = i + 3 < p1 ? place(r.w, i + 3, map.w) : 0;
    if (i >= p1) continue;
    store_four(p.page_map, i, p1, map);
    store_four(p.ref_out, i, p1, out);
  }
  cl.sync();
  const int n = fail ? 0 : used - held_below;
  for (int i = rank * kPlanThreads + tid; i < n; i += kCluster * kPlanThreads) {
    const int s = __ldcg(w.src + i), d = __ldcg(w.dst + i);
    p.page_map[s] = d;
    p.ref_out[d] = __ldcg(p.ref + s);
  }
  if (rank == 0 && tid == 0) {
    w.moves[0] = n;
    w.moves[1] = fail;
    p.n_used[0] = used;
    if (fail) report(p.status, kErrBounds);
  }
  cl.sync();
}

// Groups of threads take (move, layer, K or V) items; the number of moves is known on
// the device only, so a fixed grid walks over them. The table's entries go to the
// blocks from the last one down: with few moves those have nothing to copy.
// Pages smaller than what a block has in flight (32 KB) go to smaller groups: 15410
// pages of 2 KB a layer, 4 layers, 32.7 us, by whole blocks 85; 58450 of 4 KB 160 and
// 325. Three blocks an SM: left to itself the compiler takes 64 registers, which has
// four, and 4 GB take 340 us instead of 323.
__global__ void __launch_bounds__(256, 3) compact_apply_kernel(const CompactParams p) {
  const CompactWs w = compact_ws(p.ws, p.pool.n_pages);
  const int parts = 2 * p.pool.n_layers, tokens = 1 << p.pool.page_shift;
  const int64_t entries = (int64_t)p.B * p.max_pages;
  // threads of an item
  int threads = blockDim.x;
  while (threads > 32 && threads * kFlight * 16 > tokens * p.pool.n_kv_heads * p.pool.row_bytes) threads >>= 1;
  const int step = gridDim.x * (blockDim.x / threads), first = blockIdx.x + threadIdx.x / threads * gridDim.x;
  int i = first / parts, part = first % parts;  // item: move, layer and K or V
  int64_t e = (int64_t)(gridDim.x - 1 - blockIdx.x) * blockDim.x + threadIdx.x;
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  int page = e < entries ? __ldcg(p.table + e) : -1;
  const int2 moves = __ldcg(reinterpret_cast<const int2*>(w.moves));
  const int n = moves.x;
  const bool fail = moves.y != 0;
  for (; e < entries; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t next = e + (int64_t)gridDim.x * blockDim.x;
    const int now = page;
    if (next < entries) page = __ldcg(p.table + next);
    p.table_out[e] = fail ? now : now >= 0 && now < p.pool.n_pages ? __ldcg(p.page_map + now) : -1;
  }
  while (i < n) {
    char* base = (part & 1 ? p.pool.v : p.pool.k) + (int64_t)(part >> 1) * p.pool.layer_stride;
    const int src = __ldcg(w.src + i), dst = __ldcg(w.dst + i);
    copy_tokens(p.pool, base, src, dst, tokens, threadIdx.x & (threads - 1), threads);
    if (p.pool.scales != nullptr) copy_scales(p.pool, part >> 1, part & 1, src, dst, tokens, threadIdx.x & (threads - 1), threads);
    i += step / parts;
    part += step % parts;
    if (part >= parts) {
      part -= parts;
      ++i;
    }
  }
}

}  // namespace

size_t update_ws_bytes(int32_t B, int32_t n_pages) {
  const size_t n = ((size_t)n_pages + 3) & ~(size_t)3, b = ((size_t)B + 3) & ~(size_t)3;
  return (4 + 6 * b + 4 * n) * sizeof(int32_t);
}

size_t compact_ws_bytes(int32_t n_pages) {
  return (4 + 2 * (((size_t)n_pages / 2 + 4) & ~(size_t)3)) * sizeof(int32_t);
}

// Whether one CTA plans: its barriers are cheaper than a cluster's (8 is the
// portable size), its reads fewer at a time. Update of 16 requests and 1024 pages:
// 8.7 us, by a cluster 8.8; of 8 and 512: 8.5 and 8.7; of 64 and 1024: 12.6 and 9.6; of
// 128 and 4096: 17.5 and 10.1. Compaction of 512 pages: 10.0 and 10.4 us; of 2048: 14.4
// and 14.2; of 8192: 35.1 and 31.8.
bool one_cta(int32_t B, int32_t n_pages) { return n_pages <= 1024 && B <= 16; }

cudaError_t launch_update(const UpdateParams& p, cudaStream_t s) {
  const cudaError_t e = one_cta(p.B, p.pool.n_pages)
                            ? launch_early(update_plan_kernel<1>, dim3(1), dim3(kPlanThreads), 0, s, p)
                            : launch_early(update_plan_kernel<8>, dim3(8), dim3(kPlanThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  const int parts = 2 * p.pool.n_layers;  // (a grid's limit in y: 65535)
  return launch_early(update_apply_kernel, dim3(p.B, parts < 65535 ? parts : 65535), dim3(256), 0, s, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t s) {
  const cudaError_t e = one_cta(0, p.pool.n_pages)
                            ? launch_early(compact_plan_kernel<1>, dim3(1), dim3(kPlanThreads), 0, s, p)
                            : launch_early(compact_plan_kernel<8>, dim3(8), dim3(kPlanThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  return launch_early(compact_apply_kernel, dim3(152 * 8), dim3(256), 0, s, p);
}

}  // namespace ds
