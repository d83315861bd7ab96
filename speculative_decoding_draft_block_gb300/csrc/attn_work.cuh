// The work of attention over the paged cache, cut into equal shares, and the join
// of what was cut; shared by the tensor-core and the CUDA-core kernels.
//
// A unit is (request, KV head, block of query rows), where a request's rows are
// its tokens times the G query heads of a KV head: row = token * G + head. All
// units' key tiles, one unit after the other with kUnitCost tiles' worth of
// set-up before each, are the work list; it is cut into kShares contiguous
// shares of equal length. Lengths are read on the device only. A unit that is
// cut leaves float32 partial results (sums, reference exponent, sum of weights),
// which a second kernel joins in the order of the shares, so that no result
// depends on timing.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv_internal.h"
#include "sm100.cuh"

namespace ds {
namespace {

constexpr int kUnitCost = kAttnUnitCost;  // of a unit's set-up, in key tiles

template <int kTileKeys, int kShareCount, int kPartialRows>
struct WorkForm {
  static constexpr int kKeys = kTileKeys;          // keys of a tile
  static constexpr int kShares = kShareCount;
  static constexpr int kPartRows = kPartialRows;   // rows of a slot of partial results
  // where share v begins
  static __host__ __device__ __forceinline__ int64_t begin(int64_t total, int v) {
    return (int64_t)((uint64_t)(total * v) / (uint64_t)kShares);
  }
  // whether some of a tile's keys are seen by no row of a unit that sees keys [lo, hi)
  static __device__ __forceinline__ bool partly_seen(int tile, int lo, int hi) {
    return tile * kKeys < lo || (tile + 1) * kKeys > hi;
  }
};

// A piece of a unit: `n` key tiles from `tile0` (n = 0: the rows see nothing; n < 0: no more pieces).
struct Piece {
  int b, h, n, tile0;
  int lo, hi;             // keys that some row of the unit sees
  int token, off, rows;   // the unit's rows begin at head `off` of the KV head's, of row `token` of q
  int pos, kv;            // position of that token, cached tokens
  int whole, slot;        // the piece is the unit; else its slot of partial results
  int pad[3];
};
static_assert(sizeof(Piece) == 64, "four 16-byte words");

// What the join needs to know of a cut unit: written by the share that begins it.
struct CutUnit {
  int64_t first, total;  // its first work tile, the work list's length
  int32_t n, valid;      // key tiles
  int32_t token, off, rows, h;
};
static_assert(sizeof(CutUnit) <= 64, "record");

constexpr int kMaxShares = 2 * kMaxAttnCtas;
constexpr int kRows = kMaxShares * 2 * 128;  // rows of partial results: two slots a share

struct Partials {
  CutUnit* cut;  // [shares]
  float2* stat;  // [kRows] reference and sum
  float* out;    // [kRows][D]
};

template <int D>
__host__ __device__ inline Partials partials(char* ws) {
  Partials p;
  p.cut = reinterpret_cast<CutUnit*>(ws);
  p.stat = reinterpret_cast<float2*>(ws + kMaxShares * 64);
  p.out = reinterpret_cast<float*>(p.stat + kRows);
  return p;
}

// A unit's rows and key tiles.
struct Unit {
  int token, off, rows;  // first token (of the request), row within it, rows
  int pos;               // position of the first token
  int lo, hi;            // keys that some row sees
  int tile0, n;          // first key tile, number (0: nothing to see)
};

template <class F>
__device__ __forceinline__ Unit make_unit(const AttnParams& p, const Request& r, int u, int unit_rows) {
  Unit x;
  const int row0 = u * unit_rows;
  x.rows = min(r.n * p.group - row0, unit_rows);
  x.token = p.by_group.quotient(row0);
  x.off = row0 - x.token * p.group;
  const int last = p.by_group.quotient(row0 + x.rows - 1);
  x.pos = r.kv - r.n + x.token;
  x.hi = p.causal ? min(r.kv - r.n + last + 1, r.kv) : r.kv;
  x.lo = p.window > 0 ? max(0, x.pos - p.window + 1) : 0;
  x.n = 0;
  x.tile0 = 0;
  if (x.hi > x.lo) {
    x.tile0 = (uint32_t)x.lo / F::kKeys;
    x.n = (uint32_t)(x.hi + F::kKeys - 1) / F::kKeys - x.tile0;
  }
  return x;
}

__device__ __forceinline__ Request request_of(const AttnParams& p, int b) {
  return load_request(p.q_start, p.kv_len, b, p.T, p.max_q, (int64_t)p.max_pages << p.pool.page_shift);
}

template <class F>
__device__ __forceinline__ int64_t request_work(const AttnParams& p, const Request& r, int unit_rows) {
  int64_t w = 0;
#pragma unroll 1
  for (int u = 0; u * unit_rows < r.n * p.group; ++u) w += make_unit<F>(p, r, u, unit_rows).n + kUnitCost;
  return w * p.pool.n_kv_heads;
}

// Tiles of a unit (first work tile `first`, n key tiles) that lie before work tile x.
__host__ __device__ __forceinline__ int tiles_before(int64_t x, int64_t first, int n) {
  const int64_t t = x - first - kUnitCost;
  return t <= 0 ? 0 : t >= n ? n : (int)t;
}

// Walks over a share.
template <class F>
struct Walk {
  int64_t at, end, base;  // next work tile, end of the share, first work tile of (b, u)
  int b, u;
  Request r;

  template <class S>
  __device__ __forceinline__ void start(int64_t first, int64_t last, const S& s, int list) {
    at = first;
    end = last;
    base = s.base[list];
    b = s.b[list];
    u = 0;
    r = s.r[list];
  }
  // The next piece, or one with n < 0; a unit that begins here and is cut goes to `cut` (if given).
  __device__ __forceinline__ Piece next(const AttnParams& p, int unit_rows, CutUnit* cut, int64_t total) {
    Piece x;
    x.n = -1;
#pragma unroll 1
    while (at < end) {
      if (u * unit_rows >= r.n * p.group) {
        ++b;
        u = 0;
        if (b >= p.B) break;
        r = request_of(p, b);
        continue;
      }
      const Unit y = make_unit<F>(p, r, u, unit_rows);
      // (fits: work_fits)
      const uint32_t w = y.n + kUnitCost, all = w * p.pool.n_kv_heads;
      if (at >= base + all) {
        base += all;
        ++u;
        continue;
      }
      const int h = (int)((uint32_t)(at - base) / w);
      const int64_t first = base + (int64_t)((uint32_t)h * w);
      const int t0 = tiles_before(at, first, y.n), t1 = tiles_before(end, first, y.n);
      const bool here = y.n == 0 ? at == first : t1 > t0;
      at = first + w;
      if (!here) continue;
      x.b = b;
      x.h = h;
      x.n = t1 - t0;
      x.tile0 = y.tile0 + t0;
      x.lo = y.lo;
      x.hi = y.hi;
      x.token = r.q0 + y.token;
      x.off = y.off;
      x.rows = y.rows;
      x.pos = y.pos;
      x.kv = r.kv;
      x.whole = x.n == y.n;
      x.slot = t0 > 0 ? 0 : 1;
      if (cut != nullptr && !x.whole && x.slot == 1) {
        const CutUnit c = {first, total, y.n, 1, x.token, x.off, x.rows, h};
        *cut = c;
      }
      return x;
    }
    return x;
  }
};

// Where the walks of shares v0 .. v0 + kLists - 1 begin: a request and its first work tile.
template <int kThreads, int kLists>
struct ShareStart {
  int64_t scan[kThreads / 32];
  int64_t base[kLists];
  Request r[kLists];
  int b[kLists];
};

// Fills it in (whole block, kThreads threads); the work list's length. Not
// filled in for shares that are empty. kThreads requests at a time; with no more
// of them than that, which is the rule, one pass does for sum and search.
template <class F, int kThreads, int kLists, int kMax>
__device__ __forceinline__ int64_t locate_shares(const AttnParams& p, int unit_rows, int v0,
                                                 ShareStart<kThreads, kMax>& s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t total = 0, base = 0;
  const bool once = p.B <= kThreads;
  // pass 0 sums up, pass 1 searches (both in one if `once`)
#pragma unroll 1
  for (int pass = once ? 1 : 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + tid;
      Request r;
      int64_t w = 0;
      if (b < p.B) {
        r = request_of(p, b);
        if (!r.ok && blockIdx.x == 0) report(p.status, kErrBounds);
        w = request_work<F>(p, r, unit_rows);
      }
      int64_t inc = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += v;
      }
      if (lane == 31) s.scan[warp] = inc;
      __syncthreads();
      int64_t before = base, all = base;
#pragma unroll 4
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += s.scan[i];
        all += s.scan[i];
      }
      base = all;
      if (once) total = all;
      if (pass == 1 && w > 0) {
        const int64_t a = before + inc - w;
#pragma unroll
        for (int l = 0; l < kLists; ++l) {
          const int64_t x = F::begin(total, v0 + l);
          if (a <= x && x < a + w) {
            s.b[l] = b;
            s.base[l] = a;
            s.r[l] = r;
          }
        }
      }
      __syncthreads();
    }
    if (pass == 0) {
      total = base;
      base = 0;
    }
  }
  return total;
}

__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

constexpr float kLn2 = 0.693147180559945f;

// ---- join of the units that were cut -----------------------------------------------------
//
// Block (v, y): the unit that share v begins and does not finish, rows kRowsB y ..
// kRowsB (y + 1) - 1 of its slot. Its parts are slot 1 of v and slot 0 of the shares after
// it. A slot's rows come in tiles of `tile`, of which the first `used` stand for rows.
//
// What bounds it is the chain of loads. With few parts (kAlone shares at most) a warp
// adds up its row alone; with more (one long request: up to 304 parts a row) the parts
// go round the warps, each with all of the block's rows, and the warps' sums are
// added up in their order. One token over 100,000 cached, one KV head: 26.5 us, by
// warps alone 68; prompt chunks of two row tiles of 7 requests (up to 16 parts) 61 us,
// with the round of the warps from 5 parts on 5 us more.
constexpr int kJoinThreads = 256;
constexpr int kAlone = 16;

// N floats of a row of partial results.
template <int N>
struct Floats {
  float v[N];
  __device__ __forceinline__ void load(const float* from, bool there) {
    if (N == 4) {
      const float4 w = there ? __ldcg(reinterpret_cast<const float4*>(from)) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[0] = w.x;
      v[1] = w.y;
      v[N - 2] = w.z;
      v[N - 1] = w.w;
    } else {
      const float2 w = there ? __ldcg(reinterpret_cast<const float2*>(from)) : make_float2(0.f, 0.f);
      v[0] = w.x;
      v[1] = w.y;
    }
  }
};

template <class F, int D, typename T, int kRowsB>
__global__ void __launch_bounds__(kJoinThreads, 4) attn_join_kernel(const AttnParams p, int tile, int used) {
  constexpr int kWarps = kJoinThreads / 32, N = D / 32, kRounds = (F::kShares + 31) / 32;
  static_assert((N == 2 || N == 4) && kRowsB <= kWarps && kAlone <= 32, "a warp a row, a lane a part");
  __shared__ float factor[F::kShares][kRowsB];  // of a part in a row's sums, -1: no part
  __shared__ __align__(16) float sums[kWarps][kRowsB][D];
  const Partials part = partials<D>(p.workspace);
  const int share = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int prow0 = blockIdx.y * kRowsB, prow = prow0 + warp;  // (warp < kRowsB: its row)
  const int in_tile = prow % tile, row = prow / tile * used + in_tile;
  auto at = [&](int k, int r) { return (size_t)(k * 2 + (k == share ? 1 : 0)) * F::kPartRows + r; };
  sm100::pdl_wait();
  // The record, and, before it has arrived, the row's statistics in this share and
  // the ones after it (looked at only if the record says that they have parts): with
  // few rows the next 31, with many, which have few parts as a rule, the next 3,
  // since each statistic is a sector of its own.
  constexpr int kAhead = kRowsB <= 2 ? 32 : 4;
  CutUnit cu;
  static_assert(sizeof(CutUnit) == 40, "five 8-byte words");
#pragma unroll
  for (int i = 0; i < 5; ++i)
    reinterpret_cast<long long*>(&cu)[i] = __ldcg(reinterpret_cast<const long long*>(part.cut + share) + i);
  float2 ahead = make_float2(kNegInf, 0.f);
  if (warp < kRowsB && lane < kAhead && share + lane < F::kShares) ahead = __ldcg(part.stat + at(share + lane, prow));
  if (!cu.valid || prow0 % tile >= used || prow0 / tile * used + prow0 % tile >= cu.rows) return;
  const bool here = warp < kRowsB && in_tile < used && row < cu.rows;

  // which lane has a part (share `share` + 32 i + lane; with little work some shares
  // have nothing and have written nothing), and whether there are more shares
  auto has_part = [&](int i, bool& more) {
    const int k = share + 32 * i + lane;
    const int a = k < F::kShares ? tiles_before(F::begin(cu.total, k), cu.first, cu.n) : cu.n;
    const int z = k < F::kShares ? tiles_before(F::begin(cu.total, k + 1), cu.first, cu.n) : cu.n;
    more = __shfl_sync(0xffffffffu, z, 31) < cu.n;
    return a < z;
  };
  bool more;
  const bool part0 = has_part(0, more);
  const uint32_t parts0 = __ballot_sync(0xffffffffu, part0);
  if (part0 && here && lane >= kAhead) ahead = __ldcg(part.stat + at(share + lane, prow));
  float m = part0 ? ahead.x : kNegInf, l = 0.f, x[N];  // reference, sum of weights, sums
#pragma unroll
  for (int d = 0; d < N; ++d) x[d] = 0.f;
  if (!more && parts0 >> kAlone == 0) {
    if (!here) return;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float f = !part0 || ahead.x == kNegInf ? 0.f : ex2_approx(ahead.x - m);
    if (part0) l = ahead.y * f;
    constexpr int kBatch = 4;  // parts in flight
    const float* from = part.out + lane * N;
#pragma unroll 1
    for (int q0 = 0; parts0 >> q0 != 0; q0 += kBatch) {
      Floats<N> y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) y[i].load(from + at(share + q0 + i, prow) * D, parts0 >> (q0 + i) & 1);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float fq = __shfl_sync(0xffffffffu, f, q0 + i);
#pragma unroll
        for (int d = 0; d < N; ++d) x[d] = fmaf(y[i].v[d], fq, x[d]);
      }
    }
  } else {
    constexpr int kPass = kRowsB < 4 ? kRowsB : 4, kBatch = 8 / kPass;  // rows a pass, parts in flight
    int n = 32 - __clz(parts0);         // shares from this one to the unit's last
    {
      float2 st[kRounds];
      st[0] = ahead;
      uint32_t mine = part0 && here ? 1u : 0u;  // rounds in which this lane's share has a part
#pragma unroll
      for (int i = 1; i < kRounds; ++i) {
        if (!more) continue;
        const bool has = has_part(i, more);
        const uint32_t all = __ballot_sync(0xffffffffu, has);
        if (all) n = 32 * i + 32 - __clz(all);
        if (has && here) {
          mine |= 1u << i;
          st[i] = __ldcg(part.stat + at(share + 32 * i + lane, prow));
        }
      }
#pragma unroll
      for (int i = 1; i < kRounds; ++i)
        if (mine >> i & 1) m = fmaxf(m, st[i].x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int k = 32 * i + lane;
        if (k >= n || warp >= kRowsB) continue;
        float f = -1.f;
        if (mine >> i & 1) {
          f = st[i].x == kNegInf ? 0.f : ex2_approx(st[i].x - m);
          l = fmaf(st[i].y, f, l);
        }
        factor[k][warp] = f;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int r0 = 0; r0 < kRowsB; r0 += kPass) {
      float o[kPass][N];
#pragma unroll
      for (int r = 0; r < kPass; ++r)
#pragma unroll
        for (int d = 0; d < N; ++d) o[r][d] = 0.f;
#pragma unroll 1
      for (int j0 = warp; j0 < n; j0 += kWarps * kBatch) {
        Floats<N> y[kBatch][kPass];
        float f[kBatch][kPass];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int j = j0 + kWarps * i;
          const float* from = part.out + at(share + j, prow0 + r0) * D + lane * N;
#pragma unroll
          for (int r = 0; r < kPass; ++r) {
            f[i][r] = j < n ? factor[j][r0 + r] : -1.f;
            y[i][r].load(from + r * D, !(f[i][r] < 0.f));
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
          for (int r = 0; r < kPass; ++r)
#pragma unroll
            for (int d = 0; d < N; ++d) o[r][d] = fmaf(y[i][r].v[d], f[i][r], o[r][d]);
      }
#pragma unroll
      for (int r = 0; r < kPass; ++r)
#pragma unroll
        for (int d = 0; d < N; ++d) sums[warp][r0 + r][lane * N + d] = o[r][d];
    }
    __syncthreads();
    if (!here) return;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int d = 0; d < N; ++d) x[d] += sums[w][warp][lane * N + d];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const bool some = l > 0.f || l != l;
  const float inv = some ? 1.f / l : 0.f;
  const int at_head = cu.off + row, tok = p.by_group.quotient(at_head);
  const int head = cu.h * p.group + at_head - tok * p.group;
  const int64_t t = cu.token + tok;
  char* to = p.out + t * p.o_token + head * p.o_head;
  if (sizeof(T) == 2) {
    uint32_t y[N / 2];
#pragma unroll
    for (int d = 0; d < N / 2; ++d) y[d] = to_bf16x2(x[2 * d] * inv, x[2 * d + 1] * inv);
    if (N == 4)
      reinterpret_cast<uint2*>(to)[lane] = make_uint2(y[0], y[N / 2 - 1]);
    else
      reinterpret_cast<uint32_t*>(to)[lane] = y[0];
  } else {
#pragma unroll
    for (int d = 0; d < N; ++d) reinterpret_cast<float*>(to)[lane * N + d] = x[d] * inv;
  }
  if (p.lse != nullptr && lane == 0) p.lse[t * p.n_heads + head] = some ? (m + log2f(l)) * kLn2 : kNegInf;
}

// Launch of the join for units of at most `rows` rows of a slot. With few rows two a
// block, so that the parts in flight are more: 10 rows of float32 12.7 us, with eight
// a block 15.9; with many rows blocks of two are too many.
template <class F, int D, typename T>
cudaError_t launch_join(const AttnParams& p, cudaStream_t s, int rows, int tile, int used) {
  if (rows <= 16)
    return launch_early(attn_join_kernel<F, D, T, 2>, dim3(F::kShares, (rows + 1) / 2), dim3(kJoinThreads), 0, s, p, tile,
                        used);
  return launch_early(attn_join_kernel<F, D, T, 8>, dim3(F::kShares, (rows + 7) / 8), dim3(kJoinThreads), 0, s, p, tile,
                      used);
}

}  // namespace
}  // namespace ds
