// Attention of ragged rows over the paged cache on the tensor cores (bfloat16).
//
//   s_j = scale * (q . k_j),  out = sum_j 2^(c s'_j - r) v_j / l,  l = sum_j 2^(c s'_j - r),
// with s' = q . k, c = scale * log2(e), in one pass over the keys. Any reference
// r serves, since out and l carry the same factor 2^-r; it only has to keep the
// exponents in range. So r is the running maximum of c s', raised only when that
// has grown by more than kSlack = 8 (a factor of 256, harmless in float32 sums
// and in bfloat16 weights, whose precision is relative): rescaling the output
// accumulator, which sits in TMEM, then happens a few times a row, not once a tile.
//
// Work. A unit is (request, KV head, block of query rows): the G query heads of
// a KV head times its tokens are packed as rows of 128-row tiles (a tile holds
// 128 / G whole tokens), two tiles a unit at most. All units' key tiles (128
// keys each) in a row are the work list; CTA c of the grid takes the contiguous
// share [c W / g, (c + 1) W / g). Lengths are read on the device only, every
// share is equal to within one tile whatever the batch looks like, and a unit
// that is cut is joined by the second kernel from float32 partial results.
//
// A CTA works with two streams, each with its own score tile, output
// accumulator and softmax warpgroup. A unit of two row tiles gives each stream a
// row tile and both read every key tile (prompts: arithmetic bound); a unit of
// one row tile gives the streams the even and the odd key tiles and joins their
// accumulators in the epilogue (single tokens and verify blocks: the tensor
// work of the mostly empty rows stays below the time the keys take to arrive).
// While one stream's scores go through the softmax, the tensor core works on the
// other's.
//
//   warp 0      producer: TMA loads of Q tiles and of K and V tiles (one box per
//               page and 64 elements, 128B-swizzled) into a ring of kSlots
//   warp 1      MMA issuer: S = Q K^T (both in shared memory), O += P V (P in
//               TMEM over its scores, V in shared memory, MN-major)
//   warp 2      clears the V rows that no row sees in a unit's first and last
//               tile: a weight of zero does not cancel a NaN in a matrix product
//   warps 4-7, 8-11   softmax of streams 0 and 1: a thread a row
//
// TMEM (512 columns): scores 2 x 128, accumulators 2 x D. Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "kv_internal.h"
#include "sm100.cuh"

namespace ds {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kTile = 128;         // keys a tile, rows a tile
constexpr float kSlack = 8.f;      // growth of the exponents that is left in the sums
constexpr uint32_t kCtrlRegs = 72, kSoftRegs = 216, kLaunchRegs = 168;
static_assert(128 * kCtrlRegs + 256 * kSoftRegs <= kThreads * kLaunchRegs, "register split exceeds the launch pool");
constexpr uint32_t kWaitPolls = 1u << 16;
constexpr uint32_t kHeader = 3072;  // barriers and the streams' exchange, before the tiles

template <int D>
struct Layout {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 10;
  static constexpr uint32_t kOffQ = kHeader;
  static constexpr uint32_t kOffRing = kOffQ + 2 * kTileBytes;
  static constexpr uint32_t kBytes = kOffRing + kSlots * kTileBytes;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct Header {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[10], empty[10];
  uint64_t to_clear[10];         // the slot is being filled with a V tile some rows of which no row sees
  uint64_t cleared[10];          // and those have been cleared
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t x_ready, x_free;      // exchange of the streams' statistics
  uint64_t drain;
  uint32_t tmem;
  int abort_flag;
  int scan[kThreads / 32];
  int64_t scan64[kThreads / 32];
  int start_b;
  int64_t start_base, total;
  float2 stat[2][kTile];         // reference (times c) and sum of each row, per stream
};
static_assert(sizeof(Header) <= kHeader, "header");

// What the join needs to know of a cut unit: written by the CTA that starts it.
struct CutUnit {
  int64_t end, total;  // in work tiles
  int32_t valid, b, h, qt;
};

struct Partials {
  CutUnit* cut;  // [grid]
  float* stat;   // [grid][2][256][2]
  float* out;    // [grid][2][256][D]
};

template <int D>
__host__ __device__ inline Partials partials(char* ws) {
  Partials p;
  p.cut = reinterpret_cast<CutUnit*>(ws);
  p.stat = reinterpret_cast<float*>(ws + kMaxAttnCtas * 64);
  p.out = p.stat + (size_t)kMaxAttnCtas * 2 * 256 * 2;
  return p;
}
static_assert(sizeof(CutUnit) <= 64, "record");

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if ((i & 15) == 15 && *abort_flag) return false;
  }
  *abort_flag = 1;
  report(status, kErrTimeout);
  return false;
}

__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i <= kWaitPolls; ++i)
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return;
}

// ---- the work list -----------------------------------------------------------------

// A unit's tokens and key tiles.
struct Unit {
  int i0, n_tok, two;    // first token, tokens, whether it has two row tiles
  int lo, hi;            // keys that some row sees
  int tile0, tiles;      // first key tile, number (0: nothing to see)
};

__device__ __forceinline__ Unit make_unit(const AttnParams& p, const Request& r, int qt, int per_tile) {
  Unit u;
  u.i0 = qt * 2 * per_tile;
  u.n_tok = min(r.n - u.i0, 2 * per_tile);
  u.two = u.n_tok > per_tile;
  const int first = r.kv - r.n + u.i0, last = first + u.n_tok - 1;
  u.hi = p.causal ? min(last + 1, r.kv) : r.kv;
  u.lo = p.window > 0 ? max(0, first - p.window + 1) : 0;
  u.tiles = 0;
  u.tile0 = 0;
  if (u.hi > u.lo) {
    u.tile0 = u.lo / kTile;
    u.tiles = (u.hi + kTile - 1) / kTile - u.tile0;
  }
  return u;
}

__device__ __forceinline__ int64_t request_work(const AttnParams& p, const Request& r, int per_tile) {
  int64_t w = 0;
  for (int qt = 0; qt * 2 * per_tile < r.n; ++qt) w += max(1, make_unit(p, r, qt, per_tile).tiles);
  return w * p.pool.n_kv_heads;
}

// Walks over a CTA's share unit by unit; every role walks alike.
struct Walk {
  int64_t at, end, base;  // next work tile, end of the share, first work tile of (b, qt)
  int b, qt;
  Request r;
  // the piece: tiles [t0, t1) of the unit's `n` (n = 0: nothing to see)
  Unit u;
  int h, t0, t1, n;

  __device__ __forceinline__ void start(const AttnParams& p, const Header& sh, int64_t first, int64_t last) {
    at = first;
    end = last;
    base = sh.start_base;
    b = sh.start_b;
    qt = 0;
    if (at < end) r = request(p, b);
  }
  static __device__ __forceinline__ Request request(const AttnParams& p, int b) {
    return load_request(p.q_start, p.kv_len, b, p.T, p.max_q, (int64_t)p.max_pages << p.pool.page_shift);
  }
  __device__ __forceinline__ bool next(const AttnParams& p, int per_tile) {
    if (at >= end) return false;
    while (true) {
      if (qt * 2 * per_tile >= r.n) {
        ++b;
        qt = 0;
        if (b >= p.B) return false;
        r = request(p, b);
        continue;
      }
      u = make_unit(p, r, qt, per_tile);
      n = max(1, u.tiles);
      const int64_t all = (int64_t)n * p.pool.n_kv_heads;
      if (at >= base + all) {
        base += all;
        ++qt;
        continue;
      }
      h = (int)((at - base) / n);
      const int64_t u0 = base + (int64_t)h * n;
      t0 = (int)(at - u0);
      t1 = (int)min((int64_t)n, end - u0);
      at = u0 + t1;
      return true;
    }
  }
  __device__ __forceinline__ bool empty() const { return u.tiles == 0; }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }
  __device__ __forceinline__ int64_t unit_end() const { return base + (int64_t)(h + 1) * n; }
  // whether no row of the unit sees some of a tile's keys
  __device__ __forceinline__ bool partly_seen(int tile) const {
    return tile * kTile < u.lo || (tile + 1) * kTile > u.hi;
  }
  // place of a key tile's K or V in the order of the ring, counted from the piece's first
  __device__ __forceinline__ uint32_t k_place(int j) const { return u.two ? 2 * j : j == 0 ? 0 : 2 * j - 1; }
  __device__ __forceinline__ uint32_t v_place(int j) const {
    return u.two ? 2 * j + 1 : j == t1 - t0 - 1 ? 2 * j + 1 : 2 * j + 2;
  }
};

// ---- packed float32 pairs ------------------------------------------------------------

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 result columns of a row to memory, times `f`: bfloat16 output or float32 partial.
__device__ __forceinline__ void store_bf16(char* to, const float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 x;
    x.x = to_bf16x2(v[8 * i], v[8 * i + 1]);
    x.y = to_bf16x2(v[8 * i + 2], v[8 * i + 3]);
    x.z = to_bf16x2(v[8 * i + 4], v[8 * i + 5]);
    x.w = to_bf16x2(v[8 * i + 6], v[8 * i + 7]);
    reinterpret_cast<uint4*>(to)[i] = x;
  }
}
__device__ __forceinline__ void store_f32(float* to, const float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    reinterpret_cast<float4*>(to)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// ---- the kernel --------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV) {
  using L = Layout<D>;
  constexpr int kSlots = L::kSlots;
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  Header& sh = *reinterpret_cast<Header*>(smem);
  uint8_t* sQ = smem + L::kOffQ;
  uint8_t* sRing = smem + L::kOffRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per_tile = kTile / p.group;  // tokens of a row tile

  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle is taken from address bits
    if (tid == 0) report(p.status, kErrCuda);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.pv_done[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.to_clear[i], 1);
      mbar_init(&sh.cleared[i], 1);
    }
    mbar_init(&sh.x_ready, 8);
    mbar_init(&sh.x_free, 8);
    mbar_init(&sh.drain, 1);
    sh.abort_flag = 0;
    fence_barrier_init();
  }

  // the share: total work, then the request that holds the share's first tile
  int64_t mine = 0;
  for (int b = tid; b < p.B; b += kThreads) {
    const Request r = Walk::request(p, b);
    if (!r.ok && blockIdx.x == 0) report(p.status, kErrBounds);
    mine += request_work(p, r, per_tile);
  }
  int64_t sum = mine;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) sh.scan64[warp] = sum;
  __syncthreads();
  int64_t total = 0;
  for (int i = 0; i < kThreads / 32; ++i) total += sh.scan64[i];
  const int64_t w0 = total * blockIdx.x / gridDim.x, w1 = total * (blockIdx.x + 1) / gridDim.x;
  const Partials part = partials<D>(p.workspace);
  if (w0 >= w1) {
    if (tid == 0) part.cut[blockIdx.x].valid = 0;
    return;
  }
  __syncthreads();
  int64_t base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + tid;
    const int64_t w = b0 == 0 && p.B <= kThreads ? mine : b < p.B ? request_work(p, Walk::request(p, b), per_tile) : 0;
    int64_t inc = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += v;
    }
    if (lane == 31) sh.scan64[warp] = inc;
    __syncthreads();
    int64_t before = base, all = base;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += sh.scan64[i];
      all += sh.scan64[i];
    }
    const int64_t a = before + inc - w;
    if (w > 0 && a <= w0 && w0 < a + w) {
      sh.start_b = b;
      sh.start_base = a;
    }
    base = all;
    __syncthreads();
    if (w0 < base) break;
  }
  if (warp == 1) tmem_alloc(&sh.tmem, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* abort_flag = &sh.abort_flag;
  pdl_launch_dependents();

  Walk wk;
  wk.start(p, sh, w0, w1);

  if (warp < 4) {
    setmaxnreg_dec<kCtrlRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------------- producer
      const int shift = p.pool.page_shift, page_size = 1 << shift;
      const int rows = min(page_size, kTile);     // keys of a box
      const int boxes = kTile / rows;             // pages a tile
      const uint32_t box_bytes = (uint32_t)rows * 128u;
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
      }
      uint32_t rc = 0, qc = 0;
      bool ok = true;
      // page of this lane's box of a key tile, -1: no row of the unit sees it
      auto page_of = [&](int tile) {
        const int key = tile * kTile + lane * rows;
        if (lane >= boxes || key >= wk.u.hi || key + rows <= wk.u.lo) return -1;
        const int page = __ldg(p.block_table + (int64_t)wk.b * p.max_pages + (key >> shift));
        if (page >= 0 && page < p.pool.n_pages) return page;
        report(p.status, kErrBounds);
        return 0;
      };
      auto load = [&](const CUtensorMap* map, int tile, int page, bool is_v) {
        const uint32_t s = rc % kSlots;
        if (lane == 0) ok = wait_bar(&sh.empty[s], ((rc / kSlots) & 1) ^ 1, abort_flag, p.status);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) return;
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, page >= 0));
        if (lane == 0) {
          mbar_expect_tx(&sh.full[s], n * kHalves * box_bytes);
          if (is_v && wk.partly_seen(tile)) mbar_arrive(&sh.to_clear[s]);
        }
        __syncwarp();
        if (page >= 0) {
          uint8_t* dst = sRing + s * L::kTileBytes + lane * box_bytes;
          const int token = (tile * kTile + lane * rows) & (page_size - 1);
#pragma unroll
          for (int x = 0; x < kHalves; ++x)
            tma_load_4d_plain(dst + x * (kTile * 128), map, &sh.full[s], x * 64, token, wk.h, page);
        }
        ++rc;
      };
      while (ok && wk.next(p, per_tile)) {
        if (wk.empty()) continue;
        for (int s = 0; s <= wk.u.two && ok; ++s, ++qc) {
          if (lane == 0) {
            ok = wait_bar(&sh.q_empty[qc & 1], ((qc >> 1) & 1) ^ 1, abort_flag, p.status);
            if (ok) {
              mbar_expect_tx(&sh.q_full[qc & 1], (uint32_t)per_tile * p.group * D * 2);
              for (int x = 0; x < kHalves; ++x)
                tma_load_3d_plain(sQ + (qc & 1) * L::kTileBytes + x * (kTile * 128), &tmQ, &sh.q_full[qc & 1], x * 64,
                                  wk.h * p.group, wk.r.q0 + wk.u.i0 + s * per_tile);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        const int n = wk.t1 - wk.t0, first = wk.u.tile0 + wk.t0;
        if (!ok) break;
        int page = page_of(first);
        if (wk.u.two) {
          for (int j = 0; j < n && ok; ++j) {
            const int now = page;
            if (j + 1 < n) page = page_of(first + j + 1);
            load(&tmK, first + j, now, false);
            if (ok) load(&tmV, first + j, now, true);
          }
        } else {
          load(&tmK, first, page, false);
          for (int j = 0; j < n && ok; ++j) {
            const int now = page;
            if (j + 1 < n) {
              page = page_of(first + j + 1);
              load(&tmK, first + j + 1, page, false);
            }
            if (ok) load(&tmV, first + j, now, true);
          }
        }
      }
      // nothing of this CTA may be in flight when it exits (also after an abort)
      if (lane == 0) {
        for (uint32_t j = rc > kSlots ? rc - kSlots : 0; j < rc; ++j) drain_bar(&sh.full[j % kSlots], (j / kSlots) & 1);
        for (uint32_t j = qc > 2 ? qc - 2 : 0; j < qc; ++j) drain_bar(&sh.q_full[j & 1], (j >> 1) & 1);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      // (all lanes run the loop, one issues)
      constexpr uint32_t iqk = idesc_bf16(kTile, kTile, false, false);
      constexpr uint32_t ipv = idesc_bf16(kTile, D, false, true);
      constexpr uint64_t kbits = smem_desc_bits(16, 1024, 2);
      constexpr uint64_t vbits = smem_desc_bits(kTile * 128, 1024, 2);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = smem_desc(sQ, kbits), k_desc = smem_desc(sRing, kbits), v_desc = smem_desc(sRing, vbits);
      uint32_t rc = 0, qc = 0;
      uint32_t p_parity = 0, c_parity = 0;  // of the next phase of p_full[s] and cleared[slot], a bit each
      bool ok = true;
      while (ok && wk.next(p, per_tile)) {
        if (wk.empty()) continue;
        const int n = wk.t1 - wk.t0, two = wk.u.two;
        const int steps = two ? 2 * n : n;
        for (int s = 0; s <= two && ok; ++s)
          ok = wait_bar(&sh.q_full[(qc + s) & 1], ((qc + s) >> 1) & 1, abort_flag, p.status);
        tc_fence_after();
        auto qk = [&](int t) {
          const int s = t & 1, j = two ? t >> 1 : t;
          const uint32_t at = rc + wk.k_place(j), slot = __shfl_sync(0xffffffffu, at % kSlots, 0);
          if (!two || s == 0) {
            ok = wait_bar(&sh.full[slot], (at / kSlots) & 1, abort_flag, p.status);
            if (!ok) return;
            tc_fence_after();
          }
          const uint32_t qs = __shfl_sync(0xffffffffu, (qc + (two ? s : 0)) & 1, 0);
          const uint64_t a = q_desc + qs * (L::kTileBytes >> 4), b = k_desc + slot * (L::kTileBytes >> 4);
          const uint32_t d = tm + s * kTile;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              constexpr uint32_t kHalf = (kTile * 128) >> 4;
              const uint32_t off = (k >> 2) * kHalf + (k & 3) * 2;
              mma_bf16(d, a + off, b + off, iqk, k != 0);
            }
            mma_commit(&sh.s_full[s]);
            if (!two || s == 1) mma_commit(&sh.empty[slot]);
            // Q is free after the last product that reads it
            if (t + 1 == steps || (two && t + 2 == steps)) mma_commit(&sh.q_empty[qs]);
          }
          __syncwarp();
        };
        if (ok) qk(0);
        if (ok && steps > 1) qk(1);
        for (int t = 0; t < steps && ok; ++t) {
          const int s = t & 1, j = two ? t >> 1 : t;
          const uint32_t at = rc + wk.v_place(j), slot = __shfl_sync(0xffffffffu, at % kSlots, 0);
          if (!two || s == 0) {
            ok = wait_bar(&sh.full[slot], (at / kSlots) & 1, abort_flag, p.status);
            if (ok && wk.partly_seen(wk.u.tile0 + wk.t0 + j)) {
              ok = wait_bar(&sh.cleared[slot], (c_parity >> slot) & 1, abort_flag, p.status);
              c_parity ^= 1u << slot;
            }
            if (!ok) break;
          }
          ok = wait_bar(&sh.p_full[s], (p_parity >> s) & 1, abort_flag, p.status);
          if (!ok) break;
          p_parity ^= 1u << s;
          tc_fence_after();
          const uint64_t b = v_desc + slot * (L::kTileBytes >> 4);
          const uint32_t d = tm + 256 + s * D, a = tm + s * kTile;
          const uint32_t more = t >= 2;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) mma_bf16_ta(d, a + k * 8, b + k * (2048 >> 4), ipv, k != 0 ? 1u : more);
            mma_commit(&sh.pv_done[s]);
            if (!two || s == 1) mma_commit(&sh.empty[slot]);
          }
          __syncwarp();
          if (t + 2 < steps) qk(t + 2);
        }
        rc += 2 * n;
        qc += two + 1;
      }
      if (elect_one()) mma_commit(&sh.drain);
      __syncwarp();
      drain_bar(&sh.drain, 0);  // no product in flight when TMEM is freed
      __syncwarp();
    } else if (warp == 2) {
      // ---------------------------------------------------------------- unseen V rows
      // The producer says when it begins to fill a slot with such a tile: only
      // from then on does the parity of the slot's barrier mean this filling (a
      // barrier tells a phase from the next one, not from the one after), and the
      // slot is not filled again before the MMA issuer has seen `cleared`.
      uint32_t rc = 0, parity = 0;
      bool ok = true;
      while (ok && wk.next(p, per_tile)) {
        if (wk.empty()) continue;
        const int n = wk.t1 - wk.t0;
        for (int x = 0; x < 2 && ok; ++x) {  // the piece's first and last tile
          const int j = x == 0 ? 0 : n - 1;
          if (x == 1 && n == 1) break;
          const int key = (wk.u.tile0 + wk.t0 + j) * kTile;
          if (!wk.partly_seen(wk.u.tile0 + wk.t0 + j)) continue;
          const uint32_t at = rc + wk.v_place(j), slot = at % kSlots;
          ok = wait_bar(&sh.to_clear[slot], (parity >> slot) & 1, abort_flag, p.status) &&
               wait_bar(&sh.full[slot], (at / kSlots) & 1, abort_flag, p.status);
          if (!ok) break;
          parity ^= 1u << slot;
          uint8_t* tile = sRing + slot * L::kTileBytes;
          const int head = max(0, wk.u.lo - key), tail = min(kTile, wk.u.hi - key);
          for (int half = 0; half < kHalves; ++half) {
            uint4* v = reinterpret_cast<uint4*>(tile + half * (kTile * 128));
            for (int i = lane; i < head * 8; i += 32) v[i] = make_uint4(0, 0, 0, 0);
            for (int i = tail * 8 + lane; i < kTile * 8; i += 32) v[i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.cleared[slot]);
        }
        rc += 2 * n;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax, epilogue
    setmaxnreg_inc<kSoftRegs>();
    const int s = (warp >> 2) - 1;                 // stream
    const int row = (warp & 3) * 32 + lane;        // row of the tile = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + s * kTile, tO = tmem + lanes + 256;
    const float c = p.scale * kLog2eHi;
    uint32_t ns = 0, n_pv = 0, nx = 0;
    bool ok = true, owe_free = false;
    bool cut_written = false;
    while (ok && wk.next(p, per_tile)) {
      const int two = wk.u.two;
      const int i = wk.u.i0 + (two ? s * per_tile : 0) + row / p.group;
      const bool valid = row < per_tile * p.group && i < wk.r.n && (two || row / p.group < wk.u.n_tok);
      const int pos = wk.r.kv - wk.r.n + i;
      const int64_t t_out = wk.r.q0 + i;
      const int head = wk.h * p.group + row % p.group;
      // where the piece's result goes: the output, or a slot of partial results
      const bool whole = wk.whole();
      const int slot = wk.t0 > 0 ? 0 : 1;
      const int prow = (two ? s * kTile : 0) + row;
      float* pstat = part.stat + (((size_t)blockIdx.x * 2 + slot) * 256 + prow) * 2;
      float* pout = part.out + (((size_t)blockIdx.x * 2 + slot) * 256 + prow) * D;
      if (!whole && slot == 1 && warp == 4 && lane == 0) {
        CutUnit cu = {wk.unit_end(), total, 1, wk.b, wk.h, wk.qt};
        part.cut[blockIdx.x] = cu;
      }
      cut_written |= !whole && slot == 1;
      if (wk.empty()) {
        if (valid && (two || s == 0)) {
          for (int d = 0; d < D; d += 8)
            *reinterpret_cast<uint4*>(p.out + t_out * p.o_token + head * p.o_head + d * 2) = make_uint4(0, 0, 0, 0);
          if (p.lse != nullptr) p.lse[t_out * p.n_heads + head] = kNegInf;
        }
        continue;
      }
      // keys this row sees; a row that is not there sees all and is never stored
      const int hi = !valid ? INT32_MAX : p.causal ? min(pos + 1, wk.r.kv) : wk.r.kv;
      const int lo = valid && p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const bool work = __any_sync(0xffffffffu, valid);
      const int n = wk.t1 - wk.t0;
      const int steps = two ? n : (n + 1 - s) >> 1;
      float m = kNegInf, l = 0.f;  // reference (a score, before the factor c) and sum
      for (int it = 0; it < steps && ok; ++it) {
        const int key = (wk.u.tile0 + wk.t0 + (two ? it : 2 * it + s)) * kTile;
        ok = wait_bar(&sh.s_full[s], ns & 1, abort_flag, p.status);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        if (work) {
          uint32_t x[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32_issue(tS + 32 * q, x + 32 * q);
          tmem_ld_wait(x);
          reg_dep32(x + 32);
          reg_dep32(x + 64);
          reg_dep32(x + 96);
          if (__any_sync(0xffffffffu, key + kTile > hi || key < lo)) {
            const int a = lo - key, z = hi - key;
#pragma unroll
            for (int q = 0; q < 128; ++q)
              if (q < a || q >= z) x[q] = __float_as_uint(kNegInf);
          }
          float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
          for (int q = 0; q < 128; q += 8) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
              mx[w] = fmaxf(mx[w], fmaxf(__uint_as_float(x[q + 2 * w]), __uint_as_float(x[q + 2 * w + 1])));
          }
          const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          if (it == 0) {
            m = top;
          } else {
            const bool raise = (top - m) * c > kSlack;
            if (__any_sync(0xffffffffu, raise)) {
              const float f = raise ? ex2_approx((m - top) * c) : 1.f;
              if (raise) m = top;
              l *= f;
              ok = wait_bar(&sh.pv_done[s], (n_pv - 1) & 1, abort_flag, p.status);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16_issue(tO + s * D + 16 * q, o);
                tmem_ld16_wait(o);
#pragma unroll
                for (int w = 0; w < 16; ++w) o[w] = __float_as_uint(__uint_as_float(o[w]) * f);
                tmem_st16(tO + s * D + 16 * q, o);
              }
            }
          }
          const float r = m == kNegInf ? 0.f : m * c;
          const uint64_t c2 = pack2(c, c), r2 = pack2(-r, -r);
          uint64_t sum2[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
              const uint64_t e = fma2(pack2(__uint_as_float(x[32 * q + 2 * w]), __uint_as_float(x[32 * q + 2 * w + 1])), c2, r2);
              float2 f = unpack2(e);
              f.x = ex2_approx(f.x);
              f.y = ex2_approx(f.y);
              sum2[w & 1] = add2(sum2[w & 1], pack2(f.x, f.y));
              pk[w] = to_bf16x2(f.x, f.y);
            }
            tmem_st16(tS + 16 * q, pk);
          }
          const float2 sum = unpack2(add2(sum2[0], sum2[1]));
          l += sum.x + sum.y;
          tmem_st_wait();
        }
        if (it == 0 && owe_free) {
          // the other warpgroup may still read this stream's accumulator of the unit before
          ok = wait_bar(&sh.x_free, (nx - 1) & 1, abort_flag, p.status);
          owe_free = false;
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[s]);
        ++n_pv;
      }
      if (!ok) break;
      if (steps > 0) {
        ok = wait_bar(&sh.pv_done[s], (n_pv - 1) & 1, abort_flag, p.status);
        if (!ok) break;
      }
      tc_fence_after();
      const float ref = m == kNegInf ? kNegInf : m * c;
      if (two) {
        // each stream has its own rows
        const float f = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32_issue(tO + s * D + 32 * q, o);
          tmem_ld_wait(o);
          float v[32];
#pragma unroll
          for (int w = 0; w < 32; ++w) v[w] = __uint_as_float(o[w]) * f;
          if (valid) {
            if (whole)
              store_bf16(p.out + t_out * p.o_token + head * p.o_head + q * 64, v);
            else
              store_f32(pout + 32 * q, v);
          }
        }
        if (valid) {
          if (!whole)
            *reinterpret_cast<float2*>(pstat) = make_float2(ref, l);
          else if (p.lse != nullptr)
            p.lse[t_out * p.n_heads + head] = l > 0.f || l != l ? (ref + log2f(l)) * 0.693147180559945f : kNegInf;
        }
      } else {
        // the streams' results are two parts of the same rows: join them, half of
        // the columns in each warpgroup
        if (owe_free) {  // (a stream without a tile has not waited yet)
          ok = wait_bar(&sh.x_free, (nx - 1) & 1, abort_flag, p.status);
          owe_free = false;
          if (!ok) break;
        }
        sh.stat[s][row] = make_float2(ref, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.x_ready);
        ok = wait_bar(&sh.x_ready, nx & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const float2 other = sh.stat[s ^ 1][row];
        const float r0 = s == 0 ? ref : other.x, r1 = s == 0 ? other.x : ref;
        const float l0 = s == 0 ? l : other.y, l1 = s == 0 ? other.y : l;
        const float r = fmaxf(r0, r1);
        float f0 = r0 == kNegInf ? 0.f : ex2_approx(r0 - r);
        float f1 = r1 == kNegInf ? 0.f : ex2_approx(r1 - r);
        const float lsum = l0 * f0 + l1 * f1;
        if (whole) {
          const float inv = lsum > 0.f || lsum != lsum ? 1.f / lsum : 0.f;
          f0 *= inv;
          f1 *= inv;
        }
        const bool odd = n > 1;  // stream 1 has had a tile
        float v[D / 2];
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t a[16], b[16];
          tmem_ld16_issue(tO + s * (D / 2) + 16 * q, a);
          tmem_ld16_issue(tO + D + s * (D / 2) + 16 * q, b);
          tmem_ld16_wait(a);
          tmem_ld16_wait(b);
#pragma unroll
          for (int w = 0; w < 16; ++w)
            v[16 * q + w] = __uint_as_float(a[w]) * f0 + (odd ? __uint_as_float(b[w]) * f1 : 0.f);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.x_free);
        ++nx;
        owe_free = true;
        if (valid) {
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            if (whole)
              store_bf16(p.out + t_out * p.o_token + head * p.o_head + s * D + q * 64, v + 32 * q);
            else
              store_f32(pout + s * (D / 2) + 32 * q, v + 32 * q);
          }
          if (s == 0) {
            if (!whole)
              *reinterpret_cast<float2*>(pstat) = make_float2(r, lsum);
            else if (p.lse != nullptr)
              p.lse[t_out * p.n_heads + head] = lsum > 0.f || lsum != lsum ? (r + log2f(lsum)) * 0.693147180559945f : kNegInf;
          }
        }
      }
    }
    if (warp == 4 && lane == 0 && !cut_written) part.cut[blockIdx.x].valid = 0;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- join of the units that were cut -----------------------------------------------------
//
// Block (c, y): the unit that CTA c began and did not finish, rows 8 y .. 8 y + 7,
// a warp a row. Its parts are slot 1 of c and slot 0 of the CTAs after it, in
// that order, so the sums do not depend on timing.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnParams p, int grid) {
  pdl_wait();
  const Partials part = partials<D>(p.workspace);
  const int cta = blockIdx.x;
  const CutUnit cu = part.cut[cta];
  if (!cu.valid) return;
  const int lane = threadIdx.x & 31, prow = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int per_tile = kTile / p.group;
  const Request r = Walk::request(p, cu.b);
  const Unit u = make_unit(p, r, cu.qt, per_tile);
  const int row = prow & (kTile - 1), i = u.i0 + (prow / kTile) * per_tile + row / p.group;
  if (row >= per_tile * p.group || i >= u.i0 + u.n_tok || (prow >= kTile && !u.two)) return;
  int last = cta;  // the unit's last part
  while (cu.total * (last + 1) / grid < cu.end) ++last;
  auto at = [&](int k) { return ((size_t)k * 2 + (k == cta ? 1 : 0)) * 256 + prow; };
  // with less work than CTAs some have no share and have written nothing
  auto none = [&](int k) { return cu.total * k / grid == cu.total * (k + 1) / grid; };
  float m = kNegInf;
  for (int k = cta; k <= last; ++k)
    if (!none(k)) m = fmaxf(m, part.stat[at(k) * 2]);
  constexpr int N = D / 32;
  float l = 0.f, o[N];
#pragma unroll
  for (int d = 0; d < N; ++d) o[d] = 0.f;
  for (int k = cta; k <= last; ++k) {
    if (none(k)) continue;
    const float2 st = *reinterpret_cast<const float2*>(part.stat + at(k) * 2);
    const float f = st.x == kNegInf ? 0.f : ex2_approx(st.x - m);
    l += st.y * f;
    const float* v = part.out + at(k) * D + lane * N;
#pragma unroll
    for (int d = 0; d < N; ++d) o[d] = fmaf(v[d], f, o[d]);
  }
  const bool some = l > 0.f || l != l;
  const float inv = some ? 1.f / l : 0.f;
  const int head = cu.h * p.group + row % p.group;
  const int64_t t = r.q0 + i;
  uint32_t* to = reinterpret_cast<uint32_t*>(p.out + t * p.o_token + head * p.o_head) + lane * (N / 2);
#pragma unroll
  for (int d = 0; d < N / 2; ++d) to[d] = to_bf16x2(o[2 * d] * inv, o[2 * d + 1] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[t * p.n_heads + head] = some ? (m + log2f(l)) * 0.693147180559945f : kNegInf;
}

template <int D>
cudaError_t prepare_kernel() {
  cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
  if (e != cudaSuccess) return e;
  // an increase of registers that the launch pool cannot satisfy would never return
  cudaFuncAttributes a;
  e = cudaFuncGetAttributes(&a, attn_tc_kernel<D>);
  if (e != cudaSuccess) return e;
  return a.numRegs == (int)kLaunchRegs ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int D>
cudaError_t launch(const AttnParams& p, cudaStream_t s) {
  static const cudaError_t ready = prepare_kernel<D>();
  if (ready != cudaSuccess) return ready;
  CUtensorMap mq, mk, mv;
  const cuuint32_t per_tile = kTile / p.group;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.n_heads, (cuuint64_t)p.T};
    const cuuint64_t str[2] = {(cuuint64_t)p.q_head, (cuuint64_t)p.q_token};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.group, per_tile};
    if (!encode_tmap_bf16(&mq, p.q, 3, dims, str, box)) return cudaErrorInvalidValue;
  }
  {
    const int page = 1 << p.pool.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)page, (cuuint64_t)p.pool.n_kv_heads, (cuuint64_t)p.pool.n_pages};
    const cuuint64_t str[3] = {(cuuint64_t)p.pool.token_stride, (cuuint64_t)p.pool.head_stride, (cuuint64_t)p.pool.page_stride};
    const cuuint32_t box[4] = {64, (cuuint32_t)(page < kTile ? page : kTile), 1, 1};
    if (!encode_tmap_bf16(&mk, p.pool.k, 4, dims, str, box) || !encode_tmap_bf16(&mv, p.pool.v, 4, dims, str, box))
      return cudaErrorInvalidValue;
  }
  const int grid = kMaxAttnCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<D>::kBytes;
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, attn_tc_kernel<D>, p, mq, mk, mv);
  if (e != cudaSuccess) return e;
  const int tokens = p.max_q < 2 * (int)per_tile ? p.max_q : 2 * (int)per_tile;
  const int rows = tokens > (int)per_tile ? 2 * kTile : tokens * p.group;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid, (rows + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<D>, p, grid);
}

}  // namespace

size_t attention_ws_bytes(int32_t dtype, int32_t D) {
  (void)dtype;
  // per CTA a record and two partial results of 256 rows: D sums, reference and sum
  return (size_t)kMaxAttnCtas * (64 + 2 * 256 * (D + 2) * sizeof(float));
}

cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t s) {
  return p.D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace ds
