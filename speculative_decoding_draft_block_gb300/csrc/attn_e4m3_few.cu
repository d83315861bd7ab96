// Attention of few rows (up to 16 a KV head: single tokens, short blocks and trees) over a
// quantised cache.
//
//   s_j = scale * 2^k_j (q . K_j),  out = sum_j 2^(e_j + v_j - r') V_j 2^(r' - r) / l,
//   l = sum_j 2^(e_j - r),  e_j = s_j log2(e),
// with codes K_j, V_j and their rows' powers of two k_j, v_j (exponents). Bound by the
// codes' way from memory, half of bfloat16's, so what is done to a code decides: a
// tile restored in shared memory, as for more rows (attn_tc.cuh), costs a write of 2 and
// reads of 1 and 2 bytes a code there, more than the time that its byte takes from memory.
// Here codes go from shared memory to registers once, two of them become a pair of
// float16 by one conversion, exactly, and these are the operands of register products
// (mma.sync, with 8 rows of q as columns: 128 a tile's rows of keys would be a waste of
// tcgen05, whose operands come from shared memory). Nothing is multiplied by a code's scale:
//   - k_j multiplies a score,
//   - v_j joins the exponent of the weight. Weights are rounded to float16 (11 bits) with a
//     reference r' of their own, max(e_j + v_j) - 12 at least and never more than 15.5
//     below: they keep 8 bits down to 2^-28 of the largest term of a row and vanish
//     at 2^-37, far below what rounding the values to 4 bits has left of them.
//   - q in float16 has a row's largest value in [2^14, 2^15): its values keep
//     bfloat16's 8 bits down to 2^-31 of that.
//
// Units, shares and the join are those of attn_work.cuh, for groups of KH KV heads (the query
// heads of a group count as those of one KV head; a tile has 128 / KH keys of each): with
// tokens outside heads, a head's row of codes is 128 bytes, and memory gives those at 5.1
// TB/s one head at a time (128 requests of 4000 cached), neighbours together at 6.0, as heads
// outside tokens.
// Two blocks an SM. One warp walks over the share, one loads tiles (codes
// swizzled, a box a page, scales beside them) into a ring. Each of the other
// four takes 32 keys of every tile of one head, with references, sums
// and outputs of its own. References are raised when a lane finds that one has to be (a vote
// a tile), so no maxima go over lanes otherwise. At a piece's end a warp puts its outputs where
// its last keys' codes were, and a head's warps add them up; the next piece's q
// is on its way meanwhile.
//
// Products of a warp (m16n8k16), keys or dimensions down, rows of q across:
//   S^T[16 keys][8 rows] = K[16][D] Q^T: lane 4 g + t holds D / 4 consecutive codes of keys g and
//     g + 8, and the same columns of row g of q: the sum's order does not matter.
//   O^T[D][8 rows] += V^T P^T: the lane holds D / 8 consecutive codes of keys 2 t, 2 t + 1,
//     2 t + 8, 2 t + 9; pairs of keys are made by byte permutes. P^T comes from S^T's
//     place by a transposition of 8 x 8 pairs.
// Rows that see a NaN (a scale of 255) get it by their own weights only.
#include <cuda.h>
#include <float.h>

#include "attn_work.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace ds {
namespace {

using namespace sm100;

constexpr int kTile = kAttnTileTc;               // keys of a tile, over the heads of a group
constexpr int kAhead = 4;                        // pieces handed out ahead
constexpr float kTop = 15.5f, kRaised = 12.f;    // largest exponent of a weight, and after a raise
constexpr float kSlack = 20.f;                   // growth of the sum's exponents
constexpr uint32_t kPolls = 1u << 16;

template <int D>
struct Stage {
  static constexpr uint32_t kCodes = kTile * D;  // bytes of a tile of K or V
  static constexpr uint32_t kBytes = 2 * kCodes;
  static constexpr int kCount = D == 128 ? 3 : 6;
};

// Whether q is kept in shared memory: beside the outputs of 16 rows registers do not hold it.
template <int D, int NT>
constexpr bool kSharedQ = D == 128 && NT == 2;

template <int D, int NT, int KH, int kWarps>
struct Shared {
  Piece piece[kAhead];
  uint64_t piece_full[kAhead], piece_empty[kAhead];
  uint64_t full[Stage<D>::kCount], empty[Stage<D>::kCount], met[KH];
  float2 stat[2][kWarps][8 * NT];  // references and sums of a piece with tiles, and of the last one before it that had some
  int abort;
  ShareStart<32 * (kWarps + 2), 1> work;
  alignas(16) uint8_t scale[Stage<D>::kCount][2][kTile];
  uint4 q[kSharedQ<D, NT> ? KH : 1][D / 16][32];  // as the products take it, two eights of rows a lane
};

template <int D, int NT, int KH, int kWarps>
constexpr uint32_t header_bytes() {
  return (uint32_t)(sizeof(Shared<D, NT, KH, kWarps>) + 1023) / 1024 * 1024;
}
template <int D, int NT, int KH, int kWarps>
constexpr uint32_t smem_bytes() {
  return header_bytes<D, NT, KH, kWarps>() + Stage<D>::kCount * Stage<D>::kBytes;
}

// (A piece's beginning and end cost a block as much as three tiles: 128 requests of 300 to 8000
// cached 121.5 us, counted as one tile 138, as two 126, as four 121.5.)
template <int NT, int KH>
struct FormFew : WorkForm<kTile / KH, kMaxShares, 8 * NT * KH, true, 3> {
  static_assert(counts_in_32_bits(kMaxTableTokens, FormFew::kKeys, FormFew::kCost, kMaxKvHeads / KH), "work_fits");
};

// By all lanes of a warp; false once a wait has given up (after about a second, a minute
// with more polls).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t polls = kPolls) {
  bool ok = true;
#pragma unroll 1
  for (uint32_t i = 1; ok && !mbar_try_wait_sleep(bar, parity, 20000u); ++i)
    if ((i & 15) == 0) {
      if (i >= polls) *abort = 1;
      ok = *abort == 0;
    }
  return __all_sync(0xffffffffu, ok);
}

// The low or high two codes of a word as float16.
__device__ __forceinline__ uint32_t halves_lo(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.f16x2.e4m3x2 %0, b;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A scale's power of two, and its exponent.
__device__ __forceinline__ float power_of(uint32_t s) {
  return __uint_as_float(s == 255 ? 0x7fc00000u : s == 0 ? 0x00400000u : s << 23);
}
__device__ __forceinline__ float exponent_of(uint32_t s) {
  return s == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(0x4b000000u | s) - 8388735.f;  // 2^23 + 127
}

// The query heads of one KV head: in the parameters a group of KH heads counts as one.
struct Heads {
  int32_t group, n_kv_heads;
  Divisor by_group;
};

// NT times 8 rows a KV head; kWarps warps with keys, kG times 16 at a time, one that walks over
// the share, one that loads.
template <int D, int NT, int KH, int kWarps, int kG>
__global__ void __launch_bounds__(32 * (kWarps + 2), 2)
    attn_e4m3_few_kernel(const AttnParams p, const Heads hd, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV) {
  using F = FormFew<NT, KH>;
  using St = Stage<D>;
  using S = Shared<D, NT, KH, kWarps>;
  constexpr int kThreads = 32 * (kWarps + 2), kHeadWarps = kWarps / KH;
  constexpr int kKeys = kTile / KH, kWarpKeys = kTile / kWarps;  // keys of a tile, of a warp of it
  static_assert(kWarpKeys % (16 * kG) == 0 && kG <= 2 && 16 * NT <= kWarpKeys, "a warp's outputs in its keys' places");
  constexpr int kStages = St::kCount;
  constexpr int kRows = 8 * NT * KH;
  constexpr bool kQShared = kSharedQ<D, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  S& sh = *reinterpret_cast<S*>(smem);
  uint8_t* ring = smem + header_bytes<D, NT, KH, kWarps>();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool misplaced = (smem_u32(smem) & 1023u) != 0;  // (the swizzle is taken from address bits)
  if (tid == 0) {
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&sh.piece_full[i], 1);
      mbar_init(&sh.piece_empty[i], kWarps + 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    for (int i = 0; i < KH; ++i) mbar_init(&sh.met[i], kHeadWarps);
    sh.abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  // what stands above runs while the kernel before this one finishes
  pdl_wait();
  const Partials part = partials<D>(p.workspace);
  const int share = blockIdx.x;
  const int64_t total = locate_shares<F, kThreads, 1>(p, kRows, share, sh.work);
  if (tid == 0) part.cut[share].valid = 0;
  __syncthreads();
  pdl_launch_dependents();
  const int64_t begin = F::begin(total, share), end = F::begin(total, share + 1);
  if (misplaced || begin >= end) {
    if (misplaced && tid == 0) report(p.status, kErrCuda);
    return;
  }
  volatile int* abort = &sh.abort;
  uint32_t stage = 0, parity = 0;
  // A tile's boxes (a page's keys of all heads of the group): head by head the keys within a
  // box. Where 16 keys of head h from key r of the tile on stand, in keys.
  const int rows = min(1 << p.pool.page_shift, kKeys);
  auto stand = [&](int h, int r) { return (r & -rows) * KH + h * rows + (r & (rows - 1)); };

  if (warp == kWarps) {
    // ------------------------------------------------------------------ walk
    Walk<F> wk;
    wk.start(begin, end, sh.work, 0);
    for (uint32_t np = 0;; ++np) {
      const Piece x = wk.next(p, kRows, lane == 0 ? part.cut + share : nullptr, total);
      const uint32_t i = np % kAhead;
      // (a piece may be as long as the cache)
      if (!wait_warp(&sh.piece_empty[i], ((np / kAhead) & 1) ^ 1, abort, kPolls << 6)) break;
      if (lane == 0) {
        sh.piece[i] = x;
        mbar_arrive(&sh.piece_full[i]);
      }
      if (x.n < 0) break;
    }
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------------ loads
    const int shift = p.pool.page_shift, page_size = 1 << shift;
    const int boxes = kKeys / rows;  // pages of a tile: a lane's each
    const int64_t scale_part = (int64_t)hd.n_kv_heads << shift;
    constexpr int kNoPage = INT32_MIN;
    const int32_t* table = nullptr;
    int n = 0, tile0 = 0, lo = 0, hi = 0, head = 0, page = 0, j = 0;
    bool seen = false;
    uint32_t np = 0;
    // Whether a row sees this lane's page of a tile, and its table entry, which is looked at when
    // the tile is loaded only.
    auto find_page = [&](int tile) {
      const int key = tile * kKeys + lane * rows;
      seen = lane < boxes && key < hi && key + rows > lo;
      if (seen) page = __ldcg(table + (key >> shift));
    };
    // the next piece with tiles (n < 0: there is none), and its first page
    auto next_piece = [&] {
      do {
        const uint32_t i = np % kAhead;
        if (!wait_warp(&sh.piece_full[i], (np / kAhead) & 1, abort, kPolls << 6)) return false;
        const volatile Piece& x = sh.piece[i];
        n = x.n;
        tile0 = x.tile0;
        lo = x.lo;
        hi = x.hi;
        head = x.h * KH;
        table = p.block_table + (int64_t)x.b * p.max_pages;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.piece_empty[i]);
        ++np;
      } while (n == 0);
      j = 0;
      if (n > 0) find_page(tile0);
      return true;
    };
    bool ok = next_piece();
    while (ok && n > 0) {
      int now = seen ? max(page, -1) : kNoPage;  // (an entry may be any number)
      const int token = ((tile0 + j) * kKeys) & (page_size - 1), now_head = head;
      if (now != kNoPage && (now < 0 || now >= p.pool.n_pages)) {
        report(p.status, kErrBounds);
        now = 0;
      }
      const uint32_t some = __ballot_sync(0xffffffffu, now != kNoPage);
      // (the next tile's page is on its way before the wait for a place for this one)
      const bool last = ++j == n;
      if (!last) find_page(tile0 + j);
      ok = wait_warp(&sh.empty[stage], parity ^ 1, abort);
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(&sh.full[stage], __popc(some) * 2 * KH * rows * (D + 1));
      __syncwarp();
      if (now != kNoPage) {
        const int at = lane * KH * rows;
        uint8_t* to = ring + stage * St::kBytes + at * D;
        const uint8_t* from = p.pool.scales + 2 * (int64_t)now * scale_part + ((int64_t)now_head << shift) + token;
        tma_load_4d_plain(to, &tmK, &sh.full[stage], 0, token, now_head, now);
        tma_load_4d_plain(to + St::kCodes, &tmV, &sh.full[stage], 0, token, now_head, now);
        // (heads' scales stand a page apart: one copy if a box is a page)
        const int copies = rows == page_size ? 1 : KH, bytes = KH * rows / copies;
        for (int h = 0; h < copies; ++h) {
          bulk_load(&sh.scale[stage][0][at + h * bytes], from + (h << shift), bytes, &sh.full[stage]);
          bulk_load(&sh.scale[stage][1][at + h * bytes], from + scale_part + (h << shift), bytes, &sh.full[stage]);
        }
      }
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1;
      }
      if (last) ok = next_piece();
    }
  } else {
    // ------------------------------------------------------------------ keys
    const int g = lane >> 2, t = lane & 3;
    const int sub = warp / kHeadWarps, of_head = warp % kHeadWarps;  // its head of the group, its place there
    const float c = p.scale * kLog2eHi;
    const bool tree = p.mask != nullptr;
    uint4 w_q[NT][D / 32];  // a piece's q as it is loaded: row g of each eight, D / 4 columns from (D / 4) t
    // Row of q and head of a row of this warp's head; its place among the unit's rows.
    auto place_of = [&](const volatile Piece& x, int row, int64_t& tr, int& head) {
      const int tok = hd.by_group.quotient(row), in = sub * hd.group + row - tok * hd.group;
      tr = x.token + tok;
      head = x.h * p.group + in;
      return tok * p.group + in;
    };
    auto load_q = [&](const volatile Piece& x) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        int64_t tr;
        int head;
        const bool there = place_of(x, 8 * n + g, tr, head) < x.rows;
        const uint4* from = reinterpret_cast<const uint4*>(p.q + tr * p.q_token + head * p.q_head) + t * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w_q[n][i] = there ? __ldcg(from + i) : make_uint4(0, 0, 0, 0);
      }
    };
    uint32_t met = 0;
    if (wait_warp(&sh.piece_full[0], 0, abort, kPolls << 6)) {
      if (sh.piece[0].n > 0) load_q(sh.piece[0]);
      for (uint32_t np = 0;; ++np) {
        // (read where it is used, to keep the loop's registers few; released at the piece's end)
        const volatile Piece& x = sh.piece[np % kAhead];
        const int n_tiles = x.n, tile0 = x.tile0;
        if (n_tiles < 0) break;
        // keys that a row sees (of a tree's row: of the context), and its row of q
        auto range_of = [&](int row, int& lo, int& hi) -> int64_t {
          const int tok = hd.by_group.quotient(row), pos = x.pos + tok;
          const int64_t tr = x.token + tok;
          hi = tree ? x.ctx : p.causal ? min(pos + 1, x.kv) : x.kv;
          lo = tree ? tree_low(p, x.ctx, tr) : p.window > 0 ? max(0, pos - p.window + 1) : 0;
          return tr;
        };
        const int n_rows = x.rows / KH;  // of this warp's head
        uint32_t q[NT][D / 8];
        float c_row[NT][2];                // of rows 2 t, 2 t + 1 of each eight: factor of their scores
        int lo_all = x.lo, hi_all = x.hi;  // keys that all rows see
        const int lo_any = x.lo, hi_any = x.hi;
        float r[NT][2], dv[NT][2], l[NT][2];  // reference of the sum, and less that of the weights; sum
        float o[NT][D / 16][4];
        if (n_tiles > 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint32_t top = 0;
            constexpr uint32_t kAbs = 0x7fff7fffu;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const uint4 y = w_q[n][i];
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(y.x & kAbs, y.y & kAbs), __vmaxu2(y.z & kAbs, y.w & kAbs)));
            }
            top = max(top & 0xffffu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t up = min(268u - (top >> 7), 253u);  // exponent field of 2^(14 - E), largest value 2^E and more
            const float f = __uint_as_float(up << 23), down = __uint_as_float((254u - up) << 23);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const uint32_t y[4] = {w_q[n][i].x, w_q[n][i].y, w_q[n][i].z, w_q[n][i].w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                q[n][4 * i + k] = to_f16x2(__uint_as_float(y[k] << 16) * f, __uint_as_float(y[k] & 0xffff0000u) * f);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              c_row[n][i] = c * __shfl_sync(0xffffffffu, down, 4 * (2 * t + i));
              const int row = 8 * n + 2 * t + i;
              int lo, hi;
              if (row < n_rows) {
                range_of(row, lo, hi);
                lo_all = max(lo_all, lo);
                hi_all = min(hi_all, hi);
              }
              r[n][i] = -FLT_MAX;
              dv[n][i] = 0.f;
              l[n][i] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
          }
          lo_all = __reduce_max_sync(0xffffffffu, lo_all);
          hi_all = __reduce_min_sync(0xffffffffu, hi_all);
          if constexpr (kQShared) {
            // (a head's warps write the same; all of them have met since q was last read)
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              sh.q[sub][k][lane] = make_uint4(q[0][2 * k], q[0][2 * k + 1], q[NT - 1][2 * k], q[NT - 1][2 * k + 1]);
            __syncwarp();
          }
        }
        bool ok = true;
        for (int it = 0; it < n_tiles; ++it) {
          ok = wait_warp(&sh.full[stage], parity, abort);
          if (!ok) break;
#pragma unroll 1
          for (int k0 = 0; k0 < kWarpKeys; k0 += 16 * kG) {
            const int row0 = of_head * kWarpKeys + k0;  // of the tile's keys of this head
            const int key0 = (tile0 + it) * kKeys + row0;
            if (key0 + 16 * kG <= lo_any || key0 >= hi_any) continue;
            int off[kG];  // places of 16 keys each
#pragma unroll
            for (int u = 0; u < kG; ++u) off[u] = stand(sub, row0 + 16 * u);
            const uint8_t* kc = ring + stage * St::kBytes;
            const uint8_t* vc = kc + St::kCodes;
            const uint8_t* sc = &sh.scale[stage][0][0];
            float ev[kG][2];      // exponents of the values of keys g, g + 8 (and 16 on)
            float s[kG][NT][4];   // scores in exponents of 2; key g: rows 2 t, 2 t + 1; key g + 8
            {
              float s2[kG][NT][4];  // (two chains of products)
              uint4 w[kG][2][D / 64];
#pragma unroll
              for (int u = 0; u < kG; ++u) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int i = 0; i < 4; ++i) s[u][n][i] = s2[u][n][i] = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int row = g + 8 * i;  // (16 keys do not change the swizzle)
#pragma unroll
                  for (int k = 0; k < D / 64; ++k) {
                    const int chunk = D == 128 ? (2 * t + k) ^ (row & 7) : t ^ ((row >> 1) & 3);
                    w[u][i][k] = *reinterpret_cast<const uint4*>(kc + (off[u] + row) * D + chunk * 16);
                  }
                }
              }
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                uint32_t qk[2 * NT];
                if constexpr (kQShared) {
                  const uint4 y = sh.q[sub][k][lane];
                  qk[0] = y.x;
                  qk[1] = y.y;
                  qk[2 * NT - 2] = y.z;
                  qk[2 * NT - 1] = y.w;
                } else {
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    qk[2 * n] = q[n][2 * k];
                    qk[2 * n + 1] = q[n][2 * k + 1];
                  }
                }
#pragma unroll
                for (int u = 0; u < kG; ++u) {
                  const uint4 &y = w[u][0][k / 4], &z = w[u][1][k / 4];
                  const uint32_t a = k % 4 == 0 ? y.x : k % 4 == 1 ? y.y : k % 4 == 2 ? y.z : y.w;
                  const uint32_t b = k % 4 == 0 ? z.x : k % 4 == 1 ? z.y : k % 4 == 2 ? z.z : z.w;
                  const uint32_t f[4] = {halves_lo(a), halves_lo(b), halves_hi(a), halves_hi(b)};
#pragma unroll
                  for (int n = 0; n < NT; ++n) mma_f16(k & 1 ? s2[u][n] : s[u][n], f, qk[2 * n], qk[2 * n + 1]);
                }
              }
#pragma unroll
              for (int u = 0; u < kG; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float ks = power_of(sc[off[u] + g + 8 * i]);
                  ev[u][i] = exponent_of(sc[kTile + off[u] + g + 8 * i]);
                  // (the factors' product first: with a large scale the score alone passes float32's range)
#pragma unroll
                  for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) s[u][n][2 * i + j] = (s[u][n][2 * i + j] + s2[u][n][2 * i + j]) * (ks * c_row[n][j]);
                }
            }
            // the values' codes: 4 keys
            constexpr int kVW = D / 32;  // words of a key
            uint32_t w[kG][4][kVW];
#pragma unroll
            for (int u = 0; u < kG; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = 2 * t + (i & 1) + 8 * (i >> 1);
                const uint8_t* from = vc + (off[u] + row) * D;
                if constexpr (D == 128) {
                  const uint4 y = *reinterpret_cast<const uint4*>(from + ((g ^ (row & 7)) << 4));
                  w[u][i][0] = y.x;
                  w[u][i][1] = y.y;
                  w[u][i][kVW - 2] = y.z;
                  w[u][i][kVW - 1] = y.w;
                } else {
                  const uint2 y = *reinterpret_cast<const uint2*>(from + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
                  w[u][i][0] = y.x;
                  w[u][i][1] = y.y;
                }
              }
            if (key0 < lo_all || key0 + 16 * kG > hi_all) {
              uint32_t any = 0;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t seen = 0;
                  const int row = 8 * n + 2 * t + i;
                  if (row < n_rows) {
                    int lo, hi;
                    const int64_t tr = range_of(row, lo, hi);
                    seen = tree ? tree_seen(p.mask + tr * p.mask_words, p.mask_words, key0, lo, hi, x.kv)
                                : bits_between(lo - key0, hi - key0);
                  }
                  any |= seen;
#pragma unroll
                  for (int u = 0; u < kG; ++u) {
                    if (!(seen >> (16 * u + g) & 1)) s[u][n][i] = kNegInf;
                    if (!(seen >> (16 * u + g + 8) & 1)) s[u][n][2 + i] = kNegInf;
                  }
                }
              // keys that no row sees may hold anything: their values become zeros
              any |= __shfl_xor_sync(0xffffffffu, any, 1);
              any |= __shfl_xor_sync(0xffffffffu, any, 2);
#pragma unroll
              for (int u = 0; u < kG; ++u) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (!(any >> (16 * u + g + 8 * i) & 1)) ev[u][i] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (!(any >> (16 * u + 2 * t + (i & 1) + 8 * (i >> 1)) & 1))
#pragma unroll
                    for (int k = 0; k < kVW; ++k) w[u][i][k] = 0;
              }
            }
            // exponents over the references: of the sum's terms, of the weights
            float e[kG][NT][4], ew[kG][NT][4], top_e = kNegInf, top_w = kNegInf;
#pragma unroll
            for (int u = 0; u < kG; ++u)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  e[u][n][i] = s[u][n][i] - r[n][i & 1];
                  ew[u][n][i] = e[u][n][i] + (ev[u][i >> 1] + dv[n][i & 1]);
                  top_e = fmaxf(top_e, e[u][n][i]);
                  top_w = fmaxf(top_w, ew[u][n][i]);
                }
            if (__any_sync(0xffffffffu, top_e > kSlack || top_w > kTop)) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  float a = kNegInf, b = kNegInf;
#pragma unroll
                  for (int u = 0; u < kG; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) a = fmaxf(a, s[u][n][2 * k + i]);
#pragma unroll
                  for (int d = 4; d < 32; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
                  const float was = r[n][i];
                  if (a - was > kSlack) r[n][i] = a;
                  // (relative to r, which may be too large for what is added to it to count)
#pragma unroll
                  for (int u = 0; u < kG; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                      e[u][n][2 * k + i] = s[u][n][2 * k + i] - r[n][i];
                      b = fmaxf(b, e[u][n][2 * k + i] + ev[u][k]);
                    }
#pragma unroll
                  for (int d = 4; d < 32; d <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
                  if (r[n][i] != was || b + dv[n][i] > kTop) {
                    const float up = r[n][i] - was, now = fminf(kRaised - b, dv[n][i] + up);  // (r' does not fall)
                    const float f = ex2_approx(now - dv[n][i] - up);
                    l[n][i] *= ex2_approx(-up);
                    dv[n][i] = now;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                      o[n][j][i] *= f;
                      o[n][j][2 + i] *= f;
                    }
                  }
#pragma unroll
                  for (int u = 0; u < kG; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) ew[u][n][2 * k + i] = e[u][n][2 * k + i] + (ev[u][k] + dv[n][i]);
                }
            }
#pragma unroll
            for (int u = 0; u < kG; ++u) {
              uint32_t b0[NT], b1[NT];
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  l[n][i & 1] += ex2_approx(e[u][n][i]);
                  // (where a key is not seen, its value's scale may be NaN)
                  v[i] = e[u][n][i] == kNegInf ? 0.f : ex2_approx(ew[u][n][i]);
                }
                b0[n] = transpose8(to_f16x2(v[0], v[1]));
                b1[n] = transpose8(to_f16x2(v[2], v[3]));
              }
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
                const uint32_t a = __byte_perm(w[u][0][j / 2], w[u][1][j / 2], sel), b = __byte_perm(w[u][2][j / 2], w[u][3][j / 2], sel);
                const uint32_t f[4] = {halves_lo(a), halves_hi(a), halves_lo(b), halves_hi(b)};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(o[n][j], f, b0[n], b1[n]);
              }
            }
          }
          __syncwarp();
          if (it + 1 < n_tiles) {
            if (lane == 0) mbar_arrive(&sh.empty[stage]);
            if (++stage == kStages) {
              stage = 0;
              parity ^= 1;
            }
          }
        }
        if (!ok) break;
        // the next piece, which the producer has handed out by now as a rule, and its q
        const uint32_t nx = (np + 1) % kAhead;
        ok = wait_warp(&sh.piece_full[nx], ((np + 1) / kAhead) & 1, abort, kPolls << 6);
        if (!ok) break;
        if (sh.piece[nx].n > 0) load_q(sh.piece[nx]);
        if (n_tiles > 0) {
          // The outputs on the warp's own reference, four rows of each eight in the places of its
          // keys and four in those of its values (16-byte pieces so that accesses do not collide).
          // (By meetings, not by pieces: those that see nothing have none, and only the meeting in between
          // orders the writes to a buffer behind what a slower warp still reads there.)
          float2(&stat)[kWarps][8 * NT] = sh.stat[met & 1];
          constexpr int kChunks = D / 4;
          auto place = [&](int w, int n, int row) {
            return reinterpret_cast<float4*>(ring + stage * St::kBytes + (row >> 2) * St::kCodes +
                                             stand(sub, w * kWarpKeys + 16 * n) * D + (row & 3) * (D * 4));
          };
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], d);
              if (g == 0) stat[warp][8 * n + 2 * t + i] = make_float2(r[n][i], l[n][i]);
              // (in two halves: values at the ends of bfloat16's range have factors past float32's)
              const float f = ex2_approx(-0.5f * dv[n][i]);
              float4* to = place(of_head, n, 2 * t + i);
              // a lane's D / 8 columns from (D / 8) g: two a product
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                to[(g * (D / 32) + k) ^ t] = make_float4(o[n][2 * k][i] * f * f, o[n][2 * k][2 + i] * f * f,
                                                         o[n][2 * k + 1][i] * f * f, o[n][2 * k + 1][2 + i] * f * f);
            }
          // a head's warps meet (with a limit: one that has given up elsewhere does not come)
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.met[sub]);
          ok = wait_warp(&sh.met[sub], met & 1, abort);
          ++met;
          if (!ok) break;
          for (int i = of_head * 32 + lane; i < n_rows * kChunks; i += 32 * kHeadWarps) {
            const int row = i / kChunks, chunk = i % kChunks;
            float top = -FLT_MAX, sum = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kHeadWarps; ++w) top = fmaxf(top, stat[sub * kHeadWarps + w][row].x);
#pragma unroll
            for (int w = 0; w < kHeadWarps; ++w) {
              const float2 st = stat[sub * kHeadWarps + w][row];
              const float4 z = place(w, row >> 3, row & 7)[chunk ^ ((row & 7) >> 1)];
              const float f = ex2_approx(st.x - top);
              if (st.y == 0.f) continue;  // saw nothing
              sum = fmaf(st.y, f, sum);
              y = make_float4(fmaf(z.x, f, y.x), fmaf(z.y, f, y.y), fmaf(z.z, f, y.z), fmaf(z.w, f, y.w));
            }
            const bool some = sum > 0.f || sum != sum;
            const float f = !x.whole ? 1.f : some ? 1.f / sum : 0.f;
            int64_t tr;
            int head;
            const size_t prow = (size_t)(share * 2 + x.slot) * F::kPartRows + place_of(x, row, tr, head);
            if (x.whole)
              reinterpret_cast<uint2*>(p.out + tr * p.o_token + head * p.o_head)[chunk] =
                  make_uint2(to_bf16x2(y.x * f, y.y * f), to_bf16x2(y.z * f, y.w * f));
            else
              reinterpret_cast<float4*>(part.out + prow * D)[chunk] = y;
            if (chunk == 0) {
              if (!x.whole)
                part.stat[prow] = make_float2(some ? top : kNegInf, sum);
              else if (p.lse != nullptr)
                p.lse[tr * p.n_heads + head] = some ? (top + log2f(sum)) * kLn2 : kNegInf;
            }
          }
          fence_proxy_async_smem();  // the stage's next filling comes by TMA
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
          }
        } else {
          // nothing to see
          for (int i = of_head * 32 + lane; i < n_rows * (D / 8); i += 32 * kHeadWarps) {
            int64_t tr;
            int head;
            place_of(x, i / (D / 8), tr, head);
            reinterpret_cast<uint4*>(p.out + tr * p.o_token + head * p.o_head)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
            if (i % (D / 8) == 0 && p.lse != nullptr) p.lse[tr * p.n_heads + head] = kNegInf;
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&sh.piece_empty[np % kAhead]);
      }
    }
  }
  __syncthreads();
  if (*abort) {  // (a warp that gives up ends the others' waits)
    if (tid == 0) report(p.status, kErrTimeout);
    for (int i = 0; i < 64; ++i) __nanosleep(20000);  // (copies in flight end before the block does)
  }
}

template <int D, int NT, int KH>
cudaError_t launch(const AttnParams& given, cudaStream_t s) {
  static Readiness readiness;
  // Four warps with keys and 168 registers, 32 keys at a time: 128 requests of 4 rows 108 us; eight
  // warps and 96 registers, 16 keys at a time, 122 (spills), D = 64 80 and 86. 16 rows of D = 128
  // hold the sums of 16 keys at a time only: 142 us, 152 with 32.
  constexpr int kWarps = 4, kG = D == 128 && NT == 2 ? 1 : 2;
  constexpr uint32_t kSmem = smem_bytes<D, NT, KH, kWarps>();
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two blocks an SM");
  const auto kernel = attn_e4m3_few_kernel<D, NT, KH, kWarps, kG>;
  const cudaError_t ready =
      readiness.get([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (ready != cudaSuccess) return ready;
  CUtensorMap mk, mv;
  const int page = 1 << given.pool.page_shift, keys = kTile / KH;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)page, (cuuint64_t)given.pool.n_kv_heads, (cuuint64_t)given.pool.n_pages};
  const cuuint64_t str[3] = {(cuuint64_t)given.pool.token_stride, (cuuint64_t)given.pool.head_stride,
                             (cuuint64_t)given.pool.page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)(page < keys ? page : keys), (cuuint32_t)KH, 1};
  if (!encode_tmap_bytes(&mk, given.pool.k, 4, dims, str, box, true) || !encode_tmap_bytes(&mv, given.pool.v, 4, dims, str, box, true))
    return cudaErrorInvalidValue;
  const Heads heads = {given.group, given.pool.n_kv_heads, given.by_group};
  AttnParams p = given;
  p.group *= KH;
  p.by_group.set((uint32_t)p.group);
  p.pool.n_kv_heads /= KH;
  const cudaError_t e = launch_early(kernel, dim3(kMaxShares), dim3(32 * (kWarps + 2)), kSmem, s, p, heads, mk, mv);
  if (e != cudaSuccess) return e;
  // (four rows a block of the join: KH heads' rows stand together. Tokens of 128 requests 104.7 us,
  // of short ones 22.6; two a block 106 and 23.2)
  return launch_join<FormFew<NT, KH>, D, __nv_bfloat16, 4>(p, s, p.max_q * p.group, 8 * NT * KH, 8 * NT * KH);
}

template <int D, int NT>
cudaError_t launch_heads(const AttnParams& p, cudaStream_t s) {
  if constexpr (D == 64 && NT == 1)
    if (p.pool.n_kv_heads % 4 == 0) return launch<D, NT, 4>(p, s);
  return p.pool.n_kv_heads % 2 == 0 ? launch<D, NT, 2>(p, s) : launch<D, NT, 1>(p, s);
}

}  // namespace

cudaError_t launch_attention_e4m3_few(const AttnParams& p, cudaStream_t s) {
  const bool eight = p.max_q * p.group <= 8;
  if (p.D == 128) return eight ? launch_heads<128, 1>(p, s) : launch_heads<128, 2>(p, s);
  return eight ? launch_heads<64, 1>(p, s) : launch_heads<64, 2>(p, s);
}

}  // namespace ds
