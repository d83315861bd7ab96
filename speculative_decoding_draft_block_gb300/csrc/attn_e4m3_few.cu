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
// Units, shares and the join are those of attn_work.cuh, with tiles of 128 keys. Two
// blocks an SM. A producer warp walks over the share and loads tiles (codes
// swizzled, one box a page, scales beside them) into a ring; each of eight warps takes
// 16 keys of every tile, with references, sums and outputs of its own, which are put
// together at the end of a piece in the ring's last stage. References are raised when a lane
// finds that one has to be (a vote a tile), so no maxima go over lanes otherwise.
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

constexpr int kTile = kAttnTileTc;               // keys of a tile
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

template <int D, int NT, int kWarps>
struct Shared {
  Piece piece[kAhead];
  uint64_t piece_full[kAhead], piece_empty[kAhead];
  uint64_t full[Stage<D>::kCount], empty[Stage<D>::kCount], met;
  float2 stat[kWarps][8 * NT];  // a piece's references and sums
  int abort;
  ShareStart<32 * (kWarps + 1), 1> work;
  alignas(16) uint8_t scale[Stage<D>::kCount][2][kTile];
};

template <int D, int NT, int kWarps>
constexpr uint32_t header_bytes() {
  return (uint32_t)(sizeof(Shared<D, NT, kWarps>) + 1023) / 1024 * 1024;
}
template <int D, int NT, int kWarps>
constexpr uint32_t smem_bytes() {
  return header_bytes<D, NT, kWarps>() + Stage<D>::kCount * Stage<D>::kBytes;
}

template <int NT>
struct FormFew : WorkForm<kTile, kMaxShares, 8 * NT, true> {};

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

// A meeting of the warps with keys: a barrier with a limit, since one that has given up
// elsewhere does not come.
struct Meeting {
  uint32_t parity = 0;
  __device__ __forceinline__ bool operator()(uint64_t* bar, volatile int* abort) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    const bool ok = wait_warp(bar, parity, abort);
    parity ^= 1;
    return ok;
  }
};

// A scale's power of two, and its exponent.
__device__ __forceinline__ float power_of(uint32_t s) {
  return __uint_as_float(s == 255 ? 0x7fc00000u : s == 0 ? 0x00400000u : s << 23);
}
__device__ __forceinline__ float exponent_of(uint32_t s) {
  return s == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(0x4b000000u | s) - 8388735.f;  // 2^23 + 127
}

// NT times 8 rows, kWarps warps with keys and the producer.
template <int D, int NT, int kWarps>
__global__ void __launch_bounds__(32 * (kWarps + 1), 2)
    attn_e4m3_few_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using F = FormFew<NT>;
  using St = Stage<D>;
  using S = Shared<D, NT, kWarps>;
  constexpr int kThreads = 32 * (kWarps + 1);
  static_assert(kTile % (16 * kWarps) == 0 && kWarps * 8 * D * 4 <= (int)St::kBytes, "keys of a warp, sums in a stage");
  constexpr int kStages = St::kCount;
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(1024) uint8_t smem[];
  S& sh = *reinterpret_cast<S*>(smem);
  uint8_t* ring = smem + header_bytes<D, NT, kWarps>();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool misplaced = (smem_u32(smem) & 1023u) != 0;  // (the swizzle is taken from address bits)
  if (tid == 0) {
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&sh.piece_full[i], 1);
      mbar_init(&sh.piece_empty[i], kWarps);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    mbar_init(&sh.met, kWarps);
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

  if (warp == kWarps) {
    // ------------------------------------------------------------------ producer
    const int shift = p.pool.page_shift, page_size = 1 << shift;
    const int rows = min(page_size, kTile), boxes = kTile / rows;  // keys of a box, pages of a tile
    Walk<F> wk;
    wk.start(begin, end, sh.work, 0);
    bool ok = true;
    for (uint32_t np = 0; ok; ++np) {
      const Piece x = wk.next(p, kRows, lane == 0 ? part.cut + share : nullptr, total);
      const uint32_t i = np % kAhead;
      // (a piece may be as long as the cache)
      ok = wait_warp(&sh.piece_empty[i], ((np / kAhead) & 1) ^ 1, abort, kPolls << 6);
      if (!ok) break;
      if (lane == 0) {
        sh.piece[i] = x;
        mbar_arrive(&sh.piece_full[i]);
      }
      if (x.n < 0) break;
      const int32_t* table = p.block_table + (int64_t)x.b * p.max_pages;
      // Table entry of this lane's box of a tile, kNoPage: no row sees it.
      constexpr int kNoPage = INT32_MIN;
      auto page_of = [&](int tile) {
        const int key = tile * kTile + lane * rows;
        if (lane >= boxes || key >= x.hi || key + rows <= x.lo) return kNoPage;
        return __ldcg(table + (key >> shift));
      };
      int page = x.n > 0 ? page_of(x.tile0) : kNoPage;
      for (int j = 0; j < x.n; ++j) {
        const int tile = x.tile0 + j;
        int now = page;
        if (j + 1 < x.n) page = page_of(tile + 1);
        if (now != kNoPage && (now < 0 || now >= p.pool.n_pages)) {
          report(p.status, kErrBounds);
          now = 0;
        }
        const uint32_t some = __ballot_sync(0xffffffffu, now != kNoPage);
        const int token = (tile * kTile) & (page_size - 1);
        ok = wait_warp(&sh.empty[stage], parity ^ 1, abort);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&sh.full[stage], __popc(some) * 2 * rows * (D + 1));
        __syncwarp();
        // a lane a box
        if (now != kNoPage) {
          uint8_t* to = ring + stage * St::kBytes + lane * rows * D;
          const uint8_t* from = p.pool.scales + 2 * (int64_t)now * p.pool.scale_part() + ((int64_t)x.h << shift) + token;
          tma_load_4d_plain(to, &tmK, &sh.full[stage], 0, token, x.h, now);
          tma_load_4d_plain(to + St::kCodes, &tmV, &sh.full[stage], 0, token, x.h, now);
          bulk_load(&sh.scale[stage][0][lane * rows], from, rows, &sh.full[stage]);
          bulk_load(&sh.scale[stage][1][lane * rows], from + p.pool.scale_part(), rows, &sh.full[stage]);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ keys
    const int g = lane >> 2, t = lane & 3;
    const float c = p.scale * kLog2eHi;
    const bool tree = p.mask != nullptr;
    Meeting meet;
    for (uint32_t np = 0;; ++np) {
      const uint32_t at = np % kAhead;
      if (!wait_warp(&sh.piece_full[at], (np / kAhead) & 1, abort, kPolls << 6)) break;
      // (read where it is used, to keep the loop's registers few; released at the piece's end)
      const volatile Piece& x = sh.piece[at];
      const int n_tiles = x.n, tile0 = x.tile0;
      if (n_tiles < 0) break;
      auto head_of = [&](int row, int64_t& tok_row) {  // query head of a row, and its row of q
        const int tok = p.by_group.quotient(x.off + row);
        tok_row = x.token + tok;
        return x.h * p.group + x.off + row - tok * p.group;
      };
      if (n_tiles == 0) {
        for (int i = tid; i < x.rows * (D / 8); i += 32 * kWarps) {
          int64_t tr;
          const int row = i / (D / 8), head = head_of(row, tr);
          reinterpret_cast<uint4*>(p.out + tr * p.o_token + head * p.o_head)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
          if (i % (D / 8) == 0 && p.lse != nullptr) p.lse[tr * p.n_heads + head] = kNegInf;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.piece_empty[at]);
        continue;
      }
      // q as the products take it: row g of each eight, D / 4 columns from (D / 4) t
      uint32_t q[NT][D / 8];
      float c_row[NT][2];       // of rows 2 t, 2 t + 1 of each eight: factor of their scores
      int lo_all = x.lo, hi_all = x.hi;  // keys that all rows see
      // keys that a row sees (of a tree's row: of the context), and its row of q
      auto range_of = [&](int row, int& lo, int& hi) -> int64_t {
        const int tok = p.by_group.quotient(x.off + row), pos = x.pos + tok;
        const int64_t tr = x.token + tok;
        hi = tree ? x.ctx : p.causal ? min(pos + 1, x.kv) : x.kv;
        lo = tree ? tree_low(p, x.ctx, tr) : p.window > 0 ? max(0, pos - p.window + 1) : 0;
        return tr;
      };
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint4 w[D / 32];
        int64_t tr;
        const int row = 8 * n + g, head = head_of(row, tr);
        const bool there = row < x.rows;
        const uint4* from = reinterpret_cast<const uint4*>(p.q + tr * p.q_token + head * p.q_head) + t * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = there ? __ldcg(from + i) : make_uint4(0, 0, 0, 0);
        uint32_t top = 0;
        constexpr uint32_t kAbs = 0x7fff7fffu;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[i].x & kAbs, w[i].y & kAbs), __vmaxu2(w[i].z & kAbs, w[i].w & kAbs)));
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t up = min(268u - (top >> 7), 253u);  // exponent field of 2^(14 - E), largest value 2^E and more
        const float f = __uint_as_float(up << 23), down = __uint_as_float((254u - up) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t y[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            q[n][4 * i + k] = to_f16x2(__uint_as_float(y[k] << 16) * f, __uint_as_float(y[k] & 0xffff0000u) * f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          c_row[n][i] = c * __shfl_sync(0xffffffffu, down, 4 * (2 * t + i));
          const int r = 8 * n + 2 * t + i;
          int lo, hi;
          if (r < x.rows) {
            range_of(r, lo, hi);
            lo_all = max(lo_all, lo);
            hi_all = min(hi_all, hi);
          }
        }
      }
      lo_all = __reduce_max_sync(0xffffffffu, lo_all);
      hi_all = __reduce_min_sync(0xffffffffu, hi_all);
      const int lo_any = x.lo, hi_any = x.hi;
      float r[NT][2], rv[NT][2], l[NT][2];  // references of the sum and of the weights, sum
      float o[NT][D / 16][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          r[n][i] = rv[n][i] = -FLT_MAX;
          l[n][i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][j][i] = 0.f;
      }
      bool ok = true;
      for (int it = 0; it < n_tiles; ++it) {
        ok = wait_warp(&sh.full[stage], parity, abort);
        if (!ok) break;
#pragma unroll 1
        for (int sub = warp; sub < kTile / 16; sub += kWarps) {
          const int key0 = (tile0 + it) * kTile + 16 * sub;
          if (key0 + 16 <= lo_any || key0 >= hi_any) continue;
          const uint8_t* kc = ring + stage * St::kBytes;
          const uint8_t* vc = kc + St::kCodes;
          const uint8_t* sc = &sh.scale[stage][0][16 * sub];
          float ks[2], ev[2];  // of keys g, g + 8
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ks[i] = power_of(sc[g + 8 * i]);
            ev[i] = exponent_of(sc[kTile + g + 8 * i]);
          }
          float s[NT][4];  // key g: rows 2 t, 2 t + 1; key g + 8
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
          {
            uint4 w[2][D / 64];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = 16 * sub + g + 8 * i;
#pragma unroll
              for (int k = 0; k < D / 64; ++k) {
                const int chunk = D == 128 ? (2 * t + k) ^ (row & 7) : t ^ ((row >> 1) & 3);
                w[i][k] = *reinterpret_cast<const uint4*>(kc + row * D + chunk * 16);
              }
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint4 &y = w[0][k / 4], &z = w[1][k / 4];
              const uint32_t a = k % 4 == 0 ? y.x : k % 4 == 1 ? y.y : k % 4 == 2 ? y.z : y.w;
              const uint32_t b = k % 4 == 0 ? z.x : k % 4 == 1 ? z.y : k % 4 == 2 ? z.z : z.w;
              const uint32_t f[4] = {halves_lo(a), halves_lo(b), halves_hi(a), halves_hi(b)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(s[n], f, q[n][2 * k], q[n][2 * k + 1]);
            }
          }
          // the values' codes: 4 keys
          constexpr int kVW = D / 32;  // words of a key
          uint32_t w[4][kVW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 16 * sub + 2 * t + (i & 1) + 8 * (i >> 1);
            if constexpr (D == 128) {
              const uint4 y = *reinterpret_cast<const uint4*>(vc + row * D + ((g ^ (row & 7)) << 4));
              w[i][0] = y.x;
              w[i][1] = y.y;
              w[i][kVW - 2] = y.z;
              w[i][kVW - 1] = y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(vc + row * D + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
              w[i][0] = y.x;
              w[i][1] = y.y;
            }
          }
          float e[NT][4];  // exponents of the weights in the sum
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][i] *= ks[i >> 1];
          if (key0 < lo_all || key0 + 16 > hi_all) {
            uint32_t any = 0;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t seen = 0;
                const int row = 8 * n + 2 * t + i;
                if (row < x.rows) {
                  int lo, hi;
                  const int64_t tr = range_of(row, lo, hi);
                  seen = tree ? tree_seen(p.mask + tr * p.mask_words, p.mask_words, key0, lo, hi, x.kv)
                              : bits_between(lo - key0, hi - key0);
                }
                any |= seen;
                if (!(seen >> g & 1)) s[n][i] = kNegInf;
                if (!(seen >> (g + 8) & 1)) s[n][2 + i] = kNegInf;
              }
            // keys that no row sees may hold anything: their values become zeros
            any |= __shfl_xor_sync(0xffffffffu, any, 1);
            any |= __shfl_xor_sync(0xffffffffu, any, 2);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (!(any >> (g + 8 * i) & 1)) ev[i] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(any >> (2 * t + (i & 1) + 8 * (i >> 1)) & 1))
#pragma unroll
                for (int k = 0; k < kVW; ++k) w[i][k] = 0;
          }
          bool raise = false;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[n][i] = s[n][i] * c_row[n][i & 1];
              raise |= e[n][i] - r[n][i & 1] > kSlack || e[n][i] + ev[i >> 1] - rv[n][i & 1] > kTop;
            }
          if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float a = fmaxf(e[n][i], e[n][2 + i]), b = fmaxf(e[n][i] + ev[0], e[n][2 + i] + ev[1]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
                  b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
                }
                if (a - r[n][i] > kSlack) {
                  l[n][i] *= ex2_approx(r[n][i] - a);
                  r[n][i] = a;
                }
                if (b - rv[n][i] > kTop) {
                  const float f = ex2_approx(rv[n][i] - (b - kRaised));
                  rv[n][i] = b - kRaised;
#pragma unroll
                  for (int j = 0; j < D / 16; ++j) {
                    o[n][j][i] *= f;
                    o[n][j][2 + i] *= f;
                  }
                }
              }
          }
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              l[n][i & 1] += ex2_approx(e[n][i] - r[n][i & 1]);
              // (where a key is not seen, its value's scale may be NaN)
              v[i] = e[n][i] == kNegInf ? 0.f : ex2_approx(e[n][i] + (ev[i >> 1] - rv[n][i & 1]));
            }
            b0[n] = transpose8(to_f16x2(v[0], v[1]));
            b1[n] = transpose8(to_f16x2(v[2], v[3]));
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
            const uint32_t a = __byte_perm(w[0][j / 2], w[1][j / 2], sel), b = __byte_perm(w[2][j / 2], w[3][j / 2], sel);
            const uint32_t f[4] = {halves_lo(a), halves_hi(a), halves_lo(b), halves_hi(b)};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][j], f, b0[n], b1[n]);
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
      // The warps' sums on one reference, eight rows at a time through the last tile's stage
      // (16-byte pieces placed so that neither side's accesses collide).
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], d);
          if (g == 0) sh.stat[warp][8 * n + 2 * t + i] = make_float2(r[n][i], l[n][i]);
        }
      if (!meet(&sh.met, abort)) break;
      float4* sums = reinterpret_cast<float4*>(ring + stage * St::kBytes);
      constexpr int kChunks = D / 4;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 2 * t + i;
          float top = -FLT_MAX;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.stat[w][8 * n + row].x);
          // (in two halves: values at the ends of bfloat16's range have factors past float32's)
          const float f = rv[n][i] == -FLT_MAX ? 0.f : ex2_approx(0.5f * (rv[n][i] - top));
          // a lane's D / 8 columns from (D / 8) g: two a product
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const int chunk = g * (D / 32) + k;
            sums[(warp * 8 + row) * kChunks + (chunk ^ t)] =
                make_float4(o[n][2 * k][i] * f * f, o[n][2 * k][2 + i] * f * f, o[n][2 * k + 1][i] * f * f,
                            o[n][2 * k + 1][2 + i] * f * f);
          }
        }
        ok = meet(&sh.met, abort);
        if (!ok) break;
        for (int i = tid; i < 8 * kChunks; i += 32 * kWarps) {
          const int row = i / kChunks, chunk = i % kChunks, urow = 8 * n + row;
          if (urow >= x.rows) continue;
          float top = -FLT_MAX, sum = 0.f;
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.stat[w][urow].x);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 st = sh.stat[w][urow];
            const float4 z = sums[(w * 8 + row) * kChunks + (chunk ^ (row >> 1))];
            sum += st.y * ex2_approx(st.x - top);
            y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
          }
          const bool some = sum > 0.f || sum != sum;
          const float f = !x.whole ? 1.f : some ? 1.f / sum : 0.f;
          int64_t tr;
          const int head = head_of(urow, tr);
          const size_t prow = (size_t)(share * 2 + x.slot) * F::kPartRows + urow;
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
        ok = meet(&sh.met, abort);
        if (!ok) break;
      }
      if (!ok) break;
      fence_proxy_async_smem();  // the stage's next filling comes by TMA
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.empty[stage]);
        mbar_arrive(&sh.piece_empty[at]);
      }
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1;
      }
    }
  }
  __syncthreads();
  if (*abort) {  // (a warp that gives up ends the others' waits)
    if (tid == 0) report(p.status, kErrTimeout);
    for (int i = 0; i < 64; ++i) __nanosleep(20000);  // (copies in flight end before the block does)
  }
}

template <int D, int NT, int kWarps>
cudaError_t launch(const AttnParams& p, cudaStream_t s) {
  static Readiness readiness;
  constexpr uint32_t kSmem = smem_bytes<D, NT, kWarps>();
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two blocks an SM");
  const cudaError_t ready = readiness.get(
      [] { return cudaFuncSetAttribute(attn_e4m3_few_kernel<D, NT, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (ready != cudaSuccess) return ready;
  CUtensorMap mk, mv;
  const int page = 1 << p.pool.page_shift;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)page, (cuuint64_t)p.pool.n_kv_heads, (cuuint64_t)p.pool.n_pages};
  const cuuint64_t str[3] = {(cuuint64_t)p.pool.token_stride, (cuuint64_t)p.pool.head_stride, (cuuint64_t)p.pool.page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)(page < kTile ? page : kTile), 1, 1};
  if (!encode_tmap_bytes(&mk, p.pool.k, 4, dims, str, box, true) || !encode_tmap_bytes(&mv, p.pool.v, 4, dims, str, box, true))
    return cudaErrorInvalidValue;
  const cudaError_t e = launch_early(attn_e4m3_few_kernel<D, NT, kWarps>, dim3(kMaxShares), dim3(32 * (kWarps + 1)), kSmem, s, p, mk, mv);
  if (e != cudaSuccess) return e;
  return launch_join<FormFew<NT>, D, __nv_bfloat16>(p, s, p.max_q * p.group, 8 * NT, 8 * NT);
}

}  // namespace

cudaError_t launch_attention_e4m3_few(const AttnParams& p, cudaStream_t s) {
  const bool eight = p.max_q * p.group <= 8;
  if (p.D == 128) return eight ? launch<128, 1, 8>(p, s) : launch<128, 2, 4>(p, s);
  return eight ? launch<64, 1, 8>(p, s) : launch<64, 2, 4>(p, s);
}

}  // namespace ds
