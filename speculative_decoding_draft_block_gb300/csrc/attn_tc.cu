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
// 128 / G whole tokens). All units' key tiles (128 keys each), one after the
// other with kUnitCost tiles' worth of set-up before each unit, are the work
// list, and it is cut into equal contiguous shares. Lengths are read on the
// device only, shares are equal to within a tile whatever the batch looks like,
// and a unit that is cut is joined by the second kernel from float32 partial results.
//
// A CTA works with two streams, each with its own score tile, output
// accumulator and softmax warpgroup: while the scores of one go through the
// softmax, the tensor core works on the other's. Three forms, chosen on the host:
//   solo (requests of one row tile on average): each stream has a share of its
//        own, 2 x 152 in all, and a unit is one row tile. Bound by the keys' way
//        from memory; the tensor work of the mostly empty rows stays below it.
//        128 verify blocks of up to 17 tokens, 500 to 6000 cached (1.18 GB): 198 us,
//        5.9 TB/s. Short contexts are bound by the chain of a unit (page entry, Q, K,
//        product, softmax, product, result).
//   few (up to 16 rows a unit: single tokens, short blocks): as solo, but a row
//        stands in the lanes of all four softmax warps (Q is loaded four times), and
//        each of them takes a quarter of a tile's keys, with a reference of its own,
//        and zeros as the other quarters' weights. A lane has 32 scores to work on
//        instead of 128, which shortens the chain of a tile; a piece's quarters
//        are put together at its end, through shared memory.
//   pair (longer requests): a CTA has one share, a unit is two row tiles, one a
//        stream, and both read each key tile from shared memory. Bound by the
//        tensor core and, between its products, by the softmax that feeds it. Units
//        with one row tile run on stream 0. Prompt chunks of 2 x 2048 tokens over
//        9000 to 16384 cached: 465 to 528 us, 1.55 to 1.36 PFLOP/s by the clock.
//
//   warps 0, 1  producers: walk over the share (solo: one a stream, with its K and
//               V; pair: one for Q and K, one for V), hand its pieces to the softmax
//               and load tiles by TMA (one box per page and 64 elements,
//               128B-swizzled) into a ring of kSlots
//   warps 2, 3  MMA issuers (solo: one a stream; pair: one for both): S = Q K^T (both
//               in shared memory), O += P V (P in TMEM over its scores, V in shared
//               memory, MN-major). What to do with a tile stands in the slot's info
//               word. They also clear the V rows that no row sees in a unit's first
//               and last tile: a weight of zero does not cancel a NaN in a matrix
//               product
//   warps 4-7, 8-11   softmax of streams 0 and 1: a thread a row
//
// With one producer and one issuer warp for both streams their waits, commits and
// bookkeeping bound the solo form (4.6 TB/s).
// The ring's entries stand in a fixed order, in which every role counts by itself:
//   solo  K0 K1 | V0 K0' V1 K1' | V0' ...   (the streams' next tiles in turn)
//   pair  K V K V ...
//
// TMEM (512 columns): scores 2 x 128, accumulators 2 x D. Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>

#include "attn_work.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace ds {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kTile = kAttnTileTc;  // keys a tile, rows a tile
constexpr int kFewRows = 16;       // rows of a unit in the form for few rows
constexpr float kSlack = 8.f;      // growth of the exponents that is left in the sums
constexpr uint32_t kCtrlRegs = 88, kSoftRegs = 208, kLaunchRegs = 168;
static_assert(128 * kCtrlRegs + 256 * kSoftRegs <= kThreads * kLaunchRegs, "register split exceeds the launch pool");
constexpr uint32_t kWaitPolls = 1u << 16;
constexpr uint32_t kHeader = 3072;  // barriers and small records, before the tiles
constexpr int kAhead = 4;           // pieces handed out ahead, per stream
constexpr int kMaxSlots = 12;

template <int D>
struct Layout {
  static constexpr uint32_t kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 12;
  static constexpr uint32_t kOffQ = kHeader;
  static constexpr uint32_t kOffRing = kOffQ + 2 * kTileBytes;
  static constexpr uint32_t kBytes = kOffRing + kSlots * kTileBytes;
  static_assert(kSlots <= kMaxSlots && kBytes <= 227 * 1024, "shared memory");
};

// A ring slot's info word, for key entries: what this entry and the value entry
// of the same tile are.
enum : uint32_t {
  kNull = 1u,   // nothing: the stream has ended, the other one has not
  kEnd = 2u,    // no more entries of this stream
  kFirst = 4u,  // first tile of a piece
  kLast = 8u,   // last tile of a piece
  kTwo = 16u,   // the unit has two row tiles
  kPart = 32u   // only keys [bits 8..15, bits 16..23) of the tile are seen
};

// What the waits look at beside their barrier.
struct Watch {
  int abort;  // a wait has given up
  int anew;   // warps that compute rows again (see `anew`), which may take long
};

struct Header {
  Piece piece[2][kAhead];
  uint64_t piece_full[2][kAhead], piece_empty[2][kAhead];
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t drain[2];
  uint64_t merged[2];                   // (few rows) a piece's quarters stand in its staging slot
  float2 quarter[2][4][kFewRows];       // their references and sums
  uint32_t info[kMaxSlots];
  uint32_t entry[kMaxSlots];  // 1 + the number of the entry that the slot was last given to
  uint32_t staged[2];         // softmax warps that are done with a piece's staging slot
  int ended[2];         // tiles of a stream's share, -1 while not known
  uint32_t tmem;
  Watch watch;
  ShareStart<kThreads, 2> work;
};
static_assert(sizeof(Header) <= kHeader, "header");

// A role's place in the ring.
//
// A barrier's parity tells the phase that is awaited from the one before it and
// no more, so a role may wait for an entry's filling (its release) only once it
// knows that the slot's filling (release) before that one is over.
//   - A pair's issuer passes every entry in order: it has waited for it.
//   - The solo issuers pass their own stream's entries only, and with five slots
//     the slot's last entry is the other stream's. So they wait for the entry's
//     number in `entry` first: the producer writes it once the slot is released.
//   - So do the producers, before they wait for the release of the entry kSlots
//     before theirs: that its number stands there means that the one before it,
//     which may be another producer's, has been released.
template <int kSlots>
struct RingPos {
  uint32_t slot = 0, parity = 0, number = 0;
  __device__ __forceinline__ void add(uint32_t n) {  // n < kSlots
    number += n;
    slot += n;
    if (slot >= kSlots) {
      slot -= kSlots;
      parity ^= 1u;
    }
  }
};

enum : int { kSolo, kPairs, kFew };  // forms

// Key tiles, shares of the work list and rows of partial results of a form.
template <int kForm>
struct Form : WorkForm<kTile, kForm == kPairs ? kMaxAttnCtas : 2 * kMaxAttnCtas,
                       kForm == kPairs ? 2 * kTile : kForm == kFew ? kFewRows : kTile> {};

// Bounded waits. One that gives up sets the abort flag, which ends every role's
// loop; the status is reported once, at the kernel's end (the waits are many and
// inlined, and the warps' loops share one instruction cache). While a warp computes
// rows again, which ends by itself, the others' waits do not count.
__device__ __forceinline__ bool given_up(volatile Watch* watch, uint32_t& polled, uint32_t limit) {
  if (watch->anew != 0) polled = 0;
  if (polled >= limit) watch->abort = 1;
  return watch->abort != 0;
}

// Waits until the entry of that number stands in a slot.
__device__ __forceinline__ bool wait_number(const uint32_t* entry, uint32_t number, volatile Watch* watch) {
  const volatile uint32_t* at = entry;
#pragma unroll 1
  for (uint32_t i = 1; *at != number; ++i) {
    __nanosleep(40);
    if ((i & 255) == 0 && given_up(watch, i, kWaitPolls << 8)) return false;
  }
  return true;
}

// By one thread: about a second with kWaitPolls, a minute with kIdlePolls, for
// roles that may have nothing to do for as long as a unit lasts.
constexpr uint32_t kIdlePolls = 1u << 22;
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile Watch* watch, uint32_t polls) {
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait_sleep(bar, parity, 20000u); ++i)
    if ((i & 15) == 0 && given_up(watch, i, polls)) return false;
  return true;
}

// The same by a whole warp, with one answer for all lanes: warp-wide instructions follow.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile Watch* watch,
                                         uint32_t polls = kWaitPolls) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, watch, polls));
}

__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i <= kWaitPolls; ++i)
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return;
}

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

// One or two words, zeros if they are not there.
__device__ __forceinline__ void load_words(uint32_t (&to)[1], const char* from, bool there) {
  to[0] = there ? __ldcg(reinterpret_cast<const uint32_t*>(from)) : 0u;
}
__device__ __forceinline__ void load_words(uint32_t (&to)[2], const char* from, bool there) {
  const uint2 y = there ? __ldcg(reinterpret_cast<const uint2*>(from)) : make_uint2(0u, 0u);
  to[0] = y.x;
  to[1] = y.y;
}

// ---- the kernel --------------------------------------------------------------------------

template <int D, int kForm>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV) {
  using L = Layout<D>;
  using F = Form<kForm>;
  constexpr bool kPair = kForm == kPairs;
  constexpr int kSlots = L::kSlots;
  constexpr int kHalves = D / 64;
  constexpr int kLists = kPair ? 1 : 2;  // shares of a CTA
  extern __shared__ __align__(1024) uint8_t smem[];
  Header& sh = *reinterpret_cast<Header*>(smem);
  uint8_t* sQ = smem + L::kOffQ;
  uint8_t* sRing = smem + L::kOffRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per_tile = p.by_group.quotient(kForm == kFew ? kFewRows : kTile);  // tokens of a row tile
  const int tile_rows = per_tile * p.group;      // rows in use of a row tile
  const int unit_rows = (kPair ? 2 : 1) * tile_rows;

  // the swizzle is taken from address bits (the array's alignment; never seen otherwise)
  const bool misplaced = (smem_u32(smem) & 1023u) != 0;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.drain[i], 1);
      mbar_init(&sh.merged[i], 4);
      sh.ended[i] = -1;
      sh.staged[i] = 0;
      for (int k = 0; k < kAhead; ++k) {
        mbar_init(&sh.piece_full[i][k], 1);
        mbar_init(&sh.piece_empty[i][k], kPair ? 8 : 4);  // softmax warps
      }
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
      sh.entry[i] = 0;
    }
    sh.watch.abort = 0;
    sh.watch.anew = 0;
    fence_barrier_init();
  }

  if (warp == 2) tmem_alloc(&sh.tmem, 512);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  // what stands above runs while the kernel before this one finishes
  pdl_wait();
  const Partials part = partials<D>(p.workspace);
  const int v0 = blockIdx.x * kLists;
  const int64_t total = locate_shares<F, kThreads, kLists>(p, unit_rows, v0, sh.work);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if (misplaced || F::begin(total, v0) >= F::begin(total, v0 + kLists)) {
    if (misplaced && tid == 0) report(p.status, kErrCuda);
    if (tid < kLists) part.cut[v0 + tid].valid = 0;
    if (warp == 2) tmem_dealloc(tmem, 512);
    return;
  }
  volatile Watch* watch = &sh.watch;
  pdl_launch_dependents();

  if (warp < 4) {
    setmaxnreg_dec<kCtrlRegs>();
    if (warp < 2) {
      // ---------------------------------------------------------------- producers
      const int l = kPair ? 0 : warp;                      // share
      const bool does_k = !kPair || warp == 0, does_v = !kPair || warp == 1;
      const int shift = p.pool.page_shift, page_size = 1 << shift;
      const int rows = min(page_size, kTile);              // keys of a box
      const int boxes = kTile / rows;                      // pages a tile
      const uint32_t box_bytes = (uint32_t)rows * 128u;
      Walk<F> wk;
      wk.start(F::begin(total, v0 + l), F::begin(total, v0 + l + 1), sh.work, l);
      if (does_k && lane == 0) part.cut[v0 + l].valid = 0;
      RingPos<kSlots> kp, vp;                              // places of the next K and V entry
      if (!kPair) kp.add(l);
      vp.add(kPair ? 1 : l == 0 ? 2 : 4);
      uint32_t q_par[2] = {1, 1}, np = 0;
      int n_tiles = 0;                                     // of the share so far
      bool ok = true, ended = false;
      Piece x = {};
      int j = 0;                                           // next tile of the piece
      const int32_t* table = nullptr;
      // Table entry of this lane's box of a key tile, kNoPage: no row of the unit sees
      // it. (Looked at when the tile is loaded, a tile later as a rule.)
      constexpr int kNoPage = INT32_MIN;
      auto page_of = [&](int tile) {
        const int key = tile * kTile + lane * rows;
        if (lane >= boxes || key >= x.hi || key + rows <= x.lo) return kNoPage;
        return __ldcg(table + (key >> shift));
      };
      int page = kNoPage;                                  // of the next tile
      volatile int* ends = sh.ended;
      while (true) {
        if (!ended && j == x.n) {  // the next piece
          x = wk.next(p, unit_rows, does_k && lane == 0 ? part.cut + v0 + l : nullptr, total);
          j = 0;
          // its first tile's page is on its way while it goes to the softmax
          if (x.n > 0) {
            table = p.block_table + (int64_t)x.b * p.max_pages;
            page = page_of(x.tile0);
          }
          if (does_k) {
            const uint32_t i = np % kAhead;
            ok = wait_bar(&sh.piece_empty[l][i], ((np / kAhead) & 1) ^ 1, watch, kIdlePolls);
            if (!ok) break;
            if (lane == 0) {
              sh.piece[l][i] = x;
              mbar_arrive(&sh.piece_full[l][i]);
            }
            ++np;
          }
          if (x.n == 0) continue;
          ended = x.n < 0;
          if (ended) {
            if (!does_k) break;
            if (lane == 0) ends[l] = n_tiles;
          } else if (does_k) {
            const int s0 = kPair ? 0 : l, s1 = kPair ? (x.rows > tile_rows ? 1 : 0) : l;
#pragma unroll 1
            for (int s = s0; s <= s1; ++s) {
              ok = wait_bar(&sh.q_empty[s], s == 0 ? q_par[0] : q_par[1], watch);
              if (!ok) break;
              if (s == 0) q_par[0] ^= 1;
              if (s == 1) q_par[1] ^= 1;
              if (elect_one()) {
                constexpr int kCopies = kForm == kFew ? 4 : 1;  // (few rows: a copy for each softmax warp)
                mbar_expect_tx(&sh.q_full[s], (uint32_t)tile_rows * D * 2 * kCopies);
                for (int y = 0; y < kHalves; ++y)
                  for (int i = 0; i < kCopies; ++i)
                    tma_load_3d_plain(sQ + s * L::kTileBytes + y * (kTile * 128) + i * (32 * 128), &tmQ, &sh.q_full[s],
                                      y * 64, x.h * p.group, x.token + (kPair ? s * per_tile : 0));
              }
              __syncwarp();
            }
            if (!ok) break;
          }
        }
        // The tile's entries; once the share has ended (solo) empty ones, since the
        // other stream may have more tiles, until both have.
        const int tile = x.tile0 + j;
        int now = kNoPage;
        uint32_t word = 0;
        if (!ended) {
          now = page;
          if (j + 1 < x.n) page = page_of(tile + 1);
          word = (x.rows > tile_rows ? kTwo : 0u) | (j == 0 ? kFirst : 0u) | (j + 1 == x.n ? kLast : 0u);
          if (F::partly_seen(tile, x.lo, x.hi))
            word |= kPart | (uint32_t)max(0, x.lo - tile * kTile) << 8 | (uint32_t)min(kTile, x.hi - tile * kTile) << 16;
          if (now != kNoPage && (now < 0 || now >= p.pool.n_pages)) {
            report(p.status, kErrBounds);
            now = 0;
          }
        }
        const uint32_t some = __ballot_sync(0xffffffffu, now != kNoPage);
        const int token = (tile * kTile) & (page_size - 1);
#pragma unroll 1
        for (int kv = does_k ? 0 : 1; kv < (does_v ? 2 : 1); ++kv) {
          const uint32_t slot = kv ? vp.slot : kp.slot, parity = kv ? vp.parity : kp.parity;
          const uint32_t number = kv ? vp.number : kp.number;
          if (number >= (uint32_t)kSlots)
            ok = __all_sync(0xffffffffu, wait_number(&sh.entry[slot], number - kSlots + 1, watch));
          ok = ok && wait_bar(&sh.empty[slot], parity ^ 1, watch);
          if (!ok) break;
          if (ended) {
            // (whether the other stream has ended is read after the wait for a slot: what
            // is waited for may be its last entry, and no entry follows that one)
            const int other = kPair ? 0 : __shfl_sync(0xffffffffu, ends[l ^ 1], 0);
            word = kv == 0 && other >= 0 && (kPair || n_tiles >= other) ? kEnd : kNull;
          }
          if (lane == 0) {
            sh.info[slot] = word;
            *(volatile uint32_t*)&sh.entry[slot] = number + 1;
            mbar_expect_tx(&sh.full[slot], __popc(some) * kHalves * box_bytes);
          }
          __syncwarp();
          if (word & kEnd) break;
          const CUtensorMap* map = kv ? &tmV : &tmK;
          uint8_t* dst = sRing + slot * L::kTileBytes;
#pragma unroll 1
          for (int i = 0; i < boxes; ++i) {
            const int pg = __shfl_sync(0xffffffffu, now, i);
            if (pg != kNoPage && elect_one()) {
#pragma unroll
              for (int y = 0; y < kHalves; ++y)
                tma_load_4d_plain(dst + i * box_bytes + y * (kTile * 128), map, &sh.full[slot], y * 64, token, x.h, pg);
            }
            __syncwarp();
          }
        }
        if (!ok || (ended && (word & kEnd))) break;
        ++n_tiles;
        // (solo: K0 is followed by three other entries' places, then by four)
        kp.add(kPair ? 2 : l == 0 && n_tiles == 1 ? 3 : 4);
        vp.add(kPair ? 2 : 4);
        if (!ended) ++j;
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- MMA issuers
      // (all lanes run the loop, one issues)
      constexpr uint32_t iqk = idesc_bf16(kTile, kTile, false, false);
      constexpr uint32_t ipv = idesc_bf16(kTile, D, false, true);
      constexpr uint64_t kbits = smem_desc_bits(16, 1024, 2);
      constexpr uint64_t vbits = smem_desc_bits(kTile * 128, 1024, 2);
      const int s0 = kPair ? 0 : warp - 2;  // the issuer's stream (a pair's has both)
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = smem_desc(sQ, kbits), k_desc = smem_desc(sRing, kbits), v_desc = smem_desc(sRing, vbits);
      RingPos<kSlots> kp, vp;
      if (!kPair) kp.add(s0);
      vp.add(kPair ? 1 : s0 == 0 ? 2 : 4);
      uint32_t q_par = 0, p_par = 0;  // a bit a stream
      bool begun = false;
      auto uniform = [&](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
      // The waits stand with the products in one region of the elected lane: a
      // warp-wide wait with its vote costs the issuer 200 cycles and more, as much
      // as three products. `good`: no wait has given up (that lane's flag).
      bool good = true;
      auto wait1 = [&](uint64_t* bar, uint32_t parity) {
        good = good && wait_one(bar, parity, watch, kWaitPolls);
      };
      auto wait_entry = [&](const RingPos<kSlots>& at) {
        if (!kPair) good = good && wait_number(&sh.entry[at.slot], at.number + 1, watch);
        wait1(&sh.full[at.slot], at.parity);
      };
      // S = Q K^T of stream s with the keys in `slot`; `free_k`: nothing else needs the slot
      auto qk = [&](int s, uint32_t slot, bool last, bool free_k) {
        if (!good) return;
        tc_fence_after();
        const uint64_t a = q_desc + s * (L::kTileBytes >> 4), b = k_desc + slot * (L::kTileBytes >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * ((kTile * 128) >> 4) + (k & 3) * 2;
          mma_bf16(tm + s * kTile, a + off, b + off, iqk, k != 0);
        }
        mma_commit(&sh.s_full[s]);
        if (free_k) mma_commit(&sh.empty[slot]);
        if (last) mma_commit(&sh.q_empty[s]);
      };
      // O (+)= P V of stream s with the values in `slot`
      auto pv = [&](int s, uint32_t slot, bool first, bool last, bool free_v) {
        wait1(&sh.p_full[s], (p_par >> s) & 1);
        if (!good) return;
        tc_fence_after();
        const uint64_t b = v_desc + slot * (L::kTileBytes >> 4);
        const uint32_t more = first ? 0u : 1u;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_bf16_ta(tm + 256 + s * D, tm + s * kTile + k * 8, b + k * (2048 >> 4), ipv, k != 0 ? 1u : more);
        if (free_v) mma_commit(&sh.empty[slot]);
        if (last) mma_commit(&sh.pv_done[s]);
      };
      // within a region: the info word of the entry at `at`, or, after a wait that has
      // given up, an end without an entry; after it, that word for all lanes
      auto info_of = [&](const RingPos<kSlots>& at) {
        return good ? *(volatile uint32_t*)&sh.info[at.slot] : (uint32_t)(kEnd | kNull);
      };
      auto share_info = [&](uint32_t word) { return __reduce_or_sync(0xffffffffu, word); };
      auto next_k = [&] {
        kp.add(kPair ? 2 : s0 == 0 && !begun ? 3 : 4);
        begun = true;
      };
      auto next_v = [&] { vp.add(kPair ? 2 : 4); };
      // clears the rows of the value tile at vp that no row sees
      auto clear = [&](uint32_t info) {
        if (elect_one()) wait_entry(vp);
        __syncwarp();
        if (__any_sync(0xffffffffu, watch->abort)) return;
        const int head = (info >> 8) & 255, tail = (info >> 16) & 255;
        uint8_t* tile = sRing + vp.slot * L::kTileBytes;
#pragma unroll 1
        for (int half = 0; half < kHalves; ++half) {
          uint4* v = reinterpret_cast<uint4*>(tile + half * (kTile * 128));
#pragma unroll 1
          for (int j = lane; j < head * 8; j += 32) v[j] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
          for (int j = tail * 8 + lane; j < kTile * 8; j += 32) v[j] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      uint32_t info = 0;
      if (!kPair) {
        bool due = false;  // a tile's scores are made, its product with the values is due
        // S | O S' | O' S'' ...: a region does the product with the weights and the next scores
        uint32_t k_was = 0;
        while (true) {
          if (due && (info & (kPart | kNull)) == kPart) clear(info);
          const uint32_t k_at = uniform(kp.slot), v_at = uniform(vp.slot);
          uint32_t next = 0;
          if (elect_one()) {
            if (due) {
              if (info & kNull) mma_commit(&sh.empty[k_was]);  // (unused entries: releases after those before them)
              wait_entry(vp);
              if (info & kNull) {
                if (good) mma_commit(&sh.empty[v_at]);
              } else {
                pv(s0, v_at, info & kFirst, info & kLast, !(info & kLast));
              }
            }
            wait_entry(kp);
            next = info_of(kp);
            if (!(next & (kNull | kEnd))) {
              if (next & kFirst) wait1(&sh.q_full[s0], q_par);
              qk(s0, k_at, next & kLast, true);
            }
          }
          if (due) {
            if (!(info & kNull)) p_par ^= 1u << s0;
            next_v();
          }
          info = share_info(next);
          if (info & kEnd) break;
          due = true;
          k_was = k_at;
          if (info & kFirst) q_par ^= 1;
          next_k();
        }
      } else if (warp == 2) {
        // S0 S1 | O0 S0' O1 S1' | ...: a stream's scores are made while the other's go
        // through the softmax. One warp for both streams: products of two warps
        // interleave on the tensor core and take longer (1.01 against 1.31 PFLOP/s
        // when it was tried).
        auto scores = [&](int s, uint32_t at, uint32_t word) {
          const bool two = word & kTwo;
          if (s == 1 && !two) return;
          if (word & kFirst) wait1(&sh.q_full[s], (q_par >> s) & 1);
          qk(s, at, word & kLast, (s == 1 || !two) && !(word & kLast));
        };
        uint32_t next = 0;
        if (elect_one()) {
          wait_entry(kp);
          next = info_of(kp);
          if (!(next & kEnd)) {
            scores(0, kp.slot, next);
            scores(1, kp.slot, next);
          }
        }
        info = share_info(next);
        while (!(info & kEnd)) {
          const bool two = info & kTwo, first = info & kFirst, last = info & kLast;
          if (first) q_par ^= two ? 3u : 1u;
          next_k();
          const uint32_t k_at = uniform(kp.slot), v_at = uniform(vp.slot);
          if (info & kPart) clear(info);
          next = 0;
          if (elect_one()) {
            wait_entry(vp);
            if (!last) {
              // the next keys are there as a rule: wait for them before the weights
              wait_entry(kp);
              next = info_of(kp);
              pv(0, v_at, first, false, !two);
              scores(0, k_at, next);
              if (two) {
                pv(1, v_at, first, false, true);
                scores(1, k_at, next);
              }
            } else {
              pv(0, v_at, first, true, !two);
              if (two) pv(1, v_at, first, true, false);
              wait_entry(kp);
              next = info_of(kp);
              if (!(next & kEnd)) {
                scores(0, k_at, next);
                scores(1, k_at, next);
              }
            }
          }
          p_par ^= two ? 3u : 1u;
          next_v();
          info = share_info(next);
        }
      }
      if ((info & (kEnd | kNull)) == kEnd && elect_one()) mma_commit(&sh.empty[kp.slot]);
      __syncwarp();
      if (elect_one()) mma_commit(&sh.drain[warp - 2]);
      __syncwarp();
      drain_bar(&sh.drain[warp - 2], 0);  // no product in flight when TMEM is freed
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------------ softmax, epilogue
    setmaxnreg_inc<kSoftRegs>();
    const int s = (warp >> 2) - 1;                 // stream
    const int quarter = warp & 3;                  // its TMEM lanes
    const int row = kForm == kFew ? lane : quarter * 32 + lane;  // row of the tile
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lanes + s * kTile, tO = tmem + lanes + 256 + s * D;
    const float c = p.scale * kLog2eHi;
    const int tile_tok = p.by_group.quotient(row), g = row - tile_tok * p.group;
    const int v = v0 + (kPair ? 0 : s);            // share
    uint32_t ns = 0, np = 0;                       // score tiles and pieces so far
    uint32_t list_tiles = 0;                       // key tiles of the list so far
    const int list = kPair ? 0 : s;
    for (uint32_t k = 0;; ++k) {
      const uint32_t at = k % kAhead;
      if (!wait_bar(&sh.piece_full[list][at], (k / kAhead) & 1, watch, kIdlePolls)) break;
      const Piece x = sh.piece[list][at];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.piece_empty[list][at]);
      if (x.n < 0) break;
      list_tiles += x.n;
      if (kPair && s == 1 && x.rows <= tile_rows) continue;
      const int i = (kPair ? s * per_tile : 0) + tile_tok;  // token of the unit
      const bool valid = tile_tok < per_tile && i * p.group < x.rows;
      const int pos = x.pos + i;
      const int64_t t_out = x.token + i;
      const int head = x.h * p.group + g;
      char* out = p.out + t_out * p.o_token + head * p.o_head;
      float* lse = p.lse != nullptr ? p.lse + t_out * p.n_heads + head : nullptr;
      if (x.n == 0) {
        if (valid && (kForm != kFew || quarter == 0)) {
#pragma unroll 1
          for (int d = 0; d < D / 8; ++d) reinterpret_cast<uint4*>(out)[d] = make_uint4(0, 0, 0, 0);
          if (lse != nullptr) *lse = kNegInf;
        }
        continue;
      }
      // keys this row sees; a row that is not there sees all and is never stored
      const int hi = !valid ? INT32_MAX : p.causal ? min(pos + 1, x.kv) : x.kv;
      const int lo = valid && p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const bool work = __any_sync(0xffffffffu, valid);
      float m = kNegInf, l = 0.f;  // reference (a score, before the factor c) and sum
      bool ok = true;
      // the reference, with `top` the largest score of tile `it`
      auto raise_to = [&](float top, int it) {
        top = fmaxf(m, top);
        if (it == 0) {
          m = top;
          return;
        }
        const bool raise = valid && (top - m) * c > kSlack;
        if (!__any_sync(0xffffffffu, raise)) return;
        // the accumulator is at rest: the product with the last tile's weights was
        // issued before these scores, the next one waits for our weights
        const float f = raise ? ex2_approx((m - top) * c) : 1.f;
        if (raise) m = top;
        l *= f;
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t o[16];
          tmem_ld16_issue(tO + 16 * q, o);
          tmem_ld16_wait(o);
#pragma unroll
          for (int w = 0; w < 16; ++w) o[w] = __float_as_uint(__uint_as_float(o[w]) * f);
          tmem_st16(tO + 16 * q, o);
        }
      };
      for (int it = 0; it < x.n; ++it) {
        const int key = (x.tile0 + it) * kTile;
        ok = wait_bar(&sh.s_full[s], ns & 1, watch);
        if (!ok) break;
        tc_fence_after();
        if constexpr (kForm == kFew) {
          // this warp's keys of the tile: 32 quarter .. + 31
          const int key0 = key + 32 * quarter;
          uint32_t y[32];
          tmem_ld32_issue(tS + 32 * quarter, y);
          tmem_ld_wait(y);
          if (__any_sync(0xffffffffu, key0 + 32 > hi || key0 < lo)) {
            const int a = lo - key0;
            const uint32_t seen = (uint32_t)max(0, hi - key0 - a);
#pragma unroll
            for (int w = 0; w < 32; ++w)
              if ((uint32_t)(w - a) >= seen) y[w] = __float_as_uint(kNegInf);
          }
          float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
          for (int w = 0; w < 32; ++w) mx[w & 3] = fmaxf(mx[w & 3], __uint_as_float(y[w]));
          raise_to(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), it);
          const float r = m == kNegInf ? 0.f : m * c;
          const uint64_t c2 = pack2(c, c), r2 = pack2(-r, -r);
          uint64_t sum2[2] = {0, 0};
          uint32_t pk[16], none[16];
#pragma unroll
          for (int w = 0; w < 16; ++w) {
            const uint64_t e = fma2(pack2(__uint_as_float(y[2 * w]), __uint_as_float(y[2 * w + 1])), c2, r2);
            float2 f = unpack2(e);
            f.x = ex2_approx(f.x);
            f.y = ex2_approx(f.y);
            sum2[w & 1] = add2(sum2[w & 1], pack2(f.x, f.y));
            pk[w] = to_bf16x2(f.x, f.y);
            none[w] = 0;
          }
          tmem_st16(tS + 16 * quarter, pk);
#pragma unroll
          for (int i = 1; i < 4; ++i) tmem_st16(tS + 16 * ((quarter + i) & 3), none);
          const float2 sum = unpack2(add2(sum2[0], sum2[1]));
          l += sum.x + sum.y;
          tmem_st_wait();
        } else if (work) {
          if (__any_sync(0xffffffffu, key + kTile > hi || key < lo)) {
            // Scores that a row does not see become -inf, in place, 32 keys at a time and
            // only where there are any, so that other tiles do not pay for it. (The
            // warps' loops share one instruction cache, which selects unrolled over all
            // 128 scores would crowd.)
            const int a = lo - key, z = hi - key;
            const uint32_t seen = (uint32_t)max(0, z - a);
#pragma unroll 1
            for (int q = 0; q < kTile; q += 32) {
              if (__all_sync(0xffffffffu, q >= a && q + 32 <= z)) continue;
              uint32_t y[32];
              tmem_ld32_issue(tS + q, y);
              tmem_ld_wait(y);
#pragma unroll
              for (int w = 0; w < 32; ++w)
                if ((uint32_t)(q - a + w) >= seen) y[w] = __float_as_uint(kNegInf);
              tmem_st16(tS + q, y);
              tmem_st16(tS + q + 16, y + 16);
            }
            tmem_st_wait();
          }
          uint32_t y[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32_issue(tS + 32 * q, y + 32 * q);
          tmem_ld_wait(y);
          reg_dep32(y + 32);
          reg_dep32(y + 64);
          reg_dep32(y + 96);
          float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
          for (int q = 0; q < 128; q += 8) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
              mx[w] = fmaxf(mx[w], fmaxf(__uint_as_float(y[q + 2 * w]), __uint_as_float(y[q + 2 * w + 1])));
          }
          raise_to(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), it);
          const float r = m == kNegInf ? 0.f : m * c;
          const uint64_t c2 = pack2(c, c), r2 = pack2(-r, -r);
          uint64_t sum2[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
              const uint64_t e = fma2(pack2(__uint_as_float(y[32 * q + 2 * w]), __uint_as_float(y[32 * q + 2 * w + 1])), c2, r2);
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
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[s]);
        ++ns;
      }
      if (!ok) break;
      ok = wait_bar(&sh.pv_done[s], np & 1, watch);
      if (!ok) break;
      ++np;
      tc_fence_after();
      // The result: the output, or a row of partial results. A thread has a row and
      // would store it in 32 pieces of 16 bytes, each to a line of its own across
      // the warp (3.2 us for 256 rows). So the rows go through shared memory, a
      // warp's 32 at a time, and leave in whole lines. The staging is the ring slot of
      // the piece's last values (stream 0 of a pair: keys, since the other stream may
      // still read the values); the last warp to finish releases it.
      const float ref = m == kNegInf ? kNegInf : m * c;
      const bool some = l > 0.f || l != l;
      const float f = !x.whole ? 1.f : some ? 1.f / l : 0.f;
      const size_t prow = (size_t)(v * 2 + x.slot) * F::kPartRows + (kPair ? s * kTile : 0) + row;
      const int key0 = max(x.lo, x.tile0 * kTile), key1 = min(x.hi, (x.tile0 + x.n) * kTile);
      // A value that is not finite, of a key that other rows of the unit see and this
      // one does not, has come in with its weight of zero. Such rows (`again`: a bit a
      // lane that has a row's place, keys, reference and factor) are computed again from
      // what they see, in float32, four at a time over the same keys: each lane has D / 32
      // columns; of eight keys' 32 products every lane ends up with one sum, its weight
      // (-1: unseen), and hands it to all. A piece may be as long as the cache, so
      // the other roles' waits do not count meanwhile.
      // 58 to 217 rows x keys a us and SM: 210 rows over 100,000 keys (D = 64) 95 ms.
      auto anew = [&](uint32_t again, int t_row, int h_row, char* dst, int a, int z, float r_ref, float r_f) {
        constexpr int N = D / 32, kR = 4, kK = 8;  // columns, rows, keys
        static_assert(kR * kK == 32, "a lane a row and key");
        const int shift = p.pool.page_shift;
        if (lane == 0) atomicAdd(&sh.watch.anew, 1);
        __syncwarp();  // the rows as they were first stored
#pragma unroll 1
        while (again != 0) {
          float q[kR][N], o[kR][N];
          int from[kR];
          int my_a = 0, my_z = 0;  // of row lane % kR
          float my_ref = 0.f;
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const bool there = again != 0;
            from[r] = there ? __ffs(again) - 1 : 0;
            again &= again - 1;
            const int t = __shfl_sync(0xffffffffu, t_row, from[r]), h = __shfl_sync(0xffffffffu, h_row, from[r]);
            const __nv_bfloat16* q_row = reinterpret_cast<const __nv_bfloat16*>(p.q + (int64_t)t * p.q_token + h * p.q_head);
#pragma unroll
            for (int d = 0; d < N; ++d) {
              q[r][d] = there ? __bfloat162float(q_row[lane * N + d]) : 0.f;
              o[r][d] = 0.f;
            }
            const int ra = __shfl_sync(0xffffffffu, a, from[r]), rz = __shfl_sync(0xffffffffu, z, from[r]);
            const float rr = __shfl_sync(0xffffffffu, r_ref, from[r]);
            if ((lane & (kR - 1)) == r && there) {
              my_a = ra;
              my_z = rz;
              my_ref = rr;
            }
            if (!there) from[r] = -1;
          }
          // keys that some of the rows sees
          const int a_all = __reduce_min_sync(0xffffffffu, my_a < my_z ? my_a : INT32_MAX);
          const int z_all = __reduce_max_sync(0xffffffffu, my_a < my_z ? my_z : 0);
#pragma unroll 1
          for (int k0 = a_all; k0 < z_all; k0 += 32) {
            // where this lane's key of 32 stands, -1: nowhere (a page out of range has been reported)
            int64_t place = -1;
            if (k0 + lane < z_all) {
              const int key = k0 + lane;
              const int page = __ldcg(p.block_table + (int64_t)x.b * p.max_pages + (key >> shift));
              if (page >= 0 && page < p.pool.n_pages)
                place = (int64_t)page * p.pool.page_stride + x.h * p.pool.head_stride +
                        (int64_t)(key & ((1 << shift) - 1)) * p.pool.token_stride;
            }
#pragma unroll 1
            for (int j0 = 0; j0 < 32 && k0 + j0 < z_all; j0 += kK) {
              uint32_t kk[kK][N / 2], vv[kK][N / 2];
#pragma unroll
              for (int j = 0; j < kK; ++j) {
                const int64_t off = __shfl_sync(0xffffffffu, (long long)place, j0 + j);
                load_words(kk[j], p.pool.k + off + lane * (2 * N), off >= 0);
                load_words(vv[j], p.pool.v + off + lane * (2 * N), off >= 0);
              }
              float w[32];  // [key][row]
#pragma unroll
              for (int j = 0; j < kK; ++j)
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                  w[j * kR + r] = 0.f;
#pragma unroll
                  for (int d = 0; d < N / 2; ++d)
                    w[j * kR + r] = fmaf(q[r][2 * d], __uint_as_float(kk[j][d] << 16),
                                         fmaf(q[r][2 * d + 1], __uint_as_float(kk[j][d] & 0xffff0000u), w[j * kR + r]));
                }
              // 32 sums over the lanes, that of [i] to lane i
#pragma unroll
              for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                for (int i = 0; i < d; ++i) {
                  const bool upper = lane & d;
                  const float other = __shfl_xor_sync(0xffffffffu, upper ? w[i] : w[i + d], d);
                  w[i] = (upper ? w[i + d] : w[i]) + other;
                }
              const int key = k0 + j0 + lane / kR;
              const bool seen = __shfl_sync(0xffffffffu, place >= 0, j0 + lane / kR) && key >= my_a && key < my_z;
              const float mine = seen ? ex2_approx(fmaf(w[0], c, -my_ref)) : -1.f;
#pragma unroll
              for (int j = 0; j < kK; ++j)
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                  const float f = __shfl_sync(0xffffffffu, mine, j * kR + r);
                  if (f >= 0.f)
#pragma unroll
                    for (int d = 0; d < N / 2; ++d) {
                      o[r][2 * d] = fmaf(f, __uint_as_float(vv[j][d] << 16), o[r][2 * d]);
                      o[r][2 * d + 1] = fmaf(f, __uint_as_float(vv[j][d] & 0xffff0000u), o[r][2 * d + 1]);
                    }
                }
            }
          }
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            if (from[r] < 0) continue;
            const float f = __shfl_sync(0xffffffffu, r_f, from[r]);
            char* to = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), from[r]));
#pragma unroll
            for (int d = 0; d < N; ++d) {
              if (x.whole)
                reinterpret_cast<__nv_bfloat16*>(to)[lane * N + d] = __float2bfloat16_rn(o[r][d] * f);
              else
                reinterpret_cast<float*>(to)[lane * N + d] = o[r][d];
            }
          }
        }
        if (lane == 0) atomicSub(&sh.watch.anew, 1);
      };
      const uint32_t last_tile = list_tiles - 1;
      const uint32_t stage_at = (kPair ? 2 * last_tile + s : 4 * last_tile + (s == 0 ? 2 : 4)) % kSlots;
      if constexpr (kForm == kFew) {
        // Each warp has the sums over its quarter of the keys: to the slot, and row by row
        // from there, four quarters on one reference.
        constexpr int kChunks = D / 4;         // 16-byte pieces of a row of sums
        constexpr int kAtOnce = 32 / kChunks;  // rows of a warp at a time
        static_assert(4 * kFewRows * D * 4 <= L::kTileBytes, "the quarters' sums fill a slot at most");
        float4* stage = reinterpret_cast<float4*>(sRing + stage_at * L::kTileBytes);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32_issue(tO + 32 * q, o);
          tmem_ld_wait(o);
          if (valid) {
            const float* z = reinterpret_cast<const float*>(o);
#pragma unroll
            for (int w = 0; w < 8; ++w)
              stage[(quarter * kFewRows + lane) * kChunks + ((8 * q + w) ^ (lane & 7))] =
                  make_float4(z[4 * w], z[4 * w + 1], z[4 * w + 2], z[4 * w + 3]);
          }
        }
        if (valid) sh.quarter[s][quarter][lane] = make_float2(ref, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.merged[s]);
        ok = wait_bar(&sh.merged[s], (np - 1) & 1, watch);
        if (!ok) break;
#pragma unroll 1
        for (int r0 = quarter * kAtOnce; r0 < x.rows; r0 += 4 * kAtOnce) {
          const int r = r0 + lane / kChunks, ch = lane % kChunks;
          const bool there = r < x.rows;
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          float r_ref = kNegInf, r_l = 0.f, r_f = 1.f;
          const int tok = p.by_group.quotient(r);
          const int64_t r_t = x.token + tok;
          const int r_head = x.h * p.group + r - tok * p.group;
          const size_t r_prow = (size_t)(v * 2 + x.slot) * F::kPartRows + r;
          char* dst = x.whole ? p.out + r_t * p.o_token + r_head * p.o_head : reinterpret_cast<char*>(part.out + r_prow * D);
          if (there) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r_ref = fmaxf(r_ref, sh.quarter[s][i][r].x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 st = sh.quarter[s][i][r];
              const float w = st.x == kNegInf ? 0.f : ex2_approx(st.x - r_ref);
              if (st.x == kNegInf && st.y == 0.f) continue;  // saw nothing
              const float4 z = stage[(i * kFewRows + r) * kChunks + (ch ^ (r & 7))];
              r_l = fmaf(st.y, w, r_l);
              y = make_float4(fmaf(z.x, w, y.x), fmaf(z.y, w, y.y), fmaf(z.z, w, y.z), fmaf(z.w, w, y.w));
            }
            const bool some = r_l > 0.f || r_l != r_l;
            r_f = !x.whole ? 1.f : some ? 1.f / r_l : 0.f;
            if (x.whole)
              reinterpret_cast<uint2*>(dst)[ch] = make_uint2(to_bf16x2(y.x * r_f, y.y * r_f), to_bf16x2(y.z * r_f, y.w * r_f));
            else
              reinterpret_cast<float4*>(dst)[ch] = y;
            if (ch == 0) {
              if (!x.whole)
                part.stat[r_prow] = make_float2(r_ref, r_l);
              else if (p.lse != nullptr)
                p.lse[r_t * p.n_heads + r_head] = some ? (r_ref + log2f(r_l)) * kLn2 : kNegInf;
            }
          }
          // (also where a row sees all of the unit's keys: the other quarters' zeros
          // have met the values that are not finite)
          const float probe = fmaf(y.x, 0.f, fmaf(y.y, 0.f, fmaf(y.z, 0.f, y.w * 0.f)));
          const uint32_t bad = __ballot_sync(0xffffffffu, there && probe != probe && r_l == r_l);
          if (bad != 0) {
            const int r_pos = x.pos + tok, z = p.causal ? min(r_pos + 1, x.kv) : x.kv;
            const int a = p.window > 0 ? max(0, r_pos - p.window + 1) : 0;
            // (a bit a row: its first lane's)
            const uint32_t again = kChunks == 32 ? 1u : ((bad & 0xffffu) != 0 ? 1u : 0u) | (bad >> 16 != 0 ? 0x10000u : 0u);
            anew(again, (int)r_t, r_head, dst, max(key0, a), min(key1, z), r_ref, r_f);
          }
        }
        fence_proxy_async_smem();  // the slot's next filling comes by TMA
      } else if (work) {
        constexpr int kChunks = D / 8;       // 16-byte pieces of a staged row: D bfloat16 or D / 2 float32
        constexpr int kAtOnce = 32 / kChunks;  // rows a warp stores with one instruction
        uint4* stage = reinterpret_cast<uint4*>(sRing + stage_at * L::kTileBytes) + (warp & 3) * 32 * kChunks;
        char* to = x.whole ? out : reinterpret_cast<char*>(part.out + prow * D);
        const uint32_t there = __ballot_sync(0xffffffffu, valid);
        uint64_t probe2 = 0;  // (two float32) NaN once a sum is not finite
#pragma unroll 1
        for (int pass = 0; pass < (x.whole ? 1 : 2); ++pass) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {  // four pieces a time
            uint4 y[4];
            if (x.whole) {
              uint32_t o[32];
              tmem_ld32_issue(tO + 32 * q, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int w = 0; w < 32; w += 2) {
                const uint64_t z = fma2(pack2(__uint_as_float(o[w]), __uint_as_float(o[w + 1])), pack2(f, f), 0);
                probe2 = fma2(z, 0, probe2);
                const float2 y2 = unpack2(z);
                o[w] = __float_as_uint(y2.x);
                o[w + 1] = __float_as_uint(y2.y);
              }
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const float* z = reinterpret_cast<const float*>(o + 8 * w);
                y[w] = make_uint4(to_bf16x2(z[0], z[1]), to_bf16x2(z[2], z[3]), to_bf16x2(z[4], z[5]), to_bf16x2(z[6], z[7]));
              }
            } else {
              uint32_t o[16];
              tmem_ld16_issue(tO + pass * (D / 2) + 16 * q, o);
              tmem_ld16_wait(o);
#pragma unroll
              for (int w = 0; w < 16; w += 2)
                probe2 = fma2(pack2(__uint_as_float(o[w]), __uint_as_float(o[w + 1])), 0, probe2);
#pragma unroll
              for (int w = 0; w < 4; ++w) y[w] = make_uint4(o[4 * w], o[4 * w + 1], o[4 * w + 2], o[4 * w + 3]);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) stage[lane * kChunks + ((4 * q + w) ^ (lane & 7))] = y[w];
          }
          __syncwarp();
          const int r0 = lane / kChunks, ch = lane % kChunks;
#pragma unroll 4
          for (int r = r0; r < 32; r += kAtOnce) {
            const uint4 y = stage[r * kChunks + (ch ^ (r & 7))];
            char* dst = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), r));
            if ((there >> r) & 1) reinterpret_cast<uint4*>(dst)[pass * kChunks + ch] = y;
          }
          __syncwarp();
        }
        const float2 probes = unpack2(probe2);
        const float probe = probes.x + probes.y;
        const uint32_t again = __ballot_sync(0xffffffffu, valid && probe != probe && l == l && (lo > key0 || hi < key1));
        if (again != 0) anew(again, (int)t_out, head, to, max(key0, lo), min(key1, hi), ref, f);
        if (valid) {
          if (!x.whole)
            part.stat[prow] = make_float2(ref, l);
          else if (lse != nullptr)
            *lse = some ? (ref + log2f(l)) * kLn2 : kNegInf;
        }
        fence_proxy_async_smem();  // the slot's next filling comes by TMA
      }
      __syncwarp();
      if (lane == 0) {
        __threadfence_block();
        if ((atomicAdd(&sh.staged[s], 1u) & 3u) == 3u) {
          __threadfence_block();
          mbar_arrive(&sh.empty[stage_at]);
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  // Each load has been waited for by an issuer, except after an abort: then wait
  // (with a limit) until nothing can be in flight when the CTA exits.
  if (watch->abort) {
    if (tid == 0) report(p.status, kErrTimeout);
    for (int i = 0; i < 64; ++i) __nanosleep(20000);
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int kForm>
cudaError_t prepare_kernel() {
  cudaError_t e =
      cudaFuncSetAttribute(attn_tc_kernel<D, kForm>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
  if (e != cudaSuccess) return e;
  // an increase of registers that the launch pool cannot satisfy would never return
  cudaFuncAttributes a;
  e = cudaFuncGetAttributes(&a, attn_tc_kernel<D, kForm>);
  if (e != cudaSuccess) return e;
  return a.numRegs == (int)kLaunchRegs ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int D, int kForm>
cudaError_t launch(const AttnParams& p, cudaStream_t s) {
  static Readiness readiness;
  const cudaError_t ready = readiness.get(prepare_kernel<D, kForm>);
  if (ready != cudaSuccess) return ready;
  CUtensorMap mq, mk, mv;
  const int per_tile = (kForm == kFew ? kFewRows : kTile) / p.group;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.n_heads, (cuuint64_t)p.T};
    const cuuint64_t str[2] = {(cuuint64_t)p.q_head, (cuuint64_t)p.q_token};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)per_tile};
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
  cudaError_t e = launch_early(attn_tc_kernel<D, kForm>, dim3(kMaxAttnCtas), dim3(kThreads), Layout<D>::kBytes, s, p, mq,
                               mk, mv);
  if (e != cudaSuccess) return e;
  using F = Form<kForm>;
  const int rows = p.max_q <= per_tile ? p.max_q * p.group : F::kPartRows;
  return launch_join<F, D, __nv_bfloat16>(p, s, rows, kForm == kFew ? kFewRows : kTile, per_tile * p.group);
}

}  // namespace

cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t s) {
  // Two row tiles a unit if the requests fill more than one on average. 128 requests
  // of 136 rows each: pair 258 us, solo 386; of 8 to 136 rows: 236 and 216.
  // Few rows against solo: 128 requests of 4 rows, 300 to 8000 cached 193 us (6.4 TB/s)
  // and 197, D = 64 158 and 164; 512 of 2 rows, 1 to 300 cached 63 and 85; 64 of 16 rows
  // 111 and 113. (The quarters' sums of 16 rows fill the staging slot.)
  const int per_tile = kTile / p.group;
  const bool pair = p.max_q > per_tile && p.T > (int64_t)p.B * per_tile;
  const bool few = (int64_t)p.max_q * p.group <= kFewRows;
  if (p.D == 128) return few ? launch<128, kFew>(p, s) : pair ? launch<128, kPairs>(p, s) : launch<128, kSolo>(p, s);
  return few ? launch<64, kFew>(p, s) : pair ? launch<64, kPairs>(p, s) : launch<64, kSolo>(p, s);
}

}  // namespace ds
