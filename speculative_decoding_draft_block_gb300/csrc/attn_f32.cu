// Attention of ragged rows over the paged cache in float32, on the CUDA cores.
//
//   s_j = scale * (q . k_j),  out = sum_j 2^(c s'_j - r) v_j / l,  l = sum_j 2^(c s'_j - r),
// with s' = q . k, c = scale * log2(e) and r the running maximum of c s', in one
// pass over the keys. The float32 cache is for small models and for checking the
// bfloat16 one: its products stay float32 (the tensor cores would round them).
//
// Two forms, by the rows of a unit: few rows (below) and tiles of 16 or 64 rows.
// Units, shares and the join are those of attn_work.cuh with tiles of 64 keys. For
// tiles of rows a block of 256 threads is a 16 x 16 grid: thread (ty, tx) has the
// scores of kRM rows and of the keys tx, tx + 16, tx + 32, tx + 48, so that a row's
// 64 scores lie in half a warp (its maximum and sum are shuffles, and its weights go
// through shared memory with a warp barrier only), and then the same rows' outputs
// in D / 16 columns. With 4 x 4 scores a thread, 16 products follow each two 16-byte loads
// from shared memory. K of the next tile arrives (cp.async) during the product
// with V, V of this one during the scores.
#include "attn_work.cuh"

namespace ds {
namespace {

constexpr int kThreads = 256;
constexpr int kKeyTile = kAttnTileF32;

template <int kBM, bool kTree>
struct Form32 : WorkForm<kKeyTile, kMaxShares, kBM, kTree> {
  static_assert(Form32::kCost == kAttnUnitCost, "work_fits");
};

template <int D, int kBM>
struct Tiles {
  float q[kBM][D + 4];  // rows padded by 16 bytes: 16-byte reads of 8 rows touch all banks once
  float k[kKeyTile][D + 4];
  float v[kKeyTile][D];
  float w[kBM][kKeyTile + 4];
  int64_t place[2][kKeyTile];  // byte offset of a key's row in the pool, -1: unseen
  ShareStart<kThreads, 1> work;
};

// 16 bytes to shared memory, zeros if `from` is null.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  const uint32_t n = from != nullptr ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(to)), "l"(from), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int kBM, bool kTree>
__global__ void __launch_bounds__(kThreads) attn_f32_kernel(const AttnParams p) {
  using F = Form32<kBM, kTree>;
  constexpr int kRM = kBM / 16;      // rows of a thread
  constexpr int kC = D / 64;         // float4 output columns of a thread
  extern __shared__ __align__(16) uint8_t smem[];
  Tiles<D, kBM>& sh = *reinterpret_cast<Tiles<D, kBM>*>(smem);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Partials part = partials<D>(p.workspace);
  const int share = blockIdx.x;
  sm100::pdl_wait();
  const int64_t total = locate_shares<F, kThreads, 1>(p, kBM, share, sh.work);
  if (tid == 0) part.cut[share].valid = 0;
  sm100::pdl_launch_dependents();
  const int64_t begin = F::begin(total, share), end = F::begin(total, share + 1);
  if (begin >= end) return;
  const float c = p.scale * kLog2eHi;
  const int shift = p.pool.page_shift, mask = (1 << shift) - 1;
  Walk<F> wk;
  wk.start(begin, end, sh.work, 0);
  while (true) {
    const Piece x = wk.next(p, kBM, tid == 0 ? part.cut + share : nullptr, total);
    if (x.n < 0) break;
    // this thread's rows
    int lo[kRM], hi[kRM];
    char* out[kRM];
    float* lse[kRM];
    bool valid[kRM];
    const uint32_t* words[kRM];  // (a tree's rows: hi is the context's end)
#pragma unroll
    for (int i = 0; i < kRM; ++i) {
      const int row = ty * kRM + i, at = x.off + row, tok = p.by_group.quotient(at);
      const int head = x.h * p.group + at - tok * p.group, pos = x.pos + tok;
      valid[i] = row < x.rows;
      hi[i] = !valid[i] ? 0 : p.causal ? min(pos + 1, x.kv) : x.kv;
      lo[i] = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const int64_t t = x.token + tok;
      words[i] = nullptr;
      if (kTree && valid[i]) {
        words[i] = p.mask + t * p.mask_words;
        hi[i] = x.ctx;
        lo[i] = tree_low(p, x.ctx, t);
      }
      out[i] = p.out + t * p.o_token + head * p.o_head;
      lse[i] = p.lse != nullptr ? p.lse + t * p.n_heads + head : nullptr;
    }
    if (x.n == 0) {
#pragma unroll
      for (int i = 0; i < kRM; ++i)
        if (valid[i]) {
          for (int d = tx; d < D / 4; d += 16) reinterpret_cast<float4*>(out[i])[d] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (tx == 0 && lse[i] != nullptr) *lse[i] = kNegInf;
        }
      continue;
    }
    const int32_t* table = p.block_table + (int64_t)x.b * p.max_pages;
    auto sees = [&](int i, int key) {
      if (key >= lo[i] && key < hi[i]) return true;
      return kTree && valid[i] && key >= x.ctx && key >= 0 && key < x.kv && tree_sees(words[i], key, x.ctx);
    };
    // places of a tile's keys (by the first 64 threads)
    auto find = [&](int j) {
      if (tid < kKeyTile) {
        const int key = (x.tile0 + j) * kKeyTile + tid;
        int64_t at = -1;
        if (key >= x.lo && key < x.hi) {
          int page = __ldcg(table + (key >> shift));
          if (page < 0 || page >= p.pool.n_pages) {
            report(p.status, kErrBounds);
            page = 0;
          }
          at = (int64_t)page * p.pool.page_stride + x.h * p.pool.head_stride + (int64_t)(key & mask) * p.pool.token_stride;
        }
        sh.place[j & 1][tid] = at;
      }
    };
    auto load = [&](const char* base, int j, float* to, int stride) {
#pragma unroll 4
      for (int i = tid; i < kKeyTile * (D / 4); i += kThreads) {
        const int key = i / (D / 4), d = i - key * (D / 4);
        const int64_t at = sh.place[j & 1][key];
        copy16(to + key * stride + d * 4, at < 0 ? nullptr : base + at + d * 16);
      }
      copies_commit();
    };
    // (the tiles of the piece before are no longer read: its last barrier)
    find(0);
    for (int i = tid; i < kBM * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d = i - row * (D / 4);
      const int at = x.off + row, tok = p.by_group.quotient(at);
      const char* from = p.q + (int64_t)(x.token + tok) * p.q_token + (int64_t)(x.h * p.group + at - tok * p.group) * p.q_head;
      copy16(&sh.q[row][d * 4], row < x.rows ? from + d * 16 : nullptr);
    }
    __syncthreads();
    load(p.pool.k, 0, &sh.k[0][0], D + 4);  // (Q in the same group)
    load(p.pool.v, 0, &sh.v[0][0], D);
    float m[kRM], l[kRM];
    float4 o[kRM][kC];
#pragma unroll
    for (int i = 0; i < kRM; ++i) {
      m[i] = kNegInf;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kC; ++k) o[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int j = 0; j < x.n; ++j) {
      copies_wait<1>();  // K of this tile; its V may be on the way
      if (j + 1 < x.n) find(j + 1);
      __syncthreads();
      float s[kRM][4];
#pragma unroll
      for (int i = 0; i < kRM; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 kk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) kk[k] = *reinterpret_cast<const float4*>(&sh.k[tx + 16 * k][d]);
#pragma unroll
        for (int i = 0; i < kRM; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(&sh.q[ty * kRM + i][d]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            s[i][k] = fmaf(q.x, kk[k].x, fmaf(q.y, kk[k].y, fmaf(q.z, kk[k].z, fmaf(q.w, kk[k].w, s[i][k]))));
        }
      }
      __syncthreads();  // K is read
      if (j + 1 < x.n)
        load(p.pool.k, j + 1, &sh.k[0][0], D + 4);
      else
        copies_commit();
      const int key0 = (x.tile0 + j) * kKeyTile + tx;
#pragma unroll
      for (int i = 0; i < kRM; ++i) {
        float top = m[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = key0 + 16 * k;
          s[i][k] = sees(i, key) ? s[i][k] * c : kNegInf;
          top = fmaxf(top, s[i][k]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float ref = top == kNegInf ? 0.f : top;
        const float f = m[i] == kNegInf ? 0.f : ex2_approx(m[i] - ref);
        m[i] = top;
        l[i] *= f;
#pragma unroll
        for (int k = 0; k < kC; ++k) {
          o[i][k].x *= f;
          o[i][k].y *= f;
          o[i][k].z *= f;
          o[i][k].w *= f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float w = ex2_approx(s[i][k] - ref);
          l[i] += w;
          sh.w[ty * kRM + i][tx + 16 * k] = w;
        }
      }
      copies_wait<1>();  // V of this tile; the next K may be on the way
      __syncthreads();
#pragma unroll 2
      for (int k4 = 0; k4 < kKeyTile; k4 += 4) {
        float4 w[kRM];
#pragma unroll
        for (int i = 0; i < kRM; ++i) w[i] = *reinterpret_cast<const float4*>(&sh.w[ty * kRM + i][k4]);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
#pragma unroll
          for (int k = 0; k < kC; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(&sh.v[k4 + y][tx * 4 + 64 * k]);
#pragma unroll
            for (int i = 0; i < kRM; ++i) {
              const float f = y == 0 ? w[i].x : y == 1 ? w[i].y : y == 2 ? w[i].z : w[i].w;
              o[i][k].x = fmaf(f, v.x, o[i][k].x);
              o[i][k].y = fmaf(f, v.y, o[i][k].y);
              o[i][k].z = fmaf(f, v.z, o[i][k].z);
              o[i][k].w = fmaf(f, v.w, o[i][k].w);
            }
          }
        }
      }
      __syncthreads();  // V is read
      if (j + 1 < x.n)
        load(p.pool.v, j + 1, &sh.v[0][0], D);
      else
        copies_commit();
    }
    copies_wait<0>();
    const int key0 = max(x.lo, x.tile0 * kKeyTile), key1 = min(x.hi, (x.tile0 + x.n) * kKeyTile);
#pragma unroll
    for (int i = 0; i < kRM; ++i) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      // A value that is not finite, of a key that other rows of the unit see and this
      // one does not, has come in with its weight of zero: the row's sums again, from
      // what it sees (each thread its columns; of a tree's new tokens the window hides none).
      float probe = 0.f;
#pragma unroll
      for (int k = 0; k < kC; ++k)
        probe = fmaf(o[i][k].x, 0.f, fmaf(o[i][k].y, 0.f, fmaf(o[i][k].z, 0.f, fmaf(o[i][k].w, 0.f, probe))));
      if (valid[i] && probe != probe && l[i] == l[i] && (lo[i] > key0 || hi[i] < key1)) {
#pragma unroll
        for (int k = 0; k < kC; ++k) o[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        const float ref = m[i] == kNegInf ? 0.f : m[i];
#pragma unroll 1
        for (int key = max(key0, kTree ? min(lo[i], x.ctx) : lo[i]); key < min(key1, kTree ? x.kv : hi[i]); ++key) {
          if (kTree && !sees(i, key)) continue;
          const int page = __ldcg(table + (key >> shift));
          if (page < 0 || page >= p.pool.n_pages) break;  // (reported above)
          const int64_t at = (int64_t)page * p.pool.page_stride + x.h * p.pool.head_stride + (int64_t)(key & mask) * p.pool.token_stride;
          const float* kk = reinterpret_cast<const float*>(p.pool.k + at);
          const float* vv = reinterpret_cast<const float*>(p.pool.v + at);
          float s = 0.f;
#pragma unroll 1
          for (int d = 0; d < D; ++d) s = fmaf(sh.q[ty * kRM + i][d], kk[d], s);
          const float w = ex2_approx(s * c - ref);
#pragma unroll
          for (int k = 0; k < kC; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(vv + tx * 4 + 64 * k);
            o[i][k].x = fmaf(w, v.x, o[i][k].x);
            o[i][k].y = fmaf(w, v.y, o[i][k].y);
            o[i][k].z = fmaf(w, v.z, o[i][k].z);
            o[i][k].w = fmaf(w, v.w, o[i][k].w);
          }
        }
      }
      if (!valid[i]) continue;
      const bool some = l[i] > 0.f || l[i] != l[i];
      const float f = !x.whole ? 1.f : some ? 1.f / l[i] : 0.f;
      const size_t prow = (size_t)(share * 2 + x.slot) * F::kPartRows + ty * kRM + i;
      float* to = x.whole ? reinterpret_cast<float*>(out[i]) : part.out + prow * D;
#pragma unroll
      for (int k = 0; k < kC; ++k)
        *reinterpret_cast<float4*>(to + tx * 4 + 64 * k) =
            make_float4(o[i][k].x * f, o[i][k].y * f, o[i][k].z * f, o[i][k].w * f);
      if (tx == 0) {
        if (!x.whole)
          part.stat[prow] = make_float2(m[i], l[i]);
        else if (lse[i] != nullptr)
          *lse[i] = some ? (m[i] + log2f(l[i])) * kLn2 : kNegInf;
      }
    }
    __syncthreads();  // Q is read
  }
}

// ---- few rows --------------------------------------------------------------------------
//
// Units of up to kR rows (single tokens, short blocks), bound by the keys' way from
// memory. In the form above sixteen threads read each key and each value; here a
// key belongs to four threads (a quarter of its dimensions each, for all rows), and
// in the value product a thread has four columns of every eighth (sixteenth) group
// of keys, so that each is read from shared memory once. The groups' sums are added
// up at the end of a piece. A warp keeps the maximum and the sum of row w. Two blocks
// an SM hide each other's waits, so registers are held to 128 (with 144, 8 rows of
// D = 64 ran one block an SM: 271 us for 179). Times: see launch_rows.

template <int D, int kR>
struct FewTiles {
  float q[kR][D];
  float k[kKeyTile][D + 16];  // two keys' quarters touch all banks once
  float v[kKeyTile][D];       // (after a piece's last tile k and v hold the groups' sums)
  float s[kR][kKeyTile];      // scores, then weights
  float f[kR];                // factor of a row's sums
  float2 stat[kR];
  int lo[kR], hi[kR];
  int64_t place[2][kKeyTile];
  ShareStart<kThreads, 1> work;
};

template <int D, int kR, bool kTree>
__global__ void __launch_bounds__(kThreads, 2) attn_f32_few_kernel(const AttnParams p) {
  using F = Form32<kR, kTree>;
  constexpr int kCols = D / 4;                // threads across a row of values
  constexpr int kGroups = kThreads / kCols;   // groups of keys in the value product
  constexpr int kGroupKeys = kKeyTile / kGroups;
  constexpr int kWarps = kThreads / 32;
  static_assert(kR <= kWarps && kWarps * kR * D * 4 <= (int)(sizeof(float) * kKeyTile * (2 * D + 16)), "sums of the warps");
  extern __shared__ __align__(16) uint8_t smem[];
  FewTiles<D, kR>& sh = *reinterpret_cast<FewTiles<D, kR>*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = tid % kCols, group = tid / kCols;
  const int my_key = tid >> 2, part4 = tid & 3;
  const Partials part = partials<D>(p.workspace);
  const int share = blockIdx.x;
  sm100::pdl_wait();
  const int64_t total = locate_shares<F, kThreads, 1>(p, kR, share, sh.work);
  if (tid == 0) part.cut[share].valid = 0;
  sm100::pdl_launch_dependents();
  const int64_t begin = F::begin(total, share), end = F::begin(total, share + 1);
  if (begin >= end) return;
  const float c = p.scale * kLog2eHi;
  const int shift = p.pool.page_shift, mask = (1 << shift) - 1;
  Walk<F> wk;
  wk.start(begin, end, sh.work, 0);
  while (true) {
    const Piece x = wk.next(p, kR, tid == 0 ? part.cut + share : nullptr, total);
    if (x.n < 0) break;
    const int32_t* table = p.block_table + (int64_t)x.b * p.max_pages;
    auto head_of = [&](int row, int64_t& t) {  // query head of a row, and its row of q
      const int at = x.off + row, tok = p.by_group.quotient(at);
      t = x.token + tok;
      return x.h * p.group + at - tok * p.group;
    };
    if (x.n == 0) {
      for (int i = tid; i < x.rows * kCols; i += kThreads) {
        int64_t t;
        const int row = i / kCols, head = head_of(row, t);
        reinterpret_cast<float4*>(p.out + t * p.o_token + head * p.o_head)[i % kCols] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i % kCols == 0 && p.lse != nullptr) p.lse[t * p.n_heads + head] = kNegInf;
      }
      continue;
    }
    auto find = [&](int j) {
      if (tid < kKeyTile) {
        const int key = (x.tile0 + j) * kKeyTile + tid;
        int64_t at = -1;
        if (key >= x.lo && key < x.hi) {
          int page = __ldcg(table + (key >> shift));
          if (page < 0 || page >= p.pool.n_pages) {
            report(p.status, kErrBounds);
            page = 0;
          }
          at = (int64_t)page * p.pool.page_stride + x.h * p.pool.head_stride + (int64_t)(key & mask) * p.pool.token_stride;
        }
        sh.place[j & 1][tid] = at;
      }
    };
    auto load = [&](const char* base, int j, float* to, int stride) {
#pragma unroll 4
      for (int i = tid; i < kKeyTile * kCols; i += kThreads) {
        const int key = i / kCols, d = i % kCols;
        const int64_t at = sh.place[j & 1][key];
        copy16(to + key * stride + d * 4, at < 0 ? nullptr : base + at + d * 16);
      }
      copies_commit();
    };
    // (a tree's rows: hi is the context's end)
    auto sees = [&](int row, int key) {
      if (key >= sh.lo[row] && key < sh.hi[row]) return true;
      if (!kTree || row >= x.rows || key < x.ctx || key < 0 || key >= x.kv) return false;
      const int64_t t = x.token + p.by_group.quotient(x.off + row);
      return tree_sees(p.mask + t * p.mask_words, key, x.ctx);
    };
    find(0);
    if (tid < kR) {
      const int tok = p.by_group.quotient(x.off + tid), pos = x.pos + tok;
      sh.hi[tid] = tid >= x.rows ? 0 : kTree ? x.ctx : p.causal ? min(pos + 1, x.kv) : x.kv;
      sh.lo[tid] = kTree ? (tid < x.rows ? tree_low(p, x.ctx, x.token + tok) : 0) : p.window > 0 ? max(0, pos - p.window + 1) : 0;
    }
    for (int i = tid; i < kR * kCols; i += kThreads) {
      int64_t t;
      const int row = i / kCols, head = head_of(row, t);
      copy16(&sh.q[row][(i % kCols) * 4], row < x.rows ? p.q + t * p.q_token + head * p.q_head + (i % kCols) * 16 : nullptr);
    }
    __syncthreads();
    load(p.pool.k, 0, &sh.k[0][0], D + 16);  // (Q in the same group)
    load(p.pool.v, 0, &sh.v[0][0], D);
    float m = kNegInf, l = 0.f;  // of row `warp`
    float4 o[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < x.n; ++j) {
      copies_wait<1>();  // K of this tile
      if (j + 1 < x.n) find(j + 1);
      __syncthreads();
      {
        float s[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) s[r] = 0.f;
#pragma unroll 4
        for (int d = part4 * 4; d < D; d += 16) {
          const float4 kk = *reinterpret_cast<const float4*>(&sh.k[my_key][d]);
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const float4 q = *reinterpret_cast<const float4*>(&sh.q[r][d]);
            s[r] = fmaf(q.x, kk.x, fmaf(q.y, kk.y, fmaf(q.z, kk.z, fmaf(q.w, kk.w, s[r]))));
          }
        }
        const int key = (x.tile0 + j) * kKeyTile + my_key;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          s[r] += __shfl_xor_sync(0xffffffffu, s[r], 1);
          s[r] += __shfl_xor_sync(0xffffffffu, s[r], 2);
          if ((r & 3) == part4) sh.s[r][my_key] = sees(r, key) ? s[r] * c : kNegInf;
        }
      }
      __syncthreads();  // scores are there, K is read
      if (j + 1 < x.n)
        load(p.pool.k, j + 1, &sh.k[0][0], D + 16);
      else
        copies_commit();
      if (warp < kR) {
        const float a = sh.s[warp][lane], b = sh.s[warp][lane + 32];
        float top = fmaxf(m, fmaxf(a, b));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float ref = top == kNegInf ? 0.f : top;
        const float f = m == kNegInf ? 0.f : ex2_approx(m - ref);
        m = top;
        const float wa = ex2_approx(a - ref), wb = ex2_approx(b - ref);
        l = fmaf(l, f, wa + wb);
        sh.s[warp][lane] = wa;
        sh.s[warp][lane + 32] = wb;
        if (lane == 0) sh.f[warp] = f;
      }
      copies_wait<1>();  // V of this tile
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const float f = sh.f[r];
        o[r].x *= f;
        o[r].y *= f;
        o[r].z *= f;
        o[r].w *= f;
      }
#pragma unroll
      for (int k4 = 0; k4 < kGroupKeys; k4 += 4) {
        float4 v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) v[y] = *reinterpret_cast<const float4*>(&sh.v[group * kGroupKeys + k4 + y][col * 4]);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const float4 w = *reinterpret_cast<const float4*>(&sh.s[r][group * kGroupKeys + k4]);
          o[r].x = fmaf(w.x, v[0].x, fmaf(w.y, v[1].x, fmaf(w.z, v[2].x, fmaf(w.w, v[3].x, o[r].x))));
          o[r].y = fmaf(w.x, v[0].y, fmaf(w.y, v[1].y, fmaf(w.z, v[2].y, fmaf(w.w, v[3].y, o[r].y))));
          o[r].z = fmaf(w.x, v[0].z, fmaf(w.y, v[1].z, fmaf(w.z, v[2].z, fmaf(w.w, v[3].z, o[r].z))));
          o[r].w = fmaf(w.x, v[0].w, fmaf(w.y, v[1].w, fmaf(w.z, v[2].w, fmaf(w.w, v[3].w, o[r].w))));
        }
      }
      __syncthreads();  // V and the weights are read
      if (j + 1 < x.n)
        load(p.pool.v, j + 1, &sh.v[0][0], D);
      else
        copies_commit();
    }
    copies_wait<0>();
    // the warps' sums to shared memory
    float* sums = &sh.k[0][0];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      if (kCols == 16) {  // two groups of keys in a warp
        o[r].x += __shfl_xor_sync(0xffffffffu, o[r].x, 16);
        o[r].y += __shfl_xor_sync(0xffffffffu, o[r].y, 16);
        o[r].z += __shfl_xor_sync(0xffffffffu, o[r].z, 16);
        o[r].w += __shfl_xor_sync(0xffffffffu, o[r].w, 16);
      }
      if (lane < kCols) *reinterpret_cast<float4*>(sums + (warp * kR + r) * D + lane * 4) = o[r];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (warp < kR && lane == 0) sh.stat[warp] = make_float2(m, l);
    __syncthreads();
    const int key0 = max(x.lo, x.tile0 * kKeyTile), key1 = min(x.hi, (x.tile0 + x.n) * kKeyTile);
    for (int i = tid; i < x.rows * kCols; i += kThreads) {
      const int row = i / kCols, d = i % kCols;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(sums + (w * kR + row) * D + d * 4);
        y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
      }
      const float2 st = sh.stat[row];
      const float probe = fmaf(y.x, 0.f, fmaf(y.y, 0.f, fmaf(y.z, 0.f, y.w * 0.f)));
      if (probe != probe && st.y == st.y && (sh.lo[row] > key0 || sh.hi[row] < key1)) {
        // (values that are not finite and that this row does not see, as above)
        y = make_float4(0.f, 0.f, 0.f, 0.f);
        const float ref = st.x == kNegInf ? 0.f : st.x;
#pragma unroll 1
        for (int key = max(key0, kTree ? min(sh.lo[row], x.ctx) : sh.lo[row]); key < min(key1, kTree ? x.kv : sh.hi[row]); ++key) {
          if (kTree && !sees(row, key)) continue;
          const int page = __ldcg(table + (key >> shift));
          if (page < 0 || page >= p.pool.n_pages) break;
          const int64_t at = (int64_t)page * p.pool.page_stride + x.h * p.pool.head_stride + (int64_t)(key & mask) * p.pool.token_stride;
          const float* kk = reinterpret_cast<const float*>(p.pool.k + at);
          float s = 0.f;
#pragma unroll 1
          for (int e = 0; e < D; ++e) s = fmaf(sh.q[row][e], kk[e], s);
          const float w = ex2_approx(s * c - ref);
          const float4 v = reinterpret_cast<const float4*>(p.pool.v + at)[d];
          y = make_float4(fmaf(w, v.x, y.x), fmaf(w, v.y, y.y), fmaf(w, v.z, y.z), fmaf(w, v.w, y.w));
        }
      }
      const bool some = st.y > 0.f || st.y != st.y;
      const float f = !x.whole ? 1.f : some ? 1.f / st.y : 0.f;
      int64_t t;
      const int head = head_of(row, t);
      const size_t prow = (size_t)(share * 2 + x.slot) * F::kPartRows + row;
      float* to = x.whole ? reinterpret_cast<float*>(p.out + t * p.o_token + head * p.o_head) : part.out + prow * D;
      reinterpret_cast<float4*>(to)[d] = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
      if (d == 0) {
        if (!x.whole)
          part.stat[prow] = st;
        else if (p.lse != nullptr)
          p.lse[t * p.n_heads + head] = some ? (st.x + log2f(st.y)) * kLn2 : kNegInf;
      }
    }
    __syncthreads();  // the sums and Q are read
  }
}

// A form of the kernel with its shared memory, and the join of its cut units.
template <int D, int kBM, bool kTree>
cudaError_t launch(const AttnParams& p, cudaStream_t s, void (*kernel)(AttnParams), size_t smem, Readiness& readiness) {
  using F = Form32<kBM, kTree>;
  cudaError_t e = readiness.get(
      [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); });
  if (e != cudaSuccess) return e;
  e = launch_early(kernel, dim3(F::kShares), dim3(kThreads), smem, s, p);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)p.max_q * p.group;
  return launch_join<F, D, float>(p, s, (int)(most < kBM ? most : kBM), kBM, kBM);
}

template <int D, int kR, bool kTree>
cudaError_t launch_few(const AttnParams& p, cudaStream_t s) {
  static Readiness readiness;
  return launch<D, kR, kTree>(p, s, attn_f32_few_kernel<D, kR, kTree>, sizeof(FewTiles<D, kR>), readiness);
}

template <int D, int kBM, bool kTree>
cudaError_t launch_tiles(const AttnParams& p, cudaStream_t s) {
  static Readiness readiness;
  return launch<D, kBM, kTree>(p, s, attn_f32_kernel<D, kBM, kTree>, sizeof(Tiles<D, kBM>), readiness);
}

// Measured on 64 requests of one token over 500 to 4000 cached, 8 KV heads (D = 128:
// 0.89 GB, D = 64: 0.45 GB), few rows against tiles of 16: 4 rows 204 us (4.4 TB/s)
// against 482, D = 64 129 against 268; 8 rows 277 against 482, D = 64 179 against 268;
// 16 rows 432 against 482, but D = 64 278 against 269 and 10 rows over 33 to 1000
// cached 15.7 against 14.2: the sums of 16 rows do not leave two blocks an SM enough
// registers. Tiles of 64 rows take the rest: prompt chunks of 512 tokens 36 TFLOP/s.
template <int D, bool kTree>
cudaError_t launch_rows(const AttnParams& p, cudaStream_t s) {
  const int64_t rows = (int64_t)p.max_q * p.group;  // of the longest request, per KV head
  return rows <= 4    ? launch_few<D, 4, kTree>(p, s)
         : rows <= 8  ? launch_few<D, 8, kTree>(p, s)
         : rows <= 16 ? launch_tiles<D, 16, kTree>(p, s)
                      : launch_tiles<D, 64, kTree>(p, s);
}

}  // namespace

size_t attention_ws_bytes(int32_t D) {
  // a record a share, and rows of partial results: D sums, reference and sum
  return (size_t)kMaxShares * 64 + (size_t)kRows * (D + 2) * sizeof(float);
}

cudaError_t launch_attention_f32(const AttnParams& p, cudaStream_t s) {
  if (p.mask != nullptr) return p.D == 128 ? launch_rows<128, true>(p, s) : launch_rows<64, true>(p, s);
  return p.D == 128 ? launch_rows<128, false>(p, s) : launch_rows<64, false>(p, s);
}

}  // namespace ds
