// Attention of ragged rows over the paged cache in float32, on the CUDA cores.
//
//   s_j = scale * (q . k_j),  out = sum_j 2^(c s'_j - r) v_j / l,  l = sum_j 2^(c s'_j - r),
// with s' = q . k, c = scale * log2(e) and r the running maximum of c s', in one
// pass over the keys. The float32 cache is for small models and for checking the
// bfloat16 one: its products stay float32 (the tensor cores would round them).
//
// Units, shares and the join are those of attn_work.cuh with tiles of 64 keys. A
// block of 256 threads is a 16 x 16 grid: thread (ty, tx) has the scores of kRM
// rows and of the keys tx, tx + 16, tx + 32, tx + 48, so that a row's 64 scores
// lie in half a warp (its maximum and sum are shuffles, and its weights go through
// shared memory with a warp barrier only), and then the same rows' outputs in D / 16
// columns. With 4 x 4 scores a thread, 16 products follow each two 16-byte loads
// from shared memory. K of the next tile arrives (cp.async) during the product
// with V, V of this one during the scores.
#include "attn_work.cuh"

namespace ds {
namespace {

constexpr int kThreads = 256;
constexpr int kKeyTile = 64;

template <int kBM>
struct Form32 : WorkForm<kKeyTile, kMaxShares, kBM> {};

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

template <int D, int kBM>
__global__ void __launch_bounds__(kThreads) attn_f32_kernel(const AttnParams p) {
  using F = Form32<kBM>;
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
#pragma unroll
    for (int i = 0; i < kRM; ++i) {
      const int row = ty * kRM + i, at = x.off + row, tok = p.by_group.quotient(at);
      const int head = x.h * p.group + at - tok * p.group, pos = x.pos + tok;
      valid[i] = row < x.rows;
      hi[i] = !valid[i] ? 0 : p.causal ? min(pos + 1, x.kv) : x.kv;
      lo[i] = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const int64_t t = x.token + tok;
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
    // places of a tile's keys (by the first 64 threads)
    auto find = [&](int j) {
      if (tid < kKeyTile) {
        const int key = (x.tile0 + j) * kKeyTile + tid;
        int64_t at = -1;
        if (key >= x.lo && key < x.hi) {
          int page = __ldg(table + (key >> shift));
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
          s[i][k] = key >= lo[i] && key < hi[i] ? s[i][k] * c : kNegInf;
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
      // what it sees (each thread its columns).
      float probe = 0.f;
#pragma unroll
      for (int k = 0; k < kC; ++k)
        probe = fmaf(o[i][k].x, 0.f, fmaf(o[i][k].y, 0.f, fmaf(o[i][k].z, 0.f, fmaf(o[i][k].w, 0.f, probe))));
      if (valid[i] && probe != probe && l[i] == l[i] && (lo[i] > key0 || hi[i] < key1)) {
#pragma unroll
        for (int k = 0; k < kC; ++k) o[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        const float ref = m[i] == kNegInf ? 0.f : m[i];
#pragma unroll 1
        for (int key = max(key0, lo[i]); key < min(key1, hi[i]); ++key) {
          const int page = __ldg(table + (key >> shift));
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

template <int D, int kBM>
cudaError_t launch(const AttnParams& p, cudaStream_t s) {
  using F = Form32<kBM>;
  static const cudaError_t ready = cudaFuncSetAttribute(
      attn_f32_kernel<D, kBM>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Tiles<D, kBM>));
  if (ready != cudaSuccess) return ready;
  const cudaError_t e =
      launch_early(attn_f32_kernel<D, kBM>, dim3(F::kShares), dim3(kThreads), sizeof(Tiles<D, kBM>), s, p);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)p.max_q * p.group;
  return launch_early(attn_join_kernel<F, D, float>, dim3(F::kShares, (unsigned)(((most < kBM ? most : kBM) + 7) / 8)),
                      dim3(256), 0, s, p, kBM, kBM);
}

}  // namespace

size_t attention_ws_bytes(int32_t dtype, int32_t D) {
  (void)dtype;
  // a record a share, and rows of partial results: D sums, reference and sum
  return (size_t)kMaxShares * 64 + (size_t)kRows * (D + 2) * sizeof(float);
}

cudaError_t launch_attention_f32(const AttnParams& p, cudaStream_t s) {
  const bool few = (int64_t)p.max_q * p.group <= 16;
  if (p.D == 128) return few ? launch<128, 16>(p, s) : launch<128, 64>(p, s);
  return few ? launch<64, 16>(p, s) : launch<64, 64>(p, s);
}

}  // namespace ds
