// Attention over the paged cache on the CUDA cores: one warp a query row.
//
//   s_j = scale * (q . k_j),  m = max s_j,  l = sum 2^(s_j log2e - m log2e),
//   out = sum 2^(..) v_j / l,  lse = m + ln l
// in one pass over the row's keys with the running maximum and sum.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv_internal.h"

namespace ds {
namespace {

template <typename T, int N>
__device__ __forceinline__ void load_row(const char* p, int lane, float (&o)[N]) {
  const T* x = reinterpret_cast<const T*>(p) + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = to_f32<T>(x[i]);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <typename T, int D>
__global__ void __launch_bounds__(128) attn_rows_kernel(const AttnParams p) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z, h = blockIdx.y, i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t cap = (int64_t)p.max_pages << p.pool.page_shift;
  const Request r = load_request(p.q_start, p.kv_len, b, p.T, p.max_q, cap);
  if (!r.ok) report(p.status, kErrBounds);
  if (i >= r.n) return;
  const int64_t t = r.q0 + i;
  const int pos = r.kv - r.n + i;
  const int hi = p.causal ? min(pos + 1, r.kv) : r.kv;
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const float c = p.scale * kLog2eHi;
  float q[N], acc[N], x[N];
  load_row<T>(p.q + t * p.q_token + h * p.q_head, lane, q);
#pragma unroll
  for (int d = 0; d < N; ++d) acc[d] = 0.f;
  float m = kNegInf, l = 0.f;
  const int32_t* row = p.block_table + (int64_t)b * p.max_pages;
  const int64_t head = (int64_t)(h / p.group) * p.pool.head_stride;
  for (int j = lo; j < hi; ++j) {
    const int page = __ldg(row + (j >> p.pool.page_shift));
    if (page < 0 || page >= p.pool.n_pages) {
      report(p.status, kErrBounds);
      break;
    }
    const int64_t off = (int64_t)page * p.pool.page_stride + head +
                        (int64_t)(j & ((1 << p.pool.page_shift) - 1)) * p.pool.token_stride;
    load_row<T>(p.pool.k + off, lane, x);
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < N; ++d) s = fmaf(q[d], x[d], s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= c;
    const float m1 = fmaxf(m, s);
    const float a = m1 == kNegInf ? 1.f : exp2f(m - m1);
    const float w = m1 == kNegInf ? 0.f : exp2f(s - m1);
    load_row<T>(p.pool.v + off, lane, x);
    l = fmaf(l, a, w);
#pragma unroll
    for (int d = 0; d < N; ++d) acc[d] = fmaf(acc[d], a, w * x[d]);
    m = m1;
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  T* o = reinterpret_cast<T*>(p.out + t * p.o_token + h * p.o_head) + lane * N;
#pragma unroll
  for (int d = 0; d < N; ++d) o[d] = from_f32<T>(acc[d] * inv);
  if (p.lse != nullptr && lane == 0)
    p.lse[t * p.n_heads + h] = l > 0.f || l != l ? (m + log2f(l)) * 0.693147180559945f : kNegInf;
}

}  // namespace

cudaError_t launch_attention_simt(const AttnParams& p, cudaStream_t s) {
  const dim3 grid((p.max_q + 3) / 4, p.n_heads, p.B);
  const bool bf = p.dtype == DS_BF16;
  if (p.D == 128) {
    if (bf)
      attn_rows_kernel<__nv_bfloat16, 128><<<grid, 128, 0, s>>>(p);
    else
      attn_rows_kernel<float, 128><<<grid, 128, 0, s>>>(p);
  } else {
    if (bf)
      attn_rows_kernel<__nv_bfloat16, 64><<<grid, 128, 0, s>>>(p);
    else
      attn_rows_kernel<float, 64><<<grid, 128, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace ds
