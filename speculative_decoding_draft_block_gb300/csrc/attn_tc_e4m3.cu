// The attention kernels of attn_tc.cuh for quantised pools, rows in sequence or of trees.
#include "attn_tc.cuh"

namespace ds {

cudaError_t launch_attention_tc_e4m3(const AttnParams& p, cudaStream_t s) {
  if ((int64_t)p.max_q * p.group <= kFewRows) return launch_attention_e4m3_few(p, s);
  return launch_form<true, true>(p, s);
}

}  // namespace ds
