// The attention kernels of attn_tc.cuh for quantised pools. (Without the masks' code: 2 prompts 577 us,
// 593 with it, 128 requests of 1 to 16 rows over 100 to 500 cached 57.5 and 62.9.)
#include "attn_tc.cuh"

namespace ds {

cudaError_t launch_attention_tc_e4m3(const AttnParams& p, cudaStream_t s) {
  if ((int64_t)p.max_q * p.group <= kFewRows) return launch_attention_e4m3_few(p, s);
  return p.mask != nullptr ? launch_attention_tc_e4m3_tree(p, s) : launch_form<false, true>(p, s);
}

}  // namespace ds
