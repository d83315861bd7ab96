// The attention kernels of attn_tc.cuh for bfloat16 pools.
#include "attn_tc.cuh"

namespace ds {

cudaError_t launch_attention_tc(const AttnParams& p, cudaStream_t s) { return launch_form<false, false>(p, s); }

}  // namespace ds
