// The attention kernels of attn_tc.cuh for trees of drafted tokens over bfloat16 pools.
#include "attn_tc.cuh"

namespace ds {

cudaError_t launch_attention_tc_tree(const AttnParams& p, cudaStream_t s) { return launch_form<true, false>(p, s); }

}  // namespace ds
