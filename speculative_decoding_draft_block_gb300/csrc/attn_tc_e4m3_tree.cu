// The attention kernels of attn_tc.cuh for trees over quantised pools.
#include "attn_tc.cuh"

namespace ds {

cudaError_t launch_attention_tc_e4m3_tree(const AttnParams& p, cudaStream_t s) { return launch_form<true, true>(p, s); }

}  // namespace ds
