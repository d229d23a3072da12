// The attention kernels for fp16 queries over an e4m3 cache with exponents.
#include "k3_attn_launch.h"

namespace k3 {

hipError_t launch_attn_f16_blocks(const AttnArgs &a, hipStream_t s) { return attn_by_dim<false, true, kBlocks>(a, s); }

}  // namespace k3
