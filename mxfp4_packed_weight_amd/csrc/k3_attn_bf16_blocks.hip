// The attention kernels for bf16 queries over an e4m3 cache with exponents.
#include "k3_attn_launch.h"

namespace k3 {

hipError_t launch_attn_bf16_blocks(const AttnArgs &a, hipStream_t s) { return attn_by_dim<true, true, kBlocks>(a, s); }

}  // namespace k3
