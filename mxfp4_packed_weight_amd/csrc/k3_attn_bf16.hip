// The attention kernels for bf16 queries over a 16-bit cache.
#include "k3_attn_launch.h"

namespace k3 {

hipError_t launch_attn_bf16(const AttnArgs &a, hipStream_t s) { return attn_by_dim<true, false>(a, s); }

}  // namespace k3
