// The attention kernels for fp16 queries over a 16-bit cache.
#include "k3_attn_launch.h"

namespace k3 {

hipError_t launch_attn_f16(const AttnArgs &a, hipStream_t s) { return attn_by_dim<false, false>(a, s); }

}  // namespace k3
