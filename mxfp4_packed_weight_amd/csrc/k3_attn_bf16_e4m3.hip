// The attention kernels for bf16 queries over an e4m3 cache.
#include "k3_attn_launch.h"

namespace k3 {

hipError_t launch_attn_bf16_e4m3(const AttnArgs &a, hipStream_t s) { return attn_by_dim<true, true, kAllPlaces>(a, s); }

}  // namespace k3
