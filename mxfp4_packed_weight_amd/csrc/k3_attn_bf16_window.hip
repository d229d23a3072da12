// The attention kernels with a window for bf16 queries over a 16-bit cache.
#include "k3_attn_launch.h"

namespace k3 {

hipError_t launch_attn_bf16_window(const AttnArgs &a, hipStream_t s) { return attn_by_dim<true, false, kWindow>(a, s); }

}  // namespace k3
