// The attention kernels with a window for fp16 queries over a 16-bit cache.
#include "k3_attn_launch.h"

namespace k3 {

hipError_t launch_attn_f16_window(const AttnArgs &a, hipStream_t s) { return attn_by_dim<false, false, kWindow>(a, s); }

}  // namespace k3
