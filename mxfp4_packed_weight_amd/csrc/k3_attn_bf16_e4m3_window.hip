// The attention kernels with a window for bf16 queries over an e4m3 cache.
#include "k3_attn_launch.h"

namespace k3 {

hipError_t launch_attn_bf16_e4m3_window(const AttnArgs &a, hipStream_t s) { return attn_by_dim<true, true, kWindow>(a, s); }

}  // namespace k3
