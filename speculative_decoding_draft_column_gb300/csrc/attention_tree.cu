// The attention kernel's variants for trees of new tokens over a 16-bit cache.

#include <cuda_runtime.h>

#include "attention_launch.cuh"

namespace attn {

spec_status launch_tree(const Args &a, const Pick &p) { return launch<false, true>(a, p); }

}  // namespace attn

namespace host {

cudaError_t take_tree_attention_timeouts(unsigned int *flags) { return take_flag(g_wait_timeouts, flags); }

}  // namespace host
