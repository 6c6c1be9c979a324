// The attention kernel's variants for 8-bit caches: causal chunks and trees.

#include <cuda_runtime.h>

#include "attention_launch.cuh"

namespace attn {

spec_status launch8(const Args8 &a, const Pick &p, bool tree) { return tree ? launch<true, true>(a, p) : launch<true, false>(a, p); }

}  // namespace attn

namespace host {

cudaError_t take_attention8_timeouts(unsigned int *flags) { return take_flag(g_wait_timeouts, flags); }

}  // namespace host
