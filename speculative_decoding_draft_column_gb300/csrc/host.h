// Host state that the library's translation units share: the calling thread's
// stream and error text, and the process-wide launch count (specsel.cu holds
// them).
#pragma once

#include <cuda_runtime.h>

#include <mutex>

#include "specsel.h"

namespace host {

cudaStream_t stream();
void clear_error();
spec_status fail(spec_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
spec_status cuda_fail(cudaError_t e, const char *what);
void count_launch();

// The wait flag of a translation unit's kernels, a device variable of its own, read
// into *flags and cleared.
template <typename F>
cudaError_t take_flag(const F &flag, unsigned int *flags)
{
    cudaError_t e = cudaMemcpyFromSymbol(flags, flag, sizeof *flags);
    if (e != cudaSuccess || *flags == 0) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(flag, &zero, sizeof zero);
}

// Those of the units, for spec_device_status.
cudaError_t take_paged_timeouts(unsigned int *flags);
cudaError_t take_tree_attention_timeouts(unsigned int *flags);
cudaError_t take_attention8_timeouts(unsigned int *flags);

// The current device's scratch for a call on the calling thread's stream: a ticket a lane, zero between calls,
// and `entries` words of lists.  False where there is none to be had (it would have to grow inside
// a stream capture, or memory is out).  It stays as long as `hold` is locked, so the call is launched before that
// is let go of: spec_release, on another thread, waits for the lock and then for what was launched.
bool lane_scratch(int64_t lanes, int64_t entries, unsigned int **tickets, unsigned long long **lists,
                  std::unique_lock<std::mutex> *hold);

}  // namespace host
