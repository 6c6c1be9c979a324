// Host state that the library's translation units share: the calling thread's
// stream and error text, and the process-wide launch count (specsel.cu holds
// them).
#pragma once

#include <cuda_runtime.h>

#include "specsel.h"

namespace host {

cudaStream_t stream();
void clear_error();
spec_status fail(spec_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
spec_status cuda_fail(cudaError_t e, const char *what);
void count_launch();

// The wait flag of paged.cu's kernels (read and cleared), for spec_device_status.
cudaError_t take_paged_timeouts(unsigned int *flags);

}  // namespace host
