// What the files of the C ABI share (ra_api.cu, kv4_api.cu): the record of the streams
// that an object's kernels were queued on.
#pragma once

#include <cuda_runtime.h>

#include <vector>

#include "ra.h"

namespace ra {

// One event per stream the kernels of an object (a plan, a cache handle) were queued on,
// recorded after the latest of them: destroying the object queues the frees of its device
// memory behind exactly this work.  A slot whose event has completed is reused for a new
// stream.
struct StreamMark {
  cudaStream_t stream;
  cudaEvent_t done;
};

// Record, on `st`, that the object's device memory is in use by the work queued there so far.
ra_status mark_use(std::vector<StreamMark>* marks, cudaStream_t st);

}  // namespace ra
