// What the files with entry points share.
#pragma once

#include <cuda_runtime.h>

namespace sa {

int api_sm_count();                                    // of the current device; 0: no device
int api_status(cudaError_t err, const char *where);    // a sinkattn_status, with its detail kept
int api_failure(const char *what);                     // SINKATTN_CUDA_ERROR with this detail
bool programmatic_for(int launch_flags);               // launch mode of one call

}  // namespace sa
