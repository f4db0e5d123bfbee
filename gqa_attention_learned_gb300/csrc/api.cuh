// What the files with entry points share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace sa {

int api_sm_count();                                    // of the current device; 0: no device
int api_status(cudaError_t err, const char *where);    // a sinkattn_status, with its detail kept
int api_failure(const char *what);                     // SINKATTN_CUDA_ERROR with this detail
bool programmatic_for(int launch_flags);               // launch mode of one call

// bf16 tensor viewed as [d2][d1][64] (128-byte rows), box {64, b1, b2}, 128-byte swizzle.
bool api_encode_map(CUtensorMap *map, const void *base, unsigned long long d1, unsigned long long d2,
                    unsigned b1, unsigned b2);

}  // namespace sa
