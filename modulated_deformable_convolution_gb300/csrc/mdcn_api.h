// What the files of the C ABI share: error reporting and the device check.
#pragma once

#include <cuda_runtime.h>

#include "mdcn.h"

namespace mdcn {

// Keeps e for mdcn_last_cuda_error and returns MDCN_ERR_CUDA.
mdcn_status api_cuda_fail(cudaError_t e);
// MDCN_OK on a compute capability 10.3 device (current); *sms = its SM count.
mdcn_status api_check_device(int* sms);

}  // namespace mdcn
