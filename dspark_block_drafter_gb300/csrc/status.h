// Status reporting shared by the ABI layers: both record the calling thread's message for
// dspark_last_error and return the status.
#pragma once

#include <cuda_runtime.h>

#include <string>

#include "../../include/dspark.h"

namespace dspark {

dspark_status fail(dspark_status s, const std::string& msg);
dspark_status cuda_fail(cudaError_t e, const char* where);

}  // namespace dspark
