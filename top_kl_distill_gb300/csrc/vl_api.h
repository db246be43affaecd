// Helpers shared by the files that hold C entry points (vloss_api.cu, post_api.cu).
#pragma once

#include "vloss.h"

#include <cuda_runtime.h>

namespace vl {

// Records a printf-style message for vl_last_error_string() and returns s.
vl_status fail(vl_status s, const char* fmt, ...);
vl_status cuda_fail(cudaError_t e, const char* where);

// SMs of the current device (0 when there is none), looked up once per device.
int num_sms();

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace vl
