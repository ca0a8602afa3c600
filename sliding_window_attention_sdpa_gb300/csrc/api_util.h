// api_util.h -- what the C entry points share (defined in api.cu): the calling
// thread's error message, pointer checks and launch-error conversion.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/sdpa_bwd.h"

namespace swa {
namespace api {

// Records a printf-style message for sdpa_bwd_last_error() and returns `code`.
sdpa_status_t fail(sdpa_status_t code, const char* fmt, ...);
void clear_error();

// `ptr` is device (or managed) memory of device `device`, aligned to `align`
// bytes; NULL is accepted unless `required`.
sdpa_status_t check_device_ptr(const char* name, const void* ptr, bool required, int device, unsigned align = 16);

sdpa_status_t cuda_status(cudaError_t e, const char* what);

}  // namespace api
}  // namespace swa
