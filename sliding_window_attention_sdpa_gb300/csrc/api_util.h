// api_util.h -- what the C entry points share (defined in api.cu): the calling
// thread's error message, pointer checks and launch-error conversion.
#pragma once

#include <cstdint>

#include <cuda.h>
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

// TMA descriptor of a 16-bit tensor [n][rows][h][d] (strides in elements: n,
// row, head) in boxes of 64 features x 1 head x box_rows rows with the 128-byte
// swizzle. False if the driver takes no such descriptor.
bool make_rows_map(CUtensorMap* m, const void* base, int dtype, int64_t d, int64_t h, int64_t rows, int64_t n,
                   const int64_t* st, uint32_t box_rows);

}  // namespace api
}  // namespace swa
