// rope_internal.h -- argument block shared by the rotation's host launcher
// (rope_api.cu) and its kernels.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace swa {

// One of the two tensors, queries or keys.
struct RopeTensor {
    const uint16_t *x, *g;     // input, gradient of the output (backward)
    uint16_t* o;
    int64_t x_stride[3], g_stride[3], o_stride[3];
    const void* weight;
    float* dw;
    int32_t heads;
};

struct RopeArgs {
    RopeTensor t[2];
    int64_t rows, s;           // all rows; rows of a sequence (THD: rows)
    int32_t d, rot, n_axes;
    int32_t interleaved, weight_f32;
    float eps, weight_offset, rot_scale;
    const int32_t *positions, *axis, *seq_lens;
    const float* freq;
    int32_t splits[2], per_split;  // a token's queries, its keys are shared between so many warps, so many heads for each
    float* partial;            // backward with a norm: [ctas][2][d]
    int32_t ctas;
};

// CTAs and splits of a call (the backward's workspace holds a partial sum for each CTA).
void rope_plan(RopeArgs& a, bool backward);
cudaError_t launch_rope(const RopeArgs& a, int dtype, bool backward, cudaStream_t s);

}  // namespace swa
