/*
 * sdpa_rope.h -- C ABI of what goes into the attention, on GB300 (sm_103a): each
 * head's RMS norm of queries and keys and their position rotation in one pass,
 * and its backward pass (which takes what sdpa_bwd gives as dQ and dK).
 *
 * With x a head's d features of a token, w its tensor's norm weights and R the
 * token's rotation:
 *     y = R (x r (w + weight_offset)),   r = (mean(x^2) + eps)^(-1/2)
 * (without weights y = R x). R turns pair i of the first `rot` features by the
 * angle a = pos * freq[i] and multiplies it by rot_scale:
 *     (y_lo, y_hi) = rot_scale (lo cos a - hi sin a, hi cos a + lo sin a)
 * Pair i is (i, i + rot / 2), or (2 i, 2 i + 1) if `interleaved`; features from rot
 * on are not rotated. (Halves of a rot that is no multiple of 16 take more time: 35,000
 * rows of 54 heads, d = 128, 231 us with rot = 92, 171 with 128; backward 305 and 239.)
 * pos is the token's position on axis[i] (one axis: text; time, height and width: video).
 * Angles are exact products of the int32 position and the fp32 frequency, to 2^-24 of a
 * turn, however far the position, in either direction (|freq| up to 2^50).
 *
 * Backward, with g the gradient of y and u = R^T g:
 *     dx = r (u w' - x r^2 mean(u w' x)),  w' = w + weight_offset
 *     dw = sum over tokens and heads of u x r
 * r is computed again from x; nothing is kept from the forward call.
 * (r^2 stays within fp32 for eps from 2^-128 on; below, for heads whose mean square is, and
 * heads of zeros, whose dx is r u w'.)
 *
 * Conventions as in sdpa_bwd.h: the caller owns every buffer; calls enqueue on
 * `stream` and do not synchronise; arguments are checked on the host first, with a
 * message in sdpa_bwd_last_error(); both calls can be captured into a CUDA graph.
 * Norms, rotations and sums are formed in fp32 and rounded once; dw is summed in a
 * fixed order (bitwise repeatable).
 */
#ifndef SDPA_ROPE_H
#define SDPA_ROPE_H

#include "sdpa_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Strides are in elements: batch (THD: ignored), token, head; the feature stride is
 * 1, every other one a non-negative multiple of 8 elements, tensors of `dtype` are
 * 16-byte aligned, arrays contiguous. An output may be one of its inputs with the
 * same strides (each row is read before it is written).
 */
typedef struct sdpa_rope_params {
    int32_t dtype, layout;            /* SDPA_BF16 | SDPA_F16, SDPA_BSHD | SDPA_THD */
    int32_t interleaved;              /* pairs of neighbours, else of halves */
    int32_t weight_f32;               /* the weights are fp32, else of dtype */
    int64_t b, s, total;              /* BSHD: sequences and rows of each; THD: rows */
    int64_t h_q, h_kv, d;             /* heads (h_kv 0: queries alone), d 64 or 128 */
    int64_t rot, n_axes;              /* rotated features (even, 0 to d), axes of the positions (1 to 8) */
    float eps, weight_offset, rot_scale;
    int32_t reserved0;
    const int32_t *positions;         /* device [n_axes][b * s or total] */
    const int32_t *axis;              /* device [rot / 2], each pair's axis (an entry outside [0, n_axes) is
                                         taken as the nearer end); NULL: axis 0 */
    const float *freq;                /* device [rot / 2], finite: radians per position */
    const int32_t *seq_lens;          /* device [b] or NULL (BSHD): rows at or behind it are padding: not read,
                                         zeros in the outputs, nothing in dw */
    const void *q_weight, *k_weight;  /* device [d]; both (k's with h_kv > 0) or none: no norm */
    const void *q, *k;                /* the forward's inputs (backward without a norm: not read) */
    const void *gq, *gk;              /* backward: gradients of the forward's outputs */
    void *oq, *ok;                    /* forward: outputs; backward: gradients of q and k */
    float *dq_weight, *dk_weight;     /* backward with a norm: device fp32 [d] */
    int64_t q_stride[3], k_stride[3], gq_stride[3], gk_stride[3], oq_stride[3], ok_stride[3];
} sdpa_rope_params;

size_t sdpa_rope_params_bytes(void);

sdpa_status_t sdpa_rope_fwd(const sdpa_rope_params *params, void *stream);

/* Workspace of sdpa_rope_bwd in bytes: 0 on invalid arguments (then
 * sdpa_bwd_last_error() names one) and without a norm (it is empty, and the
 * workspace may be NULL). It needs no initialisation and is 256-byte aligned.
 * Calls that may overlap on the GPU need a workspace each. */
size_t sdpa_rope_bwd_workspace_bytes(const sdpa_rope_params *params);
sdpa_status_t sdpa_rope_bwd(const sdpa_rope_params *params, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SDPA_ROPE_H */
