// Arguments of the head norm and rotation (qk_rope.hip), filled by the C ABI.
#pragma once

#include "qg_internal.h"

namespace qg {

constexpr int ROPE_D_MAX = 512;

struct QkRopeArgs {
    const void *q, *k;
    const uint16_t *q_weight, *k_weight;  // null: that side is not normed
    const int32_t *positions;             // [axes][M]
    const uint8_t *axis;                  // [half] or null (axis 0)
    const float *inv_freq;                // [half]
    uint16_t *q_out, *k_out;
    int64_t q_stride, k_stride, qo_stride, ko_stride;  // elements between tokens
    int M, Hq, H, D, half, axes;          // H: heads of both sides; half: pairs rotated
    int parts, per_wave;                  // waves a token, heads each takes
    float eps;
};

hipError_t launch_qk_rope(QkRopeArgs a, bool x_f32, bool interleaved, hipStream_t s);

}  // namespace qg
