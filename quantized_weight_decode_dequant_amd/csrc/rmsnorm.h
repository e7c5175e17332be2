// Arguments of the norm kernel (rmsnorm.hip), filled by the C ABI.
#pragma once

#include "qg_internal.h"

namespace qg {

constexpr int64_t RMS_K_MAX = 24576;

struct RmsArgs {
    const void *x, *residual;
    void *residual_out;
    const uint16_t *weight;
    const int8_t *signs;
    uint16_t *y;
    int8_t *Xq;
    float *x_scales;
    double denom;  // 127, times sqrt(32) when rotated
    int64_t M;
    int K;
    float eps;
};

// res: 0 none, 1 bf16, 2 fp32
hipError_t launch_rmsnorm(const RmsArgs &a, bool x_f32, int res, hipStream_t s);

}  // namespace qg
