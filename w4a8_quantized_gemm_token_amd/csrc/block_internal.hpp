// block_internal.hpp -- launchers of the low-rank adapters and of what stands between two
// blocks.  Arguments are already validated; each returns hipSuccess or the launch error.
#pragma once

#include "w4a8_internal.hpp"

namespace w4a8 {

// Limits of w4a8_lora_add and w4a8_residual_norm_quantize (checked by the entry points).
constexpr int64_t kLoraMaxK = 1ll << 20, kLoraMaxN = 1ll << 23, kLoraMaxLd = 1ll << 24, kNormMaxH = 32768;
constexpr int32_t kLoraMaxL = 65536, kLoraMaxR = 256;

struct LoraArgs {
    const void *x;
    const int32_t *row_adapter;
    const void *A, *B;
    const int32_t *ranks;
    const float *scale;
    const void *base;
    void *out, *ws;
    int64_t M, K, N, ldx, ldb, ldo;
    int32_t L, R, x_type, ab_type, out_type;
};
int64_t lora_ws_bytes(int64_t M, int64_t K, int32_t L, int32_t R);
hipError_t launch_lora_add(const LoraArgs &a, hipStream_t stream);

struct NormArgs {
    const void *res, *y, *gate;
    void *res_out, *z;
    const float *post_w, *post_b, *pre_w, *pre_b;
    int8_t *qa;
    float *a_scale;
    int64_t M, H, ldr, ldy, ldg, ldro, ldz;
    double res_scale, y_scale, eps;
    int32_t res_type, y_type, gate_type, z_type, post, pre;
};
hipError_t launch_residual_norm_quantize(const NormArgs &a, hipStream_t stream);

}  // namespace w4a8
