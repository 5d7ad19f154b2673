// w8_internal.hpp -- launchers of the 8-bit-weight product and of the scored expert
// routing.  Arguments are already validated; each returns hipSuccess or the launch error.
#pragma once

#include "w4a8_internal.hpp"

namespace w4a8 {

// Dense: out[m][n] = T(a_scale[m] w_scale[n] sum_k qa[m][k] qw[n][k] + bias[n]), T by out_type.
hipError_t launch_gemm_w8a8(const int8_t *qa, const float *a_scale, int64_t M, int64_t K, const int8_t *qw,
                            const float *w_scale, int64_t N, const float *bias, void *out, int32_t out_type,
                            int64_t ldo, hipStream_t stream);

// Expert-grouped: slots expert_offsets[e] .. expert_offsets[e+1] take expert e's weights.
hipError_t launch_grouped_gemm_w8a8(const int8_t *qa, const float *a_scale, int64_t R, const int32_t *row_index,
                                    const int32_t *expert_offsets, int32_t E, int64_t K, const int8_t *qw,
                                    const float *w_scale, int64_t N, int64_t max_slots, float *out,
                                    hipStream_t stream);

struct RouteCfg {
    int32_t topk, score, n_groups, topk_groups, group_lead, renorm;
    float scale;
};
hipError_t launch_moe_route_scored(const void *logits, int32_t logits_type, int64_t ldl, const float *bias, int64_t T,
                                   int32_t E, int32_t with_shared, const RouteCfg &cfg, int32_t *ids, float *w,
                                   int32_t *offsets, int32_t *perm, int32_t *slot_row, int32_t *slot_of_pair,
                                   hipStream_t stream);

// Limits of the scored router (checked by the entry point).
constexpr int32_t kMaxRouteE = 1024, kMaxRouteK = 32, kMaxRouteGroups = 64;

}  // namespace w4a8
