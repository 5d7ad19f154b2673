// route_kernels.hip -- expert routing by scores: softmax or sigmoid of the router's logits, a
// bias per expert that steers the choice but not the weight, experts limited to the best
// groups, and weights renormalised over the picks.
//
// For token t and expert e, with x = the logit (NaN counts as -inf, values above the largest
// fp32 as that):
//     s   = 1 / (1 + exp(-x))   or   exp(x - max) / sum exp(x - max)
//     v   = s + bias[e]  (or s)           -- what groups are compared by
//     key = v            (or x)           -- what experts are compared by; without a bias the
//                                            scores have the logits' order, so x itself is exact
//     group value = the sum of the group's 1 or 2 largest v; the topk_groups largest stay
//     picks = the topk largest keys of those groups, descending, ties to the lower id
//     w   = s[pick] (/ sum of the picks' s) * scale
// An expert whose logit or bias is -inf has v = key = -inf and weight 0.  Scores and keys are
// held in fp64: two experts' keys often differ by less than an fp32 ulp, and the picks
// should be those of the formula.
#include "w8_internal.hpp"

using namespace w4a8dev;
using w4a8::RouteCfg;

namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / kWave;

__device__ __forceinline__ float logit_at(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float logit_at(const _Float16 *p, int64_t i) { return (float)p[i]; }
__device__ __forceinline__ float logit_at(const __bf16 *p, int64_t i) { return (float)p[i]; }

// NaN -> -inf (no comparison with it holds), +inf -> the largest fp32
__device__ __forceinline__ float tame(float x) { return x > -INFINITY ? fminf(x, 3.402823466e38f) : -INFINITY; }

__device__ __forceinline__ double sigmoid64(float x) { return 1.0 / (1.0 + exp(-(double)x)); }

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// Orders a wave's LDS writes before its other lanes' reads (LDS runs a wave's accesses in order;
// this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// One wave per token; lane l holds experts l, l + 64, ... (PER of them).
template <int PER, typename L>
__global__ __launch_bounds__(kRouteThreads) void route_scored_kernel(const L *__restrict__ logits, int64_t ldl,
                                                                     const float *__restrict__ bias, int64_t T,
                                                                     int32_t E, RouteCfg c, int32_t *__restrict__ ids,
                                                                     float *__restrict__ w) {
    __shared__ double val[kRouteWaves][PER * kWave];
    __shared__ double gval[kRouteWaves][w4a8::kMaxRouteGroups];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= T) return;  // whole waves; the LDS rows are each wave's own
    const L *row = logits + t * ldl;
    float x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * kWave + lane;
        x[i] = e < E ? tame(logit_at(row, e)) : -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, x[i]);
    top = wave_max(top);
    double denom = 1.0;
    if (c.score == W4A8_SCORE_SOFTMAX && top > -INFINITY) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) sum += exp((double)x[i] - (double)top);
        denom = wave_sum64(sum);
    }
    auto score = [&](float xv) -> double {
        if (!(xv > -INFINITY)) return 0.0;
        return c.score == W4A8_SCORE_SOFTMAX ? exp((double)xv - (double)top) / denom : sigmoid64(xv);
    };
    double key[PER];
    uint32_t taken = 0;  // bit i: expert i * 64 + lane is picked, outside E or in a closed group
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * kWave + lane;
        if (e >= E) taken |= 1u << i;
        double v = -INFINITY;
        const float b = bias && e < E ? tame(bias[e]) : 0.0f;
        if (x[i] > -INFINITY && b > -INFINITY && (bias || c.n_groups > 1)) v = score(x[i]) + (double)b;
        if (c.n_groups > 1) val[wave][i * kWave + lane] = v;
        key[i] = bias ? v : (double)x[i];
    }
    if (c.n_groups > 1) {
        // 64 / n_groups lanes (a power of two) walk each group, their best two are merged
        wave_lds_fence();
        const int gs = E / c.n_groups;
        int seg = 1;
        while (2 * seg * c.n_groups <= kWave) seg *= 2;
        const int g = lane / seg;
        double a = -INFINITY, b = -INFINITY;
        if (g < c.n_groups)
            for (int j = lane % seg; j < gs; j += seg) {
                const double v = val[wave][g * gs + j];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
        for (int off = 1; off < seg; off *= 2) {
            const double oa = __shfl_xor(a, off, kWave), ob = __shfl_xor(b, off, kWave);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        if (g < c.n_groups && lane % seg == 0) gval[wave][g] = c.group_lead == 2 ? a + b : a;
        wave_lds_fence();
        bool open = false;
        if (lane < c.n_groups) {
            const double mine = gval[wave][lane];
            int before = 0;
            for (int o = 0; o < c.n_groups; ++o) {
                const double ov = gval[wave][o];
                before += (ov > mine || (ov == mine && o < lane)) ? 1 : 0;
            }
            open = before < c.topk_groups;
        }
        const uint64_t mask = __ballot(open);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * kWave + lane;
            if (e < E && !((mask >> (e / gs)) & 1)) taken |= 1u << i;
        }
    }
    int mine = 0;          // lane j keeps pick j
    bool shut = false;     // its key is -inf
    for (int j = 0; j < c.topk; ++j) {
        double bv = -INFINITY;
        int bi = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * kWave + lane;
            const bool take = !((taken >> i) & 1u) && (key[i] > bv || (key[i] == bv && e < bi));
            bv = take ? key[i] : bv;
            bi = take ? e : bi;
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const double ov = __shfl_xor(bv, off, kWave);
            const int oi = __shfl_xor(bi, off, kWave);
            const bool take = ov > bv || (ov == bv && oi < bi);
            bv = take ? ov : bv;
            bi = take ? oi : bi;
        }
        if ((bi & (kWave - 1)) == lane) taken |= 1u << ((bi / kWave) & 31);
        if (lane == j) {
            mine = bi;
            shut = !(bv > -INFINITY);
        }
    }
    const bool have = lane < c.topk;
    double s = have && !shut ? score(tame(logit_at(row, mine))) : 0.0;
    if (c.renorm) {
        const double sum = wave_sum64(s);
        s = sum > 0.0 ? s / sum : 0.0;
    }
    if (have) {
        ids[t * c.topk + lane] = mine;
        w[t * c.topk + lane] = (float)(s * (double)c.scale);
    }
}

// Expert buckets: workgroup e counts the pairs of lower experts (its offset) and places its own
// in increasing pair index.  Thread i owns the contiguous pairs [i C, (i + 1) C).
// shared_T >= 0: a shared expert with that many slots follows.
constexpr int kPlaceThreads = 256;
__global__ __launch_bounds__(kPlaceThreads) void place_kernel(const int32_t *__restrict__ ids, int64_t P, int32_t E,
                                                              int32_t k, int64_t shared_T,
                                                              int32_t *__restrict__ offsets,
                                                              int32_t *__restrict__ perm,
                                                              int32_t *__restrict__ slot_row,
                                                              int32_t *__restrict__ slot_of_pair) {
    __shared__ int32_t sums[2][kPlaceThreads / kWave];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t e = blockIdx.x;
    const int64_t C = (P + kPlaceThreads - 1) / kPlaceThreads;
    const int64_t p0 = tid * C < P ? tid * C : P, p1 = p0 + C < P ? p0 + C : P;
    int32_t below = 0, own = 0;
    for (int64_t p = p0; p < p1; ++p) {
        const int32_t v = ids[p];
        below += v < e ? 1 : 0;
        own += v == e ? 1 : 0;
    }
    int32_t incl = own;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int32_t o = __shfl_up(incl, off, kWave);
        if (lane >= off) incl += o;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) below += __shfl_xor(below, off, kWave);
    if (lane == kWave - 1) sums[0][wave] = incl;
    if (lane == 0) sums[1][wave] = below;
    __syncthreads();
    int32_t start = 0, before = 0, total = 0;
    for (int i = 0; i < kPlaceThreads / kWave; ++i) {
        start += sums[1][i];
        total += sums[0][i];
        if (i < wave) before += sums[0][i];
    }
    if (tid == 0) {
        offsets[e] = start;
        if (e == E - 1) {
            offsets[E] = start + total;
            if (shared_T >= 0) offsets[E + 1] = start + total + (int32_t)shared_T;
        }
    }
    int32_t slot = start + before + incl - own;
    for (int64_t p = p0; p < p1; ++p)
        if (ids[p] == e) {
            perm[slot] = (int32_t)p;
            slot_of_pair[p] = slot;
            if (slot_row) slot_row[slot] = (int32_t)(p / k);
            ++slot;
        }
    if (slot_row)
        for (int64_t t = (int64_t)e * kPlaceThreads + tid; t < shared_T; t += (int64_t)E * kPlaceThreads)
            slot_row[P + t] = (int32_t)t;
}

}  // namespace

namespace w4a8 {

template <typename L>
static void route_typed(const L *logits, int64_t ldl, const float *bias, int64_t T, int32_t E, const RouteCfg &cfg,
                        int32_t *ids, float *w, hipStream_t stream) {
    const dim3 grid((uint32_t)((T + kRouteWaves - 1) / kRouteWaves)), block(kRouteThreads);
    const int per = (E + kWave - 1) / kWave;
#define W4A8_RS(PP)                                                                                                  \
    hipLaunchKernelGGL((route_scored_kernel<PP, L>), grid, block, 0, stream, logits, ldl, bias, T, E, cfg, ids, w)
    if (per <= 1) W4A8_RS(1);
    else if (per <= 2) W4A8_RS(2);
    else if (per <= 4) W4A8_RS(4);
    else if (per <= 8) W4A8_RS(8);
    else W4A8_RS(16);
#undef W4A8_RS
}

hipError_t launch_moe_route_scored(const void *logits, int32_t logits_type, int64_t ldl, const float *bias, int64_t T,
                                   int32_t E, int32_t with_shared, const RouteCfg &cfg, int32_t *ids, float *w,
                                   int32_t *offsets, int32_t *perm, int32_t *slot_row, int32_t *slot_of_pair,
                                   hipStream_t stream) {
    if (T > 0) {
        if (logits_type == W4A8_F16)
            route_typed((const _Float16 *)logits, ldl, bias, T, E, cfg, ids, w, stream);
        else if (logits_type == W4A8_BF16)
            route_typed((const __bf16 *)logits, ldl, bias, T, E, cfg, ids, w, stream);
        else
            route_typed((const float *)logits, ldl, bias, T, E, cfg, ids, w, stream);
        if (hipError_t err = hipGetLastError()) return err;
    }
    hipLaunchKernelGGL(place_kernel, dim3((uint32_t)E), dim3(kPlaceThreads), 0, stream, ids, T * cfg.topk, E, cfg.topk,
                       with_shared ? T : (int64_t)-1, offsets, perm, slot_row, slot_of_pair);
    return hipGetLastError();
}

}  // namespace w4a8
