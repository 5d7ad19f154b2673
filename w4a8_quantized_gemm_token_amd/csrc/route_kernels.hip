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

// Minimum over the wave, returned to every lane (DPP inside each 16-lane row, then the four rows).
template <int CTRL>
__device__ __forceinline__ int dpp_min(int v) {
    return min(v, __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ int wave_min_int(int v) {
    v = dpp_min<0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_min<0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_min<0x124>(v);  // row_ror:4
    v = dpp_min<0x128>(v);  // row_ror:8
    return min(min(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
               min(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}
__device__ __forceinline__ double readlane64(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)b, l), hi = __builtin_amdgcn_readlane((int)(b >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Orders a wave's LDS writes before its other lanes' reads (LDS runs a wave's accesses in order;
// this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Routes one token with one wave; lane l holds experts l, l + 64, ... (PER of them).
// A pick is the wave's largest key: each lane keeps its own best open key in fp64 and that rounded
// to fp32; the rounding keeps the order, so the fp32 maximum (a few DPP steps) names the winner
// unless several lanes share it, and only those are then compared in fp64, and by id.
// val, gval: the wave's own LDS, used when there are groups.
template <int PER, typename L>
__device__ __forceinline__ void route_scored_token(const L *__restrict__ row, const float *__restrict__ bias, int32_t E,
                                                   const RouteCfg &c, double *val, double *gval,
                                                   int32_t *__restrict__ ids, float *__restrict__ w) {
    const int lane = threadIdx.x & 63;
    float x[PER], b[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * kWave + lane;
        x[i] = e < E ? tame(logit_at(row, e)) : -INFINITY;
        b[i] = bias && e < E ? tame(bias[e]) : 0.0f;
    }
    const bool softmax = c.score == W4A8_SCORE_SOFTMAX;
    double top = 0.0, denom = 1.0;
    if (softmax) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) m = fmaxf(m, x[i]);
        m = wave_max(m);
        if (m > -INFINITY) {
            top = (double)m;
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += exp((double)x[i] - top);
            denom = wave_sum64(sum);
        }
    }
    auto score = [&](float xv) -> double {
        if (!(xv > -INFINITY)) return 0.0;
        return softmax ? exp((double)xv - top) / denom : sigmoid64(xv);
    };
    const bool scored = bias || c.n_groups > 1;  // else the logits themselves are the keys
    double key[PER];
    uint32_t taken = 0;  // bit i: expert i * 64 + lane is picked, outside E or in a closed group
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * kWave + lane;
        if (e >= E) taken |= 1u << i;
        double v = -INFINITY;
        if (scored && x[i] > -INFINITY && b[i] > -INFINITY) v = score(x[i]) + (double)b[i];
        if (c.n_groups > 1) val[i * kWave + lane] = v;
        key[i] = bias ? v : (double)x[i];
    }
    if (c.n_groups > 1) {
        // 64 / n_groups lanes (a power of two) walk each group; their best two are merged
        wave_lds_fence();
        const int gs = E / c.n_groups;
        int seg = 1;
        while (2 * seg * c.n_groups <= kWave) seg *= 2;
        const int g = lane / seg;
        double v1 = -INFINITY, v2 = -INFINITY;
        if (g < c.n_groups)
            for (int j = lane % seg; j < gs; j += seg) {
                const double v = val[g * gs + j];
                v2 = fmax(v2, fmin(v1, v));
                v1 = fmax(v1, v);
            }
        for (int off = 1; off < seg; off *= 2) {
            const double o1 = __shfl_xor(v1, off, kWave), o2 = __shfl_xor(v2, off, kWave);
            v2 = fmax(fmin(v1, o1), fmax(v2, o2));
            v1 = fmax(v1, o1);
        }
        if (g < c.n_groups && lane % seg == 0) gval[g] = c.group_lead == 2 ? v1 + v2 : v1;
        wave_lds_fence();
        bool open = false;
        if (lane < c.n_groups) {
            const double mine = gval[lane];
            int before = 0;
            for (int o = 0; o < c.n_groups; ++o) {
                const double ov = gval[o];
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
        wave_lds_fence();  // the next token of this wave writes val again
    }
    // this lane's best open key, of equal ones the first; i = PER: none is open
    double bv;
    float bf;
    int bi;
    auto own_best = [&]() {
        bv = -INFINITY;
        bi = PER;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool take = !((taken >> i) & 1u) & ((bi == PER) | (key[i] > bv));
            bv = take ? key[i] : bv;
            bi = take ? i : bi;
        }
        bf = (float)bv;
    };
    own_best();
    int mine = 0;       // lane j keeps pick j
    bool shut = false;  // its key is -inf
    for (int j = 0; j < c.topk; ++j) {
        const float m = wave_max(bf);
        uint64_t same = __ballot(bi < PER && bf == m);
        int l = __builtin_ctzll(same), id;
        if ((same & (same - 1)) == 0) {
            id = __builtin_amdgcn_readlane(bi, l) * kWave + l;
        } else {
            const double k0 = readlane64(bv, l);
            const bool in = (same >> lane) & 1;
            if (__ballot(in && bv != k0)) {  // the largest of the keys that round alike
                double best = k0;
                for (uint64_t r = same & (same - 1); r; r &= r - 1) best = fmax(best, readlane64(bv, __builtin_ctzll(r)));
                same = __ballot(in && bv == best);
            }
            id = wave_min_int((same >> lane) & 1 ? bi * kWave + lane : 0x7FFFFFFF);
            l = id & (kWave - 1);
        }
        const bool none = !(readlane64(bv, l) > -INFINITY);
        if (lane == j) {
            mine = id;
            shut = none;
        }
        if (lane == l) taken |= 1u << bi;
        own_best();
    }
    const bool have = lane < c.topk;
    double s = have && !shut ? score(tame(logit_at(row, mine))) : 0.0;
    if (c.renorm) {
        const double sum = wave_sum64(s);
        s = sum > 0.0 ? s / sum : 0.0;
    }
    if (have) {
        ids[lane] = mine;
        w[lane] = (float)(s * (double)c.scale);
    }
}

template <int PER, typename L>
__global__ __launch_bounds__(kRouteThreads) void route_scored_kernel(const L *__restrict__ logits, int64_t ldl,
                                                                     const float *__restrict__ bias, int64_t T,
                                                                     int32_t E, RouteCfg c, int32_t *__restrict__ ids,
                                                                     float *__restrict__ w) {
    __shared__ double val[kRouteWaves][PER * kWave];
    __shared__ double gval[kRouteWaves][w4a8::kMaxRouteGroups];
    const int wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= T) return;  // whole waves; the LDS rows are each wave's own
    route_scored_token<PER>(logits + t * ldl, bias, E, c, val[wave], gval[wave], ids + t * c.topk, w + t * c.topk);
}

// Expert buckets: a workgroup places the pairs of kPlaceE experts, in increasing pair index, behind
// the pairs of all lower experts.  Wave w owns a contiguous run of pairs and reads it twice (once to
// count, once to place), 64 pairs at a time: the ids come from L2, E / kPlaceE times over, which
// for some 10^5 pairs costs less than a scan over chunks with its extra launches.
// shared_T >= 0: a shared expert with that many slots follows.
constexpr int kPlaceE = 4;
template <int THREADS>
__global__ __launch_bounds__(THREADS) void place_kernel(const int32_t *__restrict__ ids, int64_t P, int32_t E,
                                                        int32_t k, int64_t shared_T, int32_t *__restrict__ offsets,
                                                        int32_t *__restrict__ perm, int32_t *__restrict__ slot_row,
                                                        int32_t *__restrict__ slot_of_pair) {
    constexpr int kWaves = THREADS / kWave, kDeep = 8;  // kDeep loads of 64 ids in flight
    __shared__ int32_t below_s[kWaves], own_s[kPlaceE][kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t e0 = blockIdx.x * kPlaceE;
    const int64_t C = (P + kWaves * kWave - 1) / (kWaves * kWave) * kWave;  // whole chunks of 64 per wave
    const int64_t p0 = wave * C, p1 = p0 + C < P ? p0 + C : P;
    int32_t below = 0, own[kPlaceE] = {};
    for (int64_t c = p0; c < p1; c += kDeep * kWave) {
        int32_t v[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int64_t p = c + j * kWave + lane;
            v[j] = p < p1 ? ids[p] : 0x7FFFFFFF;
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            below += v[j] < e0 ? 1 : 0;
#pragma unroll
            for (int i = 0; i < kPlaceE; ++i) own[i] += v[j] == e0 + i ? 1 : 0;
        }
    }
    auto wave_sum = [](int32_t v) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
        return v;
    };
    below = wave_sum(below);
#pragma unroll
    for (int i = 0; i < kPlaceE; ++i) own[i] = wave_sum(own[i]);
    if (lane == 0) {
        below_s[wave] = below;
#pragma unroll
        for (int i = 0; i < kPlaceE; ++i) own_s[i][wave] = own[i];
    }
    __syncthreads();
    int32_t start = 0, slot[kPlaceE];  // slot: of this wave's next pair of each expert
    for (int i = 0; i < kWaves; ++i) start += below_s[i];
#pragma unroll
    for (int i = 0; i < kPlaceE; ++i) {
        if (e0 + i < E && tid == i) offsets[e0 + i] = start;
        slot[i] = start;
        for (int j = 0; j < kWaves; ++j) {
            slot[i] += j < wave ? own_s[i][j] : 0;
            start += own_s[i][j];
        }
    }
    if (e0 + kPlaceE >= E && tid == 0) {
        offsets[E] = start;
        if (shared_T >= 0) offsets[E + 1] = start + (int32_t)shared_T;
    }
    const uint64_t lt = (1ull << lane) - 1;
    for (int64_t c = p0; c < p1; c += kDeep * kWave) {
        int32_t v[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int64_t p = c + j * kWave + lane;
            v[j] = p < p1 ? ids[p] : 0x7FFFFFFF;
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
            const int64_t p = c + j * kWave + lane;
            if (!__ballot(v[j] >= e0 && v[j] < e0 + kPlaceE)) continue;
#pragma unroll
            for (int i = 0; i < kPlaceE; ++i) {
                const uint64_t m = __ballot(v[j] == e0 + i);
                if (v[j] == e0 + i) {
                    const int32_t to = slot[i] + __popcll(m & lt);
                    perm[to] = (int32_t)p;
                    slot_of_pair[p] = to;
                    if (slot_row) slot_row[to] = (int32_t)(p / k);
                }
                slot[i] += __popcll(m);
            }
        }
    }
    if (slot_row)
        for (int64_t t = (int64_t)blockIdx.x * THREADS + tid; t < shared_T; t += (int64_t)gridDim.x * THREADS)
            slot_row[P + t] = (int32_t)t;
}

// Few tokens in one launch: one workgroup, a wave per token, then the buckets from the ids in LDS.
// With so few pairs a slot is counted outright: pair p of expert e takes the number of pairs of
// lower experts plus the number of earlier pairs of e.
constexpr int kOneTokens = 16, kOneThreads = 64 * kOneTokens, kOnePairs = kOneTokens * w4a8::kMaxRouteK;
template <int PER, typename L>
__global__ __launch_bounds__(kOneThreads) void route_scored_one_kernel(
    const L *__restrict__ logits, int64_t ldl, const float *__restrict__ bias, int32_t T, int32_t E, RouteCfg c,
    int32_t shared_T, int32_t *__restrict__ ids, float *__restrict__ w, int32_t *__restrict__ offsets,
    int32_t *__restrict__ perm, int32_t *__restrict__ slot_row, int32_t *__restrict__ slot_of_pair) {
    __shared__ double val[kOneTokens][PER * kWave];
    __shared__ double gval[kOneTokens][w4a8::kMaxRouteGroups];
    __shared__ __attribute__((aligned(16))) int32_t all[kOnePairs];
    __shared__ float all_w[kOnePairs];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int P = T * c.topk;
    for (int p = tid; p < (P + 3) / 4 * 4; p += kOneThreads) all[p] = 0x7FFFFFFF;  // whole reads of 4 below
    __syncthreads();
    if (wave < T)
        route_scored_token<PER>(logits + wave * ldl, bias, E, c, val[wave], gval[wave], all + wave * c.topk,
                                all_w + wave * c.topk);
    __syncthreads();
    // waves from the front take experts, from the back pairs
    for (int e = tid; e <= E; e += kOneThreads) {
        int32_t below = 0;
        for (int q = 0; q < P; q += 4) {
            const int4 v = *reinterpret_cast<const int4 *>(all + q);
            below += (v.x < e ? 1 : 0) + (v.y < e ? 1 : 0) + (v.z < e ? 1 : 0) + (v.w < e ? 1 : 0);
        }
        offsets[e] = below;
        if (e == E && shared_T >= 0) offsets[E + 1] = below + shared_T;
    }
    for (int p = kOneThreads - 1 - tid; p < P; p += kOneThreads) {
        const int32_t e = all[p];
        int32_t slot = 0;
        for (int q = 0; q < P; q += 4) {
            const int4 v = *reinterpret_cast<const int4 *>(all + q);
            auto before = [&](int32_t o, int i) { return (o < e || (o == e && i < p)) ? 1 : 0; };
            slot += before(v.x, q) + before(v.y, q + 1) + before(v.z, q + 2) + before(v.w, q + 3);
        }
        ids[p] = e;
        w[p] = all_w[p];
        perm[slot] = p;
        slot_of_pair[p] = slot;
        if (slot_row) slot_row[slot] = p / c.topk;
    }
    if (slot_row && tid < shared_T) slot_row[P + tid] = tid;
}

}  // namespace

namespace w4a8 {

template <typename L>
static void route_typed(const L *logits, int64_t ldl, const float *bias, int64_t T, int32_t E, int64_t shared_T,
                        const RouteCfg &cfg, int32_t *ids, float *w, int32_t *offsets, int32_t *perm,
                        int32_t *slot_row, int32_t *slot_of_pair, bool one, hipStream_t stream) {
    const dim3 grid((uint32_t)((T + kRouteWaves - 1) / kRouteWaves)), block(kRouteThreads);
    const int per = (E + kWave - 1) / kWave;
#define W4A8_RS(PP)                                                                                                  \
    do {                                                                                                             \
        if (one)                                                                                                     \
            hipLaunchKernelGGL((route_scored_one_kernel<PP, L>), dim3(1), dim3(kOneThreads), 0, stream, logits, ldl, \
                               bias, (int32_t)T, E, cfg, (int32_t)shared_T, ids, w, offsets, perm, slot_row,         \
                               slot_of_pair);                                                                        \
        else                                                                                                         \
            hipLaunchKernelGGL((route_scored_kernel<PP, L>), grid, block, 0, stream, logits, ldl, bias, T, E, cfg,   \
                               ids, w);                                                                              \
    } while (0)
    if (per <= 1) W4A8_RS(1);
    else if (per <= 2) W4A8_RS(2);
    else if (per <= 4) W4A8_RS(4);
    else if (per <= 6) W4A8_RS(6);
    else if (per <= 8) W4A8_RS(8);
    else W4A8_RS(16);
#undef W4A8_RS
}

hipError_t launch_moe_route_scored(const void *logits, int32_t logits_type, int64_t ldl, const float *bias, int64_t T,
                                   int32_t E, int32_t with_shared, const RouteCfg &cfg, int32_t *ids, float *w,
                                   int32_t *offsets, int32_t *perm, int32_t *slot_row, int32_t *slot_of_pair,
                                   hipStream_t stream) {
    const int64_t shared_T = with_shared ? T : (int64_t)-1, P = T * cfg.topk;
    const bool one = T > 0 && T <= kOneTokens;
    if (T > 0) {
#define W4A8_RT(L) \
    route_typed((const L *)logits, ldl, bias, T, E, shared_T, cfg, ids, w, offsets, perm, slot_row, slot_of_pair, one, stream)
        if (logits_type == W4A8_F16) W4A8_RT(_Float16);
        else if (logits_type == W4A8_BF16) W4A8_RT(__bf16);
        else W4A8_RT(float);
#undef W4A8_RT
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess || one) return err;
    }
    const dim3 grid((uint32_t)((E + kPlaceE - 1) / kPlaceE));
    if (P <= 2048)
        hipLaunchKernelGGL(place_kernel<256>, grid, dim3(256), 0, stream, ids, P, E, cfg.topk, shared_T, offsets, perm,
                           slot_row, slot_of_pair);
    else
        hipLaunchKernelGGL(place_kernel<1024>, grid, dim3(1024), 0, stream, ids, P, E, cfg.topk, shared_T, offsets,
                           perm, slot_row, slot_of_pair);
    return hipGetLastError();
}

}  // namespace w4a8
