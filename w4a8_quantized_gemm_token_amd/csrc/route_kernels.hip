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
//
// A few MB at most are read and written; the time is latency and instructions.  E 384, k 8,
// sigmoid + bias: one token 6.5 us (one launch), 4096 tokens 11 us here and 13 us in the placing;
// 20011 tokens, E 160, softmax in 8 groups: 27 + 21 us.
#include <type_traits>

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

// e^d for d <= 709 (-inf: 0) in fp64: d = n ln 2 + r with |r| <= ln 2 / 2, the Taylor series of e^r to
// r^13 (the rest is below 2^-57 of e^r) and a scaling by 2^n.  About 20 instructions, where the
// library's form with its special cases takes some 40, and a token needs one for each expert.
__device__ __forceinline__ double exp64(double d) {
    d = fmax(d, -1100.0);  // 2^-1587 and below: 0
    const double n = __builtin_rint(d * 1.4426950408889634);
    // Cody and Waite's reduction: ln 2 cut to its first 32 bits, which n times are exact, and the rest
    const double r = fma(n, -0x1.a39ef35793c76p-33, fma(n, -0x1.62e42feep-1, d));
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// 1 / a for 1 <= a < 2^1023: the hardware's approximate reciprocal and two Newton steps
__device__ __forceinline__ double recip64(double a) {
    double y = __builtin_amdgcn_rcp(a);
    y = fma(fma(-a, y, 1.0), y, y);
    return fma(fma(-a, y, 1.0), y, y);
}

// (e^708 is the last whole power that fp64 holds with room to spare: below -708 the score is 0)
__device__ __forceinline__ double sigmoid64(float x) {
    const double s = recip64(1.0 + exp64(fmin(-(double)x, 708.0)));
    return x < -708.0f ? 0.0 : s;
}

__device__ __forceinline__ double readlane64(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)b, l), hi = __builtin_amdgcn_readlane((int)(b >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Sum over the wave, returned to every lane: DPP inside each 16-lane row, then the four rows.
template <int CTRL>
__device__ __forceinline__ double dpp_add64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, false);
    return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_sum64(double v) {
    v = dpp_add64<0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_add64<0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_add64<0x124>(v);  // row_ror:4
    v = dpp_add64<0x128>(v);  // row_ror:8
    return (readlane64(v, 0) + readlane64(v, 16)) + (readlane64(v, 32) + readlane64(v, 48));
}

// Maximum over the wave, returned to every lane.
template <int CTRL>
__device__ __forceinline__ int dpp_max_int(int v) {
    return max(v, __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ int wave_max_int(int v) {
    v = dpp_max_int<0xB1>(v);   // quad_perm [1,0,3,2]
    v = dpp_max_int<0x4E>(v);   // quad_perm [2,3,0,1]
    v = dpp_max_int<0x124>(v);  // row_ror:4
    v = dpp_max_int<0x128>(v);  // row_ror:8
    return max(max(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
               max(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

// Orders a wave's LDS writes before its other lanes' reads (LDS runs a wave's accesses in order;
// this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Routes one token with one wave; lane l holds experts l, l + 64, ... (PER of them).
// The picks go by the keys rounded to fp32, as integers of the same order (the rounding keeps the
// order of the keys): a pick is the wave's maximum, a few DPP steps, and nearly always one expert
// has it.  Where several do, their fp64 keys decide, and then the lower id.
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
    const bool scored = bias || c.n_groups > 1;  // else the logits themselves are the keys
    double top = 0.0, inv = 1.0;
    double key[PER];
    if (softmax) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) m = fmaxf(m, x[i]);
        m = wave_max(m);
        top = m > -INFINITY ? (double)m : 0.0;  // no live logit: every exp is 0, and so is every score
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = exp64((double)x[i] - top);
            sum += key[i];
        }
        sum = wave_sum64(sum);
        inv = sum > 0.0 ? 1.0 / sum : 0.0;
    } else if (scored) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = sigmoid64(x[i]);
    }
    constexpr int kClosed = -0x7FFFFFFF - 1;  // picked, outside E or in a closed group (-inf is above it)
    int ord[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (scored) {
            const double v = x[i] > -INFINITY && b[i] > -INFINITY ? key[i] * inv + (double)b[i] : -INFINITY;
            if (c.n_groups > 1) val[i * kWave + lane] = v;
            key[i] = bias ? v : (double)x[i];
        } else {
            key[i] = (double)x[i];
        }
        const int f = __builtin_bit_cast(int, (float)key[i] + 0.0f);  // (-0 as 0)
        ord[i] = i * kWave + lane < E ? f ^ ((f >> 31) & 0x7FFFFFFF) : kClosed;
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
        // e / gs: (e + 1/2) / gs is 1 / (2 gs) from a whole number at least, far more than fp32 errs
        const float per_gs = 1.0f / (float)gs;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = i * kWave + lane;
            if (e < E && !((mask >> (int)(((float)e + 0.5f) * per_gs)) & 1)) ord[i] = kClosed;
        }
        wave_lds_fence();  // the next token of this wave writes val again
    }
    constexpr int kOrdInf = (int)0xFF800000 ^ 0x7FFFFFFF;  // the order of -inf
    int mine = 0;  // lane j keeps pick j, and its logit (-inf: weight 0)
    float mine_x = -INFINITY;
    for (int j = 0; j < c.topk; ++j) {
        int m = ord[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = max(m, ord[i]);
        m = wave_max_int(m);
        int count = 0, id = 0;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {  // the lowest id with the maximum, and how many have it
            const uint64_t same = __ballot(ord[i] == m);
            count += __popcll(same);
            if (same) id = i * kWave + __builtin_ctzll(same);
        }
        if (count > 1) {
            double best = 0.0;
            bool first = true;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                uint64_t same = __ballot(ord[i] == m);
                if (!same) continue;
                if (first) {
                    best = readlane64(key[i], __builtin_ctzll(same));
                    first = false;
                }
                // the lanes whose key is above the best so far, in turn (equal ones: none)
                for (uint64_t up = __ballot(ord[i] == m && key[i] > best); up;
                     up = __ballot(ord[i] == m && key[i] > best)) {
                    const int l = __builtin_ctzll(up);
                    best = readlane64(key[i], l);
                    id = i * kWave + l;
                }
            }
        }
        const int l = id & (kWave - 1);
        float px = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (id / kWave == i) {
                px = x[i];
                if (lane == l) ord[i] = kClosed;
            }
        px = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, px), l));
        if (lane == j) {
            mine = id;
            mine_x = m == kOrdInf ? -INFINITY : px;  // a key of -inf: no weight
        }
    }
    const bool have = lane < c.topk;
    // a lane without a pick, or with a masked one, has score 0
    double s = softmax ? exp64((double)mine_x - top) * inv : sigmoid64(mine_x);  // -inf: 0
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

// Expert buckets: workgroup e places the pairs of expert e, in increasing pair index, behind the
// pairs of all lower experts.  Each wave owns a contiguous run of pairs and reads it twice (to count,
// then to place), 256 pairs at a time, four neighbours per lane, counting with ballots.  The ids
// come from L2, E times over, and that is the time: 32768 pairs, E 384 12.8 us (71 with a contiguous
// run of pairs per thread).  A count per chunk and a scan over the chunks, which would read them
// twice in all, has not been measured.
// shared_T >= 0: a shared expert with that many slots follows.
typedef int32_t ids4 __attribute__((ext_vector_type(4), aligned(4)));
template <int THREADS>
__global__ __launch_bounds__(THREADS) void place_kernel(const int32_t *__restrict__ ids, int32_t P, int32_t E,
                                                        int32_t k, int32_t shared_T, int32_t *__restrict__ offsets,
                                                        int32_t *__restrict__ perm, int32_t *__restrict__ slot_row,
                                                        int32_t *__restrict__ slot_of_pair) {
    constexpr int kWaves = THREADS / kWave, kChunk = 4 * kWave, kList = 8 * THREADS;
    __shared__ int32_t below_s[kWaves], own_s[kWaves], list[kList];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t e = blockIdx.x;
    const int64_t chunks = ((int64_t)P + kChunk - 1) / kChunk;
    const int64_t p0 = chunks * wave / kWaves * kChunk, p1 = chunks * (wave + 1) / kWaves * kChunk;
    // calls f(c, ids of the pairs c + 4 lane + 0..3) for the wave's chunks from `from` on while more(), with
    // the loads of 8 or 2 of them in flight (their latency is most of the time); past the end the ids
    // are above all
    auto walk = [&](int64_t from, auto more, auto f) {
        const int64_t whole = p1 < P ? p1 : P;
        int64_t c = from;
        auto batch = [&](auto deep) {
            constexpr int D = decltype(deep)::value;
            for (; c + D * kChunk <= whole && more(); c += D * kChunk) {
                ids4 v[D];
#pragma unroll
                for (int d = 0; d < D; ++d) v[d] = *reinterpret_cast<const ids4 *>(ids + c + d * kChunk + 4 * lane);
#pragma unroll
                for (int d = 0; d < D; ++d) f(c + d * kChunk, v[d]);
            }
        };
        batch(std::integral_constant<int, 8>{});
        batch(std::integral_constant<int, 2>{});
        for (; c < p1 && more(); c += kChunk) {
            ids4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t p = c + 4 * lane + j;
                const int32_t id = ids[p < P ? p : P - 1];
                v[j] = p < P ? id : 0x7FFFFFFF;
            }
            f(c, v);
        }
    };
    int32_t below = 0, own = 0;
    walk(p0, [] { return true; }, [&](int64_t, const ids4 &v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            below += __popcll(__ballot(v[j] < e));
            own += __popcll(__ballot(v[j] == e));
        }
    });
    if (lane == 0) {
        below_s[wave] = below;
        own_s[wave] = own;
    }
    __syncthreads();
    int32_t start = 0, before = 0, total = 0;  // before: the expert's pairs in earlier waves' runs
    for (int i = 0; i < kWaves; ++i) {
        start += below_s[i];
        before += i < wave ? own_s[i] : 0;
        total += own_s[i];
    }
    if (tid == 0) {
        offsets[e] = start;
        if (e == E - 1) {
            offsets[E] = start + total;
            if (shared_T >= 0) offsets[E + 1] = start + total + shared_T;
        }
    }
    // The expert's pairs go through a list in LDS, kList of them a round, so that the scattered
    // writes and the division are made by full waves, not by the one lane in 64 that found a pair.
    // A wave starts a round in the chunk where its last one filled the list, so each id is read a
    // bounded number of times whatever the length of the bucket (2^21 tokens of 3 pairs in the same
    // three buckets: 8.0 ms, 156 with every round from the start).  A single round keeps no such
    // place (24 us against 25 for 32768 pairs, E 384).
    const uint64_t lt = (1ull << lane) - 1;
    int64_t at = p0;
    int32_t rank = before;  // number of the expert's pairs before the chunk `at`
    auto round = [&](int32_t base, auto single) {
        constexpr bool kSingle = decltype(single)::value;
        int32_t next = rank - base;  // list place of this wave's next pair
        if (own > 0)
            walk(at, [&] { return kSingle || next < kList; }, [&](int64_t c, const ids4 &v) {
                uint64_t m[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) m[j] = __ballot(v[j] == e);
                if (m[0] | m[1] | m[2] | m[3]) {
                    int32_t to = next;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        to += __popcll(m[j] & lt);
                        next += __popcll(m[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (v[j] == e) {
                            const int32_t p = (int32_t)(c + 4 * lane + j);
                            if (kSingle) list[to & (kList - 1)] = p;  // to < total
                            else if (to >= 0 && to < kList) list[to] = p;
                            ++to;
                        }
                }
                if (!kSingle && next <= kList) {  // else the next round takes this chunk again
                    at = c + kChunk;
                    rank = base + next;
                }
            });
        __syncthreads();
        const int32_t n = total - base < kList ? total - base : kList;
        for (int32_t i = tid; i < n; i += THREADS) {
            const int32_t p = list[i], slot = start + base + i;
            perm[slot] = p;
            slot_of_pair[p] = slot;
            if (slot_row) slot_row[slot] = p / k;
        }
        __syncthreads();
    };
    if (total <= kList) round(0, std::true_type{});
    else
        for (int32_t base = 0; base < total; base += kList) round(base, std::false_type{});
    if (slot_row)
        for (int64_t t = (int64_t)e * THREADS + tid; t < shared_T; t += (int64_t)E * THREADS)
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
    // one launch per kLaunchTokens: its threads, 64 a token, have to stay below 2^32
    constexpr int64_t kLaunchTokens = 1ll << 24;
    const int per = (E + kWave - 1) / kWave;
#define W4A8_RS(PP)                                                                                                  \
    do {                                                                                                             \
        if (one)                                                                                                     \
            hipLaunchKernelGGL((route_scored_one_kernel<PP, L>), dim3(1), dim3(kOneThreads), 0, stream, logits, ldl, \
                               bias, (int32_t)T, E, cfg, (int32_t)shared_T, ids, w, offsets, perm, slot_row,         \
                               slot_of_pair);                                                                        \
        else                                                                                                         \
            for (int64_t t = 0; t < T; t += kLaunchTokens) {                                                         \
                const int64_t n = T - t < kLaunchTokens ? T - t : kLaunchTokens;                                     \
                hipLaunchKernelGGL((route_scored_kernel<PP, L>), dim3((uint32_t)((n + kRouteWaves - 1) / kRouteWaves)), \
                                   dim3(kRouteThreads), 0, stream, logits + t * ldl, ldl, bias, n, E, cfg,           \
                                   ids + t * cfg.topk, w + t * cfg.topk);                                            \
            }                                                                                                        \
    } while (0)
    if (per <= 1) W4A8_RS(1);
    else if (per <= 2) W4A8_RS(2);
    else if (per <= 3) W4A8_RS(3);
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
    if (P <= 2048)
        hipLaunchKernelGGL((place_kernel<256>), dim3((uint32_t)E), dim3(256), 0, stream, ids, (int32_t)P, E, cfg.topk,
                           (int32_t)shared_T, offsets, perm, slot_row, slot_of_pair);
    else
        hipLaunchKernelGGL((place_kernel<1024>), dim3((uint32_t)E), dim3(1024), 0, stream, ids, (int32_t)P, E, cfg.topk,
                           (int32_t)shared_T, offsets, perm, slot_row, slot_of_pair);
    return hipGetLastError();
}

}  // namespace w4a8
