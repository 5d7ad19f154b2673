// norm_kernels.hip -- between two blocks of a model: the post-norm of a block's output, its gate
// and the residual join, the next block's norm, and the INT8 codes that its products read.
//
// One workgroup per row, the row in registers: y and the stream are read once, everything is
// written once.  The arithmetic up to z is fp64 (see the entry point).  A row passes up to five
// reductions (mean and mean square of each norm, the maximum); each is four DPP steps inside 16
// lanes, four scalar reads, one LDS exchange and one barrier.
//
// HBM bounds it where there are many rows: 4096 rows of 7168 (fp32 in, bf16 stream, codes) 54 us, 4.9 TB/s, and 20011 rows
// with a post-norm, a gate, z and codes 316 us, 5.0 TB/s, the rate of a large copy.  4096 rows of 8192 with an fp32
// stream and a gate per row take 111 us, 5.4 TB/s.  A few rows wait for one row's chain: one token 5.0 us, 64 rows of
// 8192 6.0 us, 77 rows of 5003 with two layer norms (five reductions) 8.5 us.  The chain is the reductions, and besides
// the norms' vectors and the gate, each loaded where it is used, behind the reduction before it and once a chunk,
// and the stream's store, which the second norm's sums wait for as compiled (they wait for all loads that may be under way
// there, and stores count with loads).  One row of 16384 takes 7.5 us, of 28672 (four chunks a thread) 11.7 us.  Tried and slower: workgroups that walk
// rows with the next row's loads ahead, and four rows a workgroup.
#include "block_internal.hpp"

#include <algorithm>

using namespace w4a8;
using namespace w4a8dev;

namespace {

constexpr int kMaxThreads = 1024;

// ------------------------------------------------------------------ elements
// A thread owns C chunks of 8 elements in a row, chunk c from element (c T + t) 8; n is the number of the row's
// elements from there on, and chunks with none are skipped.  Chunks that lie whole in the row are read and written 16
// bytes at a time at any alignment of the rows (the type's own).  TAIL: the row's last chunk does not, and goes element
// by element, with 0 past the row's end (read as the row's last 8 elements and moved down in registers it took longer:
// 77 rows of 5003 with a gate per row 9.3 us against 8.4).
// Loads keep the bits of the type, and what uses them converts: beside the load a conversion would wait for it before
// the next load is under way (4096 rows of 7168 82 us against 62).
template <typename T>
using Eight = T __attribute__((ext_vector_type(8)));

template <bool TAIL, typename T>
__device__ __forceinline__ Eight<T> load8(const T *p, int n) {
    typedef T t8 __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    if (!TAIL || n >= 8) return *reinterpret_cast<const t8 *>(p);
    Eight<T> x = {};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) x[e] = p[e];
    return x;
}
template <bool TAIL, typename T>
__device__ __forceinline__ Eight<float> floats_at(const void *p, int64_t at, int n) {
    const Eight<T> x = load8<TAIL>((const T *)p + at, n);
    Eight<float> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
    return v;
}
template <bool TAIL>
__device__ __forceinline__ Eight<float> floats_at(const void *p, int64_t at, int type, int n) {
    if (type == W4A8_F32) return floats_at<TAIL, float>(p, at, n);
    if (type == W4A8_F16) return floats_at<TAIL, _Float16>(p, at, n);
    return floats_at<TAIL, __bf16>(p, at, n);
}

template <bool TAIL, typename T>
__device__ __forceinline__ void store8(T *p, int n, const Eight<float> &v) {
    if (!TAIL || n >= 8) {
        typedef T t8 __attribute__((ext_vector_type(8), aligned(sizeof(T))));
        Eight<T> x;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (T)v[e];
        *reinterpret_cast<t8 *>(p) = x;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = (T)v[e];
    }
}
template <bool TAIL>
__device__ __forceinline__ void store8(void *p, int64_t at, int type, int n, const Eight<float> &v) {
    if (type == W4A8_F32) store8<TAIL>((float *)p + at, n, v);
    else if (type == W4A8_F16) store8<TAIL>((_Float16 *)p + at, n, v);
    else store8<TAIL>((__bf16 *)p + at, n, v);
}

// ------------------------------------------------------------------ reductions
template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_of(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double row16_sum(double v) {
    v = dpp_add<0xB1>(v);      // quad_perm [1,0,3,2]
    v = dpp_add<0x4E>(v);      // quad_perm [2,3,0,1]
    v = dpp_add<0x124>(v);     // row_ror:4
    return dpp_add<0x128>(v);  // row_ror:8
}
__device__ __forceinline__ double wave_sum(double v) {
    v = row16_sum(v);
    return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// A barrier for what passes through LDS.  (__syncthreads would also wait for the stores to memory that are under way.)
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Sums and maxima over the workgroup.  Two exchange buffers in turn: a wave writes one only after
// the barrier of the reduction between, which every wave passes after it has read it.
struct Block {
    double *red;  // [2][16]
    int waves, turn = 0;

    __device__ __forceinline__ double sum(double v) {
        v = wave_sum(v);
        if (waves == 1) return v;
        double *r = red + 16 * (turn ^= 1);
        if (threadIdx.x % kWave == 0) r[threadIdx.x / kWave] = v;
        lds_barrier();
        const int i = threadIdx.x % 16;
        return row16_sum(i < waves ? r[i] : 0.0);
    }
    // of values that are not negative
    __device__ __forceinline__ float max(float v) {
        v = wave_max(v);
        if (waves == 1) return v;
        float *r = reinterpret_cast<float *>(red + 16 * (turn ^= 1));
        if (threadIdx.x % kWave == 0) r[threadIdx.x / kWave] = v;
        lds_barrier();
        const int i = threadIdx.x % 16;
        v = i < waves ? r[i] : 0.0f;
        v = dpp_max<0xB1>(v);
        v = dpp_max<0x4E>(v);
        v = dpp_max<0x124>(v);
        return dpp_max<0x128>(v);
    }
};

// 1 / sqrt(x) and 1 / x in fp64: the hardware's estimate (about 2^-24) and two Newton steps, each of which squares
// the error, so a few 2^-53 where the library's root and quotient take some sixty instructions in every lane.
__device__ __forceinline__ double rsqrt64(double x) {
    double y = __builtin_amdgcn_rsq(x);
    const double y0 = y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const double e = fma(-x * y, y, 1.0);
        y = fma(0.5 * y, e, y);
    }
    return x == __builtin_inf() ? y0 : y;  // 0
}
__device__ __forceinline__ double rcp64(double x) {
    double y = __builtin_amdgcn_rcp(x);
#pragma unroll
    for (int i = 0; i < 2; ++i) y = fma(fma(-x, y, 1.0), y, y);
    return y;
}

// Mean (LAYER) and 1 / sqrt(mean square about it + eps) of the row in v.
template <typename T, int C, bool TAIL>
__device__ __forceinline__ void stats(int kind, const Eight<T> (&v)[C], const int (&n)[C], double inv_h, double eps,
                                      Block &b, double &mean, double &inv) {
    mean = 0.0;
    inv = 1.0;
    if (kind == W4A8_NORM_NONE) return;
    double s = 0.0;
    if (kind == W4A8_NORM_LAYER) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n[c] > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) s += (double)(float)v[c][e];
            }
        mean = b.sum(s) * inv_h;
        s = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n[c] > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double d = !TAIL || e < n[c] ? (double)(float)v[c][e] - mean : 0.0;
                    s = fma(d, d, s);
                }
            }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n[c] > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fma((double)(float)v[c][e], (double)(float)v[c][e], s);
            }
    }
    inv = rsqrt64(fma(b.sum(s), inv_h, eps));
}

template <typename TY, typename TR, int C, bool TAIL>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(const NormArgs a, double inv_h, int64_t m0) {
    __shared__ double red[32];
    const int64_t m = m0 + blockIdx.x;
    const int H = (int)a.H, t = threadIdx.x, T = blockDim.x;
    Block b{red, T / kWave};
    Eight<TY> y[C];
    Eight<TR> x[C];
    int n[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int h = (c * T + t) * 8;
        n[c] = H - h;
        if (n[c] <= 0) continue;
        if (a.y) y[c] = load8<TAIL>((const TY *)a.y + m * a.ldy + h, n[c]);
        if (a.res) x[c] = load8<TAIL>((const TR *)a.res + m * a.ldr + h, n[c]);
    }
    double mean, inv;
    if (a.y) stats<TY, C, TAIL>(a.post, y, n, inv_h, a.eps, b, mean, inv);
    const double first = a.post_b ? inv : inv * a.y_scale;
    Eight<float> r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (n[c] <= 0) continue;
        const int h = (c * T + t) * 8;
        double v[8];
        if (a.y) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (double)(float)y[c][e];
            if (a.post == W4A8_NORM_LAYER) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] -= mean;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= first;
            if (a.post_w) {
                const Eight<float> w = floats_at<TAIL, float>(a.post_w, h, n[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= (double)w[e];
            }
            if (a.post_b) {
                const Eight<float> o = floats_at<TAIL, float>(a.post_b, h, n[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (v[e] + (double)o[e]) * a.y_scale;
            }
            if (a.gate) {
                const Eight<float> g = floats_at<TAIL>(a.gate, m * a.ldg + h, a.gate_type, n[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= (double)g[e];
            }
            if (a.res) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fma((double)(float)x[c][e], a.res_scale, v[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (double)(float)x[c][e] * a.res_scale;
        }
        // rounded to fp32 and to the stream's type
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] = !TAIL || e < n[c] ? (float)(TR)(float)v[e] : 0.0f;
        if (a.res_out) store8<TAIL>((TR *)a.res_out + m * a.ldro + h, n[c], r[c]);
    }
    stats<float, C, TAIL>(a.pre, r, n, inv_h, a.eps, b, mean, inv);
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (n[c] <= 0) continue;
        const int h = (c * T + t) * 8;
        double v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (double)r[c][e];
        if (a.pre == W4A8_NORM_LAYER) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] -= mean;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= inv;
        if (a.pre_w) {
            const Eight<float> w = floats_at<TAIL, float>(a.pre_w, h, n[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= (double)w[e];
        }
        if (a.pre_b) {
            const Eight<float> o = floats_at<TAIL, float>(a.pre_b, h, n[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += (double)o[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r[c][e] = (float)v[e];
            if (!TAIL || e < n[c]) top = fmaxf(top, fabsf(r[c][e]));
        }
        if (a.z) store8<TAIL>(a.z, m * a.ldz + h, a.z_type, n[c], r[c]);
    }
    if (!a.qa) return;
    const float s = b.max(top) * (1.0f / 127.0f);
    if (t == 0) a.a_scale[m] = s;
    // The fp32 quotient z / s, rounded to nearest: z times the fp64 reciprocal of s is within 2^-51 of it, relative,
    // and a quotient of two 24-bit numbers is 2^-49 away from the middle of two fp32 numbers at least.
    const double to_code = s == 0.0f ? 0.0 : rcp64((double)s);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (n[c] <= 0) continue;
        int q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float f = __builtin_rintf((float)((double)r[c][e] * to_code));
            q[e] = (int)fminf(fmaxf(f, -127.0f), 127.0f);
        }
        int8_t *out = a.qa + m * H + (c * T + t) * 8;
        if (!TAIL || n[c] >= 8) {
            typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(1)));
            u2 o;
            o.x = (q[0] & 0xFF) | (q[1] & 0xFF) << 8 | (q[2] & 0xFF) << 16 | (uint32_t)q[3] << 24;
            o.y = (q[4] & 0xFF) | (q[5] & 0xFF) << 8 | (q[6] & 0xFF) << 16 | (uint32_t)q[7] << 24;
            *reinterpret_cast<u2 *>(out) = o;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n[c]) out[e] = (int8_t)q[e];
        }
    }
}

template <typename TY, typename TR>
hipError_t launch_typed(const NormArgs &a, hipStream_t stream) {
    // Chunks a thread.  One, unless 1024 threads do not hold the row, or more than two rows a CU pass and a row would
    // take more than 512 threads: 20011 rows of 7168 take 318 us with two and 365 with one (fewer waves meet at each
    // reduction and do its scalar steps), 64 rows of 8192 6.5 us with two and 6.1 with one; 16384 rows of 1024
    // 41.2 against 39.3.
    const int chunks = (int)((a.H + 7) / 8);
    const int C = chunks > 2 * kMaxThreads ? 4 : chunks > kMaxThreads || (chunks > kMaxThreads / 2 && a.M > 512) ? 2 : 1;
    const int T = ((chunks + C - 1) / C + 63) / 64 * 64;
    const double inv_h = 1.0 / (double)a.H;
    const bool tail = a.H % 8 != 0;
    constexpr int64_t kRows = 1 << 21;  // rows per launch: fewer than 2^32 threads
    for (int64_t m0 = 0; m0 < a.M; m0 += kRows) {
        const dim3 grid((uint32_t)std::min(a.M - m0, kRows));
#define W4A8_NORM(CC)                                                                    \
    (tail ? norm_kernel<TY, TR, CC, true><<<grid, T, 0, stream>>>(a, inv_h, m0)          \
          : norm_kernel<TY, TR, CC, false><<<grid, T, 0, stream>>>(a, inv_h, m0))
        if (C == 1) W4A8_NORM(1);
        else if (C == 2) W4A8_NORM(2);
        else W4A8_NORM(4);
#undef W4A8_NORM
        if (hipError_t err = hipGetLastError(); err != hipSuccess) return err;
    }
    return hipSuccess;
}

template <typename TY>
hipError_t launch_y(const NormArgs &a, hipStream_t stream) {
    if (a.res_type == W4A8_F32) return launch_typed<TY, float>(a, stream);
    if (a.res_type == W4A8_F16) return launch_typed<TY, _Float16>(a, stream);
    return launch_typed<TY, __bf16>(a, stream);
}

}  // namespace

namespace w4a8 {

hipError_t launch_residual_norm_quantize(const NormArgs &a, hipStream_t stream) {
    if (!a.y || a.y_type == W4A8_F32) return launch_y<float>(a, stream);
    if (a.y_type == W4A8_F16) return launch_y<_Float16>(a, stream);
    return launch_y<__bf16>(a, stream);
}

}  // namespace w4a8
