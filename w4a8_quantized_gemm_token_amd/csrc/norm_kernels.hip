// norm_kernels.hip -- between two blocks of a model: the post-norm of a block's output, its gate
// and the residual join, the next block's norm, and the INT8 codes that its products read.
//
// The simple form: a workgroup per row that reads the row again for every reduction.  The
// arithmetic up to z is fp64 (see the entry point).
#include "block_internal.hpp"

using namespace w4a8;
using namespace w4a8dev;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

__device__ __forceinline__ float value_at(const void *p, int64_t i, int type) {
    if (type == W4A8_F32) return ((const float *)p)[i];
    if (type == W4A8_F16) return (float)((const _Float16 *)p)[i];
    return (float)((const __bf16 *)p)[i];
}

// v as its type holds it, through fp32
__device__ __forceinline__ float rounded(float v, int type) {
    if (type == W4A8_F16) return (float)(_Float16)v;
    if (type == W4A8_BF16) return (float)(__bf16)v;
    return v;
}
__device__ __forceinline__ void store_at(void *p, int64_t i, int type, float v) {
    if (type == W4A8_F32) ((float *)p)[i] = v;
    else if (type == W4A8_F16) ((_Float16 *)p)[i] = (_Float16)v;
    else ((__bf16 *)p)[i] = (__bf16)v;
}

template <typename T, typename Op>
__device__ T block_all(T v, T *red, Op op) {
    for (int o = 32; o > 0; o >>= 1) v = op(v, __shfl_xor(v, o, kWave));
    __syncthreads();
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kWaves; ++i) v = op(v, red[i]);
    return v;
}

__global__ __launch_bounds__(kThreads) void norm_kernel(const NormArgs a, int64_t m0) {
    __shared__ double red[kWaves];
    __shared__ float fred[kWaves];
    __shared__ float row[kNormMaxH];  // the stream's row, then z's
    const int64_t m = m0 + blockIdx.x;
    const int H = (int)a.H, t = threadIdx.x;
    const auto add = [](double p, double q) { return p + q; };
    // mean and 1 / sqrt(mean square + eps) of a row of values
    const auto stats = [&](int kind, auto at, double &mean, double &inv) {
        mean = 0.0;
        inv = 1.0;
        if (kind == W4A8_NORM_NONE) return;
        double s = 0.0;
        if (kind == W4A8_NORM_LAYER) {
            for (int h = t; h < H; h += kThreads) s += at(h);
            mean = block_all(s, red, add) / H;
            s = 0.0;
        }
        for (int h = t; h < H; h += kThreads) {
            const double d = at(h) - mean;
            s = fma(d, d, s);
        }
        inv = 1.0 / sqrt(block_all(s, red, add) / H + a.eps);
    };
    const auto y_at = [&](int h) { return (double)value_at(a.y, m * a.ldy + h, a.y_type); };
    double mean = 0.0, inv = 1.0;
    if (a.y) stats(a.post, y_at, mean, inv);
    for (int h = t; h < H; h += kThreads) {
        double v = 0.0;
        if (a.y) {
            v = (y_at(h) - mean) * inv;
            if (a.post_w) v *= a.post_w[h];
            if (a.post_b) v += a.post_b[h];
            if (a.gate) v *= value_at(a.gate, m * a.ldg + h, a.gate_type);
            v *= a.y_scale;
        }
        if (a.res) v += a.res_scale * value_at(a.res, m * a.ldr + h, a.res_type);
        const float r = (float)v;
        if (a.res_out) store_at(a.res_out, m * a.ldro + h, a.res_type, r);
        row[h] = rounded(r, a.res_type);
    }
    stats(a.pre, [&](int h) { return (double)row[h]; }, mean, inv);  // each thread reads what it wrote
    float top = 0.0f;
    for (int h = t; h < H; h += kThreads) {
        double v = ((double)row[h] - mean) * inv;
        if (a.pre_w) v *= a.pre_w[h];
        if (a.pre_b) v += a.pre_b[h];
        const float z = (float)v;
        if (a.z) store_at(a.z, m * a.ldz + h, a.z_type, z);
        row[h] = z;
        top = fmaxf(top, fabsf(z));
    }
    if (!a.qa) return;
    top = block_all(top, fred, [](float p, float q) { return fmaxf(p, q); });
    const float s = top * (1.0f / 127.0f);
    if (t == 0) a.a_scale[m] = s;
    for (int h = t; h < H; h += kThreads) a.qa[m * H + h] = (int8_t)quantize_i8(row[h], s);
}

}  // namespace

namespace w4a8 {

hipError_t launch_residual_norm_quantize(const NormArgs &a, hipStream_t stream) {
    constexpr int64_t kRows = 1 << 22;  // rows per launch: fewer than 2^32 threads
    for (int64_t m0 = 0; m0 < a.M; m0 += kRows) {
        norm_kernel<<<dim3((uint32_t)(a.M - m0 < kRows ? a.M - m0 : kRows)), kThreads, 0, stream>>>(a, m0);
        if (hipError_t err = hipGetLastError(); err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace w4a8
