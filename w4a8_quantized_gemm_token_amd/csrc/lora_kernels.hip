// lora_kernels.hip -- low-rank adapters of many requests beside a shared projection.
//
// For row m with adapter a: v = A_a x[m] (rank values), out[m] = base[m] + scale_a B_a v.
// The simple form: a wave per entry of v, a thread per output, all in fp32.
#include "block_internal.hpp"

using namespace w4a8;

namespace {

constexpr int kThreads = 256;
constexpr int64_t kSlab = 32768;  // rows per pair of launches

__device__ __forceinline__ float value_at(const void *p, int64_t i, int type) {
    if (type == W4A8_F32) return ((const float *)p)[i];
    if (type == W4A8_F16) return (float)((const _Float16 *)p)[i];
    return (float)((const __bf16 *)p)[i];
}

__device__ __forceinline__ int rank_of(const LoraArgs &a, int id) {
    const int r = a.ranks ? a.ranks[id] : a.R;
    return r < 0 ? 0 : r > a.R ? a.R : r;
}

__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(const LoraArgs a, int64_t m0) {
    const int64_t m = m0 + blockIdx.x;
    const int id = a.row_adapter[m];
    if ((uint32_t)id >= (uint32_t)a.L) return;
    const int j = blockIdx.y * (kThreads / 64) + threadIdx.x / 64, lane = threadIdx.x % 64;
    if (j >= rank_of(a, id)) return;
    const int64_t row = ((int64_t)id * a.R + j) * a.K;
    float s = 0.0f;
    for (int64_t k = lane; k < a.K; k += 64)
        s = fmaf(value_at(a.x, m * a.ldx + k, a.x_type), value_at(a.A, row + k, a.ab_type), s);
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if (lane == 0) ((float *)a.ws)[(m - m0) * a.R + j] = s;
}

__global__ __launch_bounds__(kThreads) void lora_expand_kernel(const LoraArgs a, int64_t m0) {
    const int64_t m = m0 + blockIdx.y, n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (n >= a.N) return;
    const int id = a.row_adapter[m];
    const bool none = (uint32_t)id >= (uint32_t)a.L;
    if (none && a.base == a.out) return;
    float s = 0.0f;
    const int rank = none ? 0 : rank_of(a, id);
    for (int j = 0; j < rank; ++j)
        s = fmaf(((const float *)a.ws)[(m - m0) * a.R + j], value_at(a.B, ((int64_t)id * a.N + n) * a.R + j, a.ab_type), s);
    const float b = value_at(a.base, m * a.ldb + n, a.out_type);
    const float r = rank ? b + (a.scale ? a.scale[id] : 1.0f) * s : b;
    if (a.out_type == W4A8_F32) ((float *)a.out)[m * a.ldo + n] = r;
    else if (a.out_type == W4A8_F16) ((_Float16 *)a.out)[m * a.ldo + n] = (_Float16)r;
    else ((__bf16 *)a.out)[m * a.ldo + n] = (__bf16)r;
}

}  // namespace

namespace w4a8 {

int64_t lora_ws_bytes(int64_t M, int64_t, int32_t, int32_t R) { return 4 * (M < kSlab ? M : kSlab) * R; }

hipError_t launch_lora_add(const LoraArgs &a, hipStream_t stream) {
    for (int64_t m0 = 0; m0 < a.M; m0 += kSlab) {
        const uint32_t rows = (uint32_t)(a.M - m0 < kSlab ? a.M - m0 : kSlab);
        lora_shrink_kernel<<<dim3(rows, (a.R + 3) / 4), kThreads, 0, stream>>>(a, m0);
        lora_expand_kernel<<<dim3((uint32_t)((a.N + kThreads - 1) / kThreads), rows), kThreads, 0, stream>>>(a, m0);
        if (hipError_t err = hipGetLastError(); err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace w4a8
