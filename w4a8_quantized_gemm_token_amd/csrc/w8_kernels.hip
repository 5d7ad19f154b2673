// w8_kernels.hip -- the W8A8 product on gfx950 (CDNA4) matrix cores: INT8 activations with a
// scale per token, INT8 weights with a scale per output channel.
//
//     isum[m][n] = sum_k qa[m][k] qw[n][k]                         (int32, exact: K < 2^17)
//     out[m][n]  = T(fp32(isum) * a_scale[m] * w_scale[n] + bias[n])
//
// The same product runs dense, and per expert over the slot lists of the router.  The sums are
// integers, so neither the order of k nor a split of it changes a result.
#include <algorithm>

#include "w8_internal.hpp"

using namespace w4a8dev;

namespace {

// One step of the epilogue: three fp32 roundings (the sum's conversion and two products) and
// one for the bias, then one to the output's type.
template <typename T>
__device__ __forceinline__ T finish(int32_t s, float as, float ws, float b, bool has_bias) {
    float v = ((float)s * as) * ws;
    if (has_bias) v += b;
    return (T)v;
}

__device__ __forceinline__ int64_t clamp_slots(int64_t v, int64_t max_slots) {
    return v < 0 ? 0 : (v > max_slots ? max_slots : v);
}

// ------------------------------------------------------------------ tile
// A 256-thread workgroup computes a 64 x 64 tile, four waves of 32 x 32 on
// v_mfma_i32_16x16x64_i8; 64 bytes of k are staged per step through registers into LDS rows
// padded to 80 bytes.  Rows and columns outside, and k past K, are staged as zeros.
constexpr int kTileThreads = 256, kTile = 64, kStepK = 64, kRow = 80;

template <typename T, typename SrcRow>
__device__ __forceinline__ void tile_unit(uint8_t *lds, const int8_t *__restrict__ qa,
                                          const float *__restrict__ a_scale, SrcRow src_row, int64_t slot0, int rows,
                                          int64_t K, const int8_t *__restrict__ qw,
                                          const float *__restrict__ w_scale, int64_t N, int64_t n0,
                                          const float *__restrict__ bias, T *__restrict__ out, int64_t ldo) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int lr = tid >> 2, lc = (tid & 3) * 16;
    const int64_t arow = lr < rows ? src_row(lr) : -1;
    const int64_t col = n0 + lr;
    v4i acc[2][2] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kStepK) {
        const bool kin = k0 + lc < K;
        v4i a = {}, b = {};
        if (kin && arow >= 0) a = *reinterpret_cast<const v4i *>(qa + arow * K + k0 + lc);
        if (kin && col < N) b = *reinterpret_cast<const v4i *>(qw + col * K + k0 + lc);
        __syncthreads();
        *reinterpret_cast<v4i *>(lds + lr * kRow + lc) = a;
        *reinterpret_cast<v4i *>(lds + (kTile + lr) * kRow + lc) = b;
        __syncthreads();
        v4i af[2], bf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            af[i] = *reinterpret_cast<const v4i *>(lds + (wm * 32 + i * 16 + (lane & 15)) * kRow + (lane >> 4) * 16);
            bf[i] = *reinterpret_cast<const v4i *>(lds + (kTile + wn * 32 + i * 16 + (lane & 15)) * kRow +
                                                   (lane >> 4) * 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i], bf[j], acc[i][j], 0, 0, 0);
    }
    // accumulator: rows 4 (l >> 4) + r, column l & 15
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int m = wm * 32 + i * 16 + 4 * (lane >> 4) + r;
            const int64_t row = m < rows ? src_row(m) : -1;
            if (row < 0) continue;
            const float as = a_scale[row];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t n = n0 + wn * 32 + j * 16 + (lane & 15);
                if (n < N)
                    out[(slot0 + m) * ldo + n] =
                        finish<T>(acc[i][j][r], as, w_scale[n], bias ? bias[n] : 0.0f, bias != nullptr);
            }
        }
    __syncthreads();
}

template <typename T>
__global__ __launch_bounds__(kTileThreads) void gemm_w8a8_kernel(const int8_t *__restrict__ qa,
                                                                 const float *__restrict__ a_scale, int64_t M,
                                                                 int64_t K, const int8_t *__restrict__ qw,
                                                                 const float *__restrict__ w_scale, int64_t N,
                                                                 const float *__restrict__ bias, T *__restrict__ out,
                                                                 int64_t ldo) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kTile * kRow];
    const int64_t nt = (N + kTile - 1) / kTile;
    const int64_t m0 = (int64_t)blockIdx.x / nt * kTile, n0 = (int64_t)blockIdx.x % nt * kTile;
    const int rows = (int)((M - m0) < kTile ? (M - m0) : kTile);
    tile_unit<T>(lds, qa, a_scale, [&](int r) { return m0 + r; }, m0, rows, K, qw, w_scale, N, n0, bias, out, ldo);
}

// One workgroup per (64-column tile, expert), walking the expert's slots 64 at a time.
__global__ __launch_bounds__(kTileThreads) void grouped_w8a8_kernel(
    const int8_t *__restrict__ qa, const float *__restrict__ a_scale, int64_t R, const int32_t *__restrict__ row_index,
    const int32_t *__restrict__ offsets, int64_t K, const int8_t *__restrict__ qw, const float *__restrict__ w_scale,
    int64_t N, int64_t max_slots, float *__restrict__ out) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kTile * kRow];
    const int64_t e = blockIdx.y, n0 = (int64_t)blockIdx.x * kTile;
    const int64_t s0 = clamp_slots(offsets[e], max_slots), s1 = clamp_slots(offsets[e + 1], max_slots);
    for (int64_t s = s0; s < s1; s += kTile) {
        const int rows = (int)((s1 - s) < kTile ? (s1 - s) : kTile);
        auto src = [&](int r) -> int64_t {
            const int64_t row = row_index ? (int64_t)row_index[s + r] : s + r;
            return row >= 0 && row < R ? row : -1;
        };
        tile_unit<float>(lds, qa, a_scale, src, s, rows, K, qw + e * N * K, w_scale + e * N, N, n0, nullptr, out, N);
    }
}

}  // namespace

namespace w4a8 {

template <typename T>
static hipError_t gemm_w8a8_typed(const int8_t *qa, const float *a_scale, int64_t M, int64_t K, const int8_t *qw,
                                  const float *w_scale, int64_t N, const float *bias, T *out, int64_t ldo,
                                  hipStream_t stream) {
    const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
    hipLaunchKernelGGL(gemm_w8a8_kernel<T>, dim3((uint32_t)tiles), dim3(kTileThreads), 0, stream, qa, a_scale, M, K,
                       qw, w_scale, N, bias, out, ldo);
    return hipGetLastError();
}

hipError_t launch_gemm_w8a8(const int8_t *qa, const float *a_scale, int64_t M, int64_t K, const int8_t *qw,
                            const float *w_scale, int64_t N, const float *bias, void *out, int32_t out_type,
                            int64_t ldo, hipStream_t stream) {
    switch (out_type) {
    case W4A8_F16:
        return gemm_w8a8_typed(qa, a_scale, M, K, qw, w_scale, N, bias, (_Float16 *)out, ldo, stream);
    case W4A8_BF16:
        return gemm_w8a8_typed(qa, a_scale, M, K, qw, w_scale, N, bias, (__bf16 *)out, ldo, stream);
    default:
        return gemm_w8a8_typed(qa, a_scale, M, K, qw, w_scale, N, bias, (float *)out, ldo, stream);
    }
}

hipError_t launch_grouped_gemm_w8a8(const int8_t *qa, const float *a_scale, int64_t R, const int32_t *row_index,
                                    const int32_t *expert_offsets, int32_t E, int64_t K, const int8_t *qw,
                                    const float *w_scale, int64_t N, int64_t max_slots, float *out,
                                    hipStream_t stream) {
    const dim3 grid((uint32_t)((N + kTile - 1) / kTile), (uint32_t)E);
    hipLaunchKernelGGL(grouped_w8a8_kernel, grid, dim3(kTileThreads), 0, stream, qa, a_scale, R, row_index,
                       expert_offsets, K, qw, w_scale, N, max_slots, out);
    return hipGetLastError();
}

}  // namespace w4a8
