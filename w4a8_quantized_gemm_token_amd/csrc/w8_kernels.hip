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
// A workgroup of WM x WN waves computes a BM x BN tile, each wave RB x CB blocks of 16 x 16 on
// v_mfma_i32_16x16x64_i8 with the weights as the first operand: a lane then holds, of one row
// m, four neighbouring output channels per block, and the weight rows of a wave's blocks are
// taken so that its CB blocks make 4 CB neighbours (see wrow below), which it stores as whole
// 16-byte pieces.
// Both operands go straight from memory into LDS (16 bytes per lane), 128 bytes of k per stage,
// NST stages.  LDS rows are 128 bytes; the 16-byte chunk c of row r sits at chunk c ^ key(r), so
// that the 16 rows of a fragment read fall in distinct banks.
// A stage is computed in two halves of 64 k.  The fragments of a half are read while the half
// before it is multiplied, so the one barrier per stage stands between the halves of stage g:
// there every wave holds the fragments of its second half in registers (the stage's buffer is
// free for stage g + NST) and stage g + 1 has landed (its first half may be read).
typedef __attribute__((address_space(3))) void *lds_ptr_t;
typedef const __attribute__((address_space(1))) void *glb_ptr_t;

// s_waitcnt immediate: at most vm memory loads and lgkm LDS accesses outstanding
constexpr int waitcnt(int vm, int lgkm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)0xFFFFFFFF, 0x00020000);
}

template <int BM_, int BN_, int WM_, int WN_, int NST_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_;
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int RB = BM / WM / 16, CB = BN / WN / 16;
    static constexpr int LA = BM / 8 / kWaves, LB = BN / 8 / kWaves;  // 1 KB loads per wave and stage
    static constexpr int kStageA = BM * 128, kStage = (BM + BN) * 128, kLds = NST * kStage;
    static_assert(LA * 8 * kWaves == BM && LB * 8 * kWaves == BN, "whole loads per wave");
    static_assert(kLds <= 160 * 1024, "LDS of one CU");
    // the fragment row i (0..15) of a wave's column block cb is its weight row wrow(i, cb)
    __device__ static int wrow(int i, int cb) { return 4 * CB * (i >> 2) + 4 * cb + (i & 3); }
    __device__ static int key_a(int r) { return (r >> 1) & 7; }
    __device__ static int key_b(int r) { return ((r >> 1) & 1) | (((r / (4 * CB)) & 3) << 1); }
};

// src_row(r), r < rows: activation row of the tile's row r, or -1 (computed as row 0, not stored).
// VEC: output rows start 16-byte aligned.
template <typename C, typename T, typename SrcRow>
__device__ __forceinline__ void tile_unit(uint8_t *lds, const int8_t *__restrict__ qa,
                                          const float *__restrict__ a_scale, SrcRow src_row, int64_t slot0, int rows,
                                          int64_t K, const int8_t *__restrict__ qw,
                                          const float *__restrict__ w_scale, int64_t N, int64_t n0,
                                          const float *__restrict__ bias, T *__restrict__ out, int64_t ldo, bool vec) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int full = (int)(K >> 7), steps = (int)((K + 127) >> 7);  // whole stages, all stages
    const int tail = (int)(K & 127) >> 4;                          // chunks of a last part stage

    // ---- loads: lane L of load j fills chunk L & 7 of row 8 (L? wave + j) + (L >> 3)
    const int8_t *aptr[C::LA];
    uint32_t boff[C::LB];
    int ach[C::LA], bch[C::LB];
#pragma unroll
    for (int j = 0; j < C::LA; ++j) {
        const int r = 8 * (C::LA * wave + j) + (lane >> 3);
        int64_t src = src_row(r < rows ? r : rows - 1);
        if (src < 0) src = 0;
        ach[j] = (lane & 7) ^ C::key_a(r);
        aptr[j] = qa + src * K + 16 * ach[j];
    }
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(qw + n0 * K);
#pragma unroll
    for (int j = 0; j < C::LB; ++j) {
        const int r = 8 * (C::LB * wave + j) + (lane >> 3);
        const int64_t c = n0 + r < N ? r : N - 1 - n0;
        bch[j] = (lane & 7) ^ C::key_b(r);
        boff[j] = (uint32_t)(c * K) + 16u * (uint32_t)bch[j];
    }
    auto issue = [&](int g, int st) {
        uint8_t *da = lds + st * C::kStage + 1024 * (C::LA * wave);
        uint8_t *db = lds + st * C::kStage + C::kStageA + 1024 * (C::LB * wave);
        if (g < full) {
#pragma unroll
            for (int j = 0; j < C::LB; ++j)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(db + 1024 * j), 16, (int)boff[j], g * 128, 0, 0);
#pragma unroll
            for (int j = 0; j < C::LA; ++j)
                __builtin_amdgcn_global_load_lds((glb_ptr_t)(aptr[j] + (int64_t)g * 128), (lds_ptr_t)(da + 1024 * j), 16,
                                                 0, 0);
        } else {
            // the part stage: chunks past K are zeros on the activations' side (whatever the other
            // side's buffer holds there) and not loaded
#pragma unroll
            for (int j = 0; j < C::LB; ++j)
                if (bch[j] < tail)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(db + 1024 * j), 16, (int)boff[j], g * 128,
                                                             0, 0);
#pragma unroll
            for (int j = 0; j < C::LA; ++j) {
                if (ach[j] < tail)
                    __builtin_amdgcn_global_load_lds((glb_ptr_t)(aptr[j] + (int64_t)g * 128),
                                                     (lds_ptr_t)(da + 1024 * j), 16, 0, 0);
                else *reinterpret_cast<v4i *>(da + 1024 * j + 16 * lane) = v4i{0, 0, 0, 0};
            }
        }
    };

    // ---- fragments: lane l takes row (l & 15) of a block, chunk 4 ks + (l >> 4)
    const int fr = lane & 15, qd = lane >> 4;
    int aofs[2], bofs[2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const int ra = wm * C::RB * 16 + fr, rw = wn * C::CB * 16 + C::wrow(fr, 0);
        aofs[ks] = ra * 128 + (((4 * ks + qd) ^ C::key_a(ra)) << 4);
        bofs[ks] = C::kStageA + rw * 128 + (((4 * ks + qd) ^ C::key_b(rw)) << 4);
    }
    struct Frags {
        v4i a[C::RB], b[C::CB];
    };
    auto read = [&](Frags &f, int st, int ks) {
        const uint8_t *pa = lds + st * C::kStage + aofs[ks], *pb = lds + st * C::kStage + bofs[ks];
#pragma unroll
        for (int j = 0; j < C::CB; ++j) f.b[j] = *reinterpret_cast<const v4i *>(pb + 512 * j);  // wrow steps by 4
#pragma unroll
        for (int i = 0; i < C::RB; ++i) f.a[i] = *reinterpret_cast<const v4i *>(pa + 2048 * i);
    };
    v4i acc[C::RB][C::CB] = {};
    auto mul = [&](const Frags &f) {
#pragma unroll
        for (int i = 0; i < C::RB; ++i)
#pragma unroll
            for (int j = 0; j < C::CB; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
    };
    // reads of the next half spread between the products of this one
    auto interleave = [&]() {
        constexpr int R = C::RB + C::CB, M = C::RB * C::CB, PER = M / R > 0 ? M / R : 1;
#pragma unroll
        for (int q = 0; q < R; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
    };

    // ---- prologue
#pragma unroll
    for (int g = 0; g < C::NST; ++g)
        if (g < steps) issue(g, g);
    __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    Frags f0, f1;
    read(f0, 0, 0);
    int st = 0;
    for (int g = 0; g < steps - 1; ++g) {
        read(f1, st, 1);
        mul(f0);
        interleave();
        __asm__ volatile("" ::: "memory");
        // stage g + 1 has landed; the NST - 2 stages behind it may be in flight (a part stage
        // among them has fewer loads: wait for all)
        if (C::NST > 2 && g + C::NST - 1 < full)
            __builtin_amdgcn_s_waitcnt(waitcnt((C::NST - 2) * (C::LA + C::LB), 0));
        else __builtin_amdgcn_s_waitcnt(waitcnt(0, 0));
        __builtin_amdgcn_s_barrier();
        __asm__ volatile("" ::: "memory");
        if (g + C::NST < steps) issue(g + C::NST, st);
        st = st + 1 == C::NST ? 0 : st + 1;
        read(f0, st, 0);
        mul(f1);
        interleave();
    }
    read(f1, st, 1);
    mul(f0);
    interleave();
    mul(f1);

    // ---- epilogue: lane l holds row 16 i + (l & 15) and, of block j, channels 4 CB (l >> 4) + 4 j + r
    const int64_t nb = n0 + wn * C::CB * 16 + 4 * C::CB * qd;
    float ws[4 * C::CB], bv[4 * C::CB];
#pragma unroll
    for (int c = 0; c < 4 * C::CB; ++c) {
        const int64_t n = nb + c < N ? nb + c : N - 1;
        ws[c] = w_scale[n];
        bv[c] = bias ? bias[n] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < C::RB; ++i) {
        const int m = wm * C::RB * 16 + 16 * i + fr;
        const int64_t row = m < rows ? src_row(m) : -1;
        if (row < 0) continue;
        const float as = a_scale[row];
        T *o = out + (slot0 + m) * ldo + nb;
        constexpr int V = 16 / sizeof(T);  // elements of a 16-byte store
        if constexpr (4 * C::CB >= V) {
#pragma unroll
            for (int c0 = 0; c0 < 4 * C::CB; c0 += V) {
                typedef T vt __attribute__((ext_vector_type(V)));
                vt v;
#pragma unroll
                for (int c = 0; c < V; ++c)
                    v[c] = finish<T>(acc[i][(c0 + c) >> 2][(c0 + c) & 3], as, ws[c0 + c], bv[c0 + c], bias != nullptr);
                if (vec && nb + c0 + V <= N) *reinterpret_cast<vt *>(o + c0) = v;
                else {
#pragma unroll
                    for (int c = 0; c < V; ++c)
                        if (nb + c0 + c < N) o[c0 + c] = v[c];
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4 * C::CB; ++c)
                if (nb + c < N)
                    o[c] = finish<T>(acc[i][c >> 2][c & 3], as, ws[c], bv[c], bias != nullptr);
        }
    }
}

// Bijective XCD-aware order: workgroup b runs on XCD b % 8; each XCD gets a contiguous range of
// tiles, taken in panels of PM row tiles, so the tiles that an XCD runs at a time share rows
// and columns in its L2.
template <int PM>
__device__ __forceinline__ void panel_tile(int64_t b, int64_t mt, int64_t nt, int64_t &tm, int64_t &tn) {
    const int64_t q = mt * nt / 8, r = mt * nt % 8, x = b % 8;
    const int64_t i = x * q + (x < r ? x : r) + b / 8;
    const int64_t p = i / (PM * nt);
    const int64_t pm = (mt - PM * p) < PM ? (mt - PM * p) : PM;
    const int64_t ip = i - p * PM * nt;
    tm = PM * p + ip % pm;
    tn = ip / pm;
}

template <typename C, typename T>
__global__ __launch_bounds__(C::kThreads) void gemm_w8a8_tile_kernel(const int8_t *__restrict__ qa,
                                                                     const float *__restrict__ a_scale, int64_t M,
                                                                     int64_t K, const int8_t *__restrict__ qw,
                                                                     const float *__restrict__ w_scale, int64_t N,
                                                                     const float *__restrict__ bias,
                                                                     T *__restrict__ out, int64_t ldo, bool vec) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
    const int64_t mt = (M + C::BM - 1) / C::BM, nt = (N + C::BN - 1) / C::BN;
    int64_t tm, tn;
    panel_tile<4>(blockIdx.x, mt, nt, tm, tn);
    const int64_t m0 = tm * C::BM;
    const int rows = (int)((M - m0) < C::BM ? (M - m0) : C::BM);
    tile_unit<C, T>(lds, qa, a_scale, [&](int r) { return m0 + r; }, m0, rows, K, qw, w_scale, N, tn * C::BN, bias, out,
                    ldo, vec);
}

using Tile256 = Tile<256, 256, 2, 4, 2>;
using Tile128 = Tile<128, 128, 2, 2, 2>;

// ------------------------------------------------------------------ plain tile
// A 256-thread workgroup computes a 64 x 64 tile, four waves of 32 x 32 on
// v_mfma_i32_16x16x64_i8; 64 bytes of k are staged per step through registers into LDS rows
// padded to 80 bytes.  Rows and columns outside, and k past K, are staged as zeros.
constexpr int kTileThreads = 256, kTile = 64, kStepK = 64, kRow = 80;

template <typename T, typename SrcRow>
__device__ __forceinline__ void plain_unit(uint8_t *lds, const int8_t *__restrict__ qa,
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
__global__ __launch_bounds__(kTileThreads) void gemm_w8a8_plain_kernel(const int8_t *__restrict__ qa,
                                                                 const float *__restrict__ a_scale, int64_t M,
                                                                 int64_t K, const int8_t *__restrict__ qw,
                                                                 const float *__restrict__ w_scale, int64_t N,
                                                                 const float *__restrict__ bias, T *__restrict__ out,
                                                                 int64_t ldo) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kTile * kRow];
    const int64_t nt = (N + kTile - 1) / kTile;
    const int64_t m0 = (int64_t)blockIdx.x / nt * kTile, n0 = (int64_t)blockIdx.x % nt * kTile;
    const int rows = (int)((M - m0) < kTile ? (M - m0) : kTile);
    plain_unit<T>(lds, qa, a_scale, [&](int r) { return m0 + r; }, m0, rows, K, qw, w_scale, N, n0, bias, out, ldo);
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
        plain_unit<float>(lds, qa, a_scale, src, s, rows, K, qw + e * N * K, w_scale + e * N, N, n0, nullptr, out, N);
    }
}

}  // namespace

namespace w4a8 {

template <typename C, typename T>
static hipError_t launch_tile(const int8_t *qa, const float *a_scale, int64_t M, int64_t K, const int8_t *qw,
                              const float *w_scale, int64_t N, const float *bias, T *out, int64_t ldo, bool vec,
                              hipStream_t stream) {
    const int64_t tiles = ((M + C::BM - 1) / C::BM) * ((N + C::BN - 1) / C::BN);
    hipLaunchKernelGGL((gemm_w8a8_tile_kernel<C, T>), dim3((uint32_t)tiles), dim3(C::kThreads), 0, stream, qa,
                       a_scale, M, K, qw, w_scale, N, bias, out, ldo, vec);
    return hipGetLastError();
}

template <typename T>
static hipError_t gemm_w8a8_typed(const int8_t *qa, const float *a_scale, int64_t M, int64_t K, const int8_t *qw,
                                  const float *w_scale, int64_t N, const float *bias, T *out, int64_t ldo,
                                  hipStream_t stream) {
    const bool vec = (uintptr_t)out % 16 == 0 && ldo * (int64_t)sizeof(T) % 16 == 0;
    if (M > 128) return launch_tile<Tile256>(qa, a_scale, M, K, qw, w_scale, N, bias, out, ldo, vec, stream);
    return launch_tile<Tile128>(qa, a_scale, M, K, qw, w_scale, N, bias, out, ldo, vec, stream);
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
