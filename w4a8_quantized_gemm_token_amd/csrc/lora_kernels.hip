// lora_kernels.hip -- low-rank adapters of many requests beside a shared projection.
//
// For row m with adapter a: v = A_a x[m] (rank values), out[m] = base[m] + scale_a B_a v.
// Two launches: the shrink product leaves parts of v per range of k in the workspace, the expand
// product adds them up and walks the output.  Both go by tiles of 64 rows as they stand: a wave's
// lanes hold the 64 adapter ids, the distinct ones are found with ballots, and each one's rows are
// gathered into 16-row columns of the matrix instruction, so rows of one adapter share its loads
// without being sorted beforehand, and no row can be met twice.
//
// Arithmetic: the matrix cores take 16-bit operands.  fp32 values enter as sums of bf16 parts, each
// the next 8 bits cut off the rest (three hold all 24, two hold 16, which 16-bit outputs do with);
// an fp16 value beside bf16 is two such parts, exactly.  v meets fp16 weights as two fp16 parts (22
// bits) after a scaling of its row by a power of two.  All sums are fp32.
#include "block_internal.hpp"

#include <algorithm>
#include <type_traits>

using namespace w4a8;
using namespace w4a8dev;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 64;         // rows of a tile, one a lane
constexpr int kWindow = 64;       // k of a wave's step: 16 a lane group, two matrix instructions
constexpr int64_t kSlab = 32768;  // rows per pair of launches

typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
template <typename T>
using Eight = T __attribute__((ext_vector_type(8)));

// Eight elements in a row at their type's alignment.
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T *p) {
    typedef T t8 __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    return *reinterpret_cast<const t8 *>(p);
}
template <typename T>
__device__ __forceinline__ Eight<T> zero8() {
    Eight<T> z = {};
    return z;
}

__device__ __forceinline__ f4 mfma(bf8 a, bf8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// ------------------------------------------------------------------ operands in parts
// part[i] = the next 8 bits of v, cut off; an infinity has no rest.
template <int N>
__device__ __forceinline__ void split(const float (&v)[8], bf8 (&part)[N]) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v4u o;
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            o[e / 2] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, r[e + 1]), __builtin_bit_cast(uint32_t, r[e]),
                                             0x07060302);
        part[i] = __builtin_bit_cast(bf8, o);
        if (i + 1 < N) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float head = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, r[e]) & 0xFFFF0000u);
                const float rest = r[e] - head;
                r[e] = i == 0 && __builtin_amdgcn_classf(r[e], 0x204) ? 0.0f : rest;
            }
        }
    }
}

// The operand of type T beside one of type U: itself where both are the same 16-bit type, parts otherwise (P for fp32).
template <typename T, typename U, int P>
struct Operand {
    static constexpr int kParts = std::is_same<T, float>::value ? P : std::is_same<T, _Float16>::value ? 2 : 1;
    typedef bf8 V;
    static __device__ __forceinline__ void of(const Eight<T> &x, V (&part)[kParts]) {
        if constexpr (std::is_same<T, __bf16>::value) {
            part[0] = x;
        } else {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
            split<kParts>(v, part);
        }
    }
};
template <int P>
struct Operand<_Float16, _Float16, P> {
    static constexpr int kParts = 1;
    typedef h8 V;
    static __device__ __forceinline__ void of(const Eight<_Float16> &x, V (&part)[1]) { part[0] = x; }
};

// ------------------------------------------------------------------ groups of a tile
// Calls f(adapter, mask of its lanes) for each distinct valid id, those whose turn modulo `of` is `turn`.
template <typename F>
__device__ __forceinline__ void for_each_adapter(int id, bool valid, int turn, int of, F &&f) {
    uint64_t left = __ballot(valid);
    for (int c = 0; left; c = c + 1 == of ? 0 : c + 1) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t mask = __ballot(valid && id == a);
        left &= ~mask;
        if (c == turn) f(a, mask);
    }
}

__device__ __forceinline__ int rank_of(const LoraArgs &a, int id) {
    const int r = a.ranks ? a.ranks[id] : a.R;
    return r < 0 ? 0 : r > a.R ? a.R : r;
}

// The lanes of mask in a row in list[]; all threads of the workgroup, between barriers.
__device__ __forceinline__ void gather_rows(uint64_t mask, uint8_t *list) {
    __syncthreads();
    if (threadIdx.x < kTile && (mask >> threadIdx.x & 1))
        list[__popcll(mask & ((1ull << threadIdx.x) - 1))] = (uint8_t)threadIdx.x;
    __syncthreads();
}

// ------------------------------------------------------------------ shrink
// v[token][j] over windows [w0, w1) of k for cnt rows in list and 16 RT ranks from j0; waves take windows in turn.
// Matrix rows are ranks, matrix columns tokens.
template <typename X, typename W, int P, int TT, int RT>
__device__ __forceinline__ void shrink_group(const LoraArgs &a, int64_t row0, int64_t slab, int id, int rank, int j0, int cnt,
                                             const uint8_t *list, int w0, int w1, float *part, f4 (*red)[RT][kWave]) {
    using OX = Operand<X, W, P>;
    using OW = Operand<W, X, P>;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, col = lane % 16, g = lane / 16;
    const X *px[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int i = t * 16 + col;
        px[t] = (const X *)a.x + (row0 + list[i < cnt ? i : 0]) * a.ldx + 16 * g;
    }
    const W *pw[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int j = j0 + r * 16 + col;
        pw[r] = (const W *)a.A + ((int64_t)id * a.R + (j < rank ? j : rank - 1)) * a.K + 16 * g;
    }
    f4 acc[TT][RT] = {};
    const auto step = [&](const Eight<W> (&rw)[RT][2], const Eight<X> (&rx)[TT][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            typename OW::V fw[RT][OW::kParts];
#pragma unroll
            for (int r = 0; r < RT; ++r) OW::of(rw[r][h], fw[r]);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                typename OX::V fx[OX::kParts];
                OX::of(rx[t][h], fx);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int p = 0; p < OX::kParts; ++p)
#pragma unroll
                        for (int q = 0; q < OW::kParts; ++q)
                            // products of parts that lie below what the parts hold are left out
                            if (q == 0 || p + q < (OX::kParts > 1 ? OX::kParts : 2)) acc[t][r] = mfma(fw[r][q], fx[p], acc[t][r]);
            }
        }
    };
    const int whole = (int)(a.K / kWindow);
    for (int w = w0 + wave; w < w1; w += kWaves) {
        Eight<W> rw[RT][2];
        Eight<X> rx[TT][2];
        const int64_t k = (int64_t)w * kWindow;
        if (w < whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int r = 0; r < RT; ++r) rw[r][h] = load8(pw[r] + k + 8 * h);
#pragma unroll
                for (int t = 0; t < TT; ++t) rx[t][h] = load8(px[t] + k + 8 * h);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = k + 16 * g + 8 * h < a.K;
#pragma unroll
                for (int r = 0; r < RT; ++r) rw[r][h] = in ? load8(pw[r] + k + 8 * h) : zero8<W>();
#pragma unroll
                for (int t = 0; t < TT; ++t) rx[t][h] = in ? load8(px[t] + k + 8 * h) : zero8<X>();
            }
        }
        step(rw, rx);
    }
    // the waves' sums together, and to the workspace: lane has ranks 4 g .. 4 g + 3 of its tile, token col
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        if (t) __syncthreads();
#pragma unroll
        for (int r = 0; r < RT; ++r) red[wave][r][lane] = acc[t][r];
        __syncthreads();
        const int i = t * 16 + col;
        for (int r = wave; r < RT; r += kWaves) {
            const int j = j0 + r * 16 + 4 * g;
            f4 s = red[0][r][lane];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) s += red[w][r][lane];
            if (i < cnt && j < a.R) *reinterpret_cast<f4 *>(part + (slab + list[i]) * a.R + j) = s;
        }
    }
}

template <typename X, typename W, int P, int RT>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(const LoraArgs a, int64_t m0, int rows, int turns, int per) {
    __shared__ f4 red[kWaves][RT][kWave];
    __shared__ uint8_t list[kTile];
    const int split = blockIdx.y / turns, turn = blockIdx.y % turns, j0 = blockIdx.z * RT * 16;
    const int row = blockIdx.x * kTile + threadIdx.x % kWave;
    const int id = row < rows ? a.row_adapter[m0 + row] : -1;
    const int windows = (int)((a.K + kWindow - 1) / kWindow);
    const int w0 = split * per, w1 = min(w0 + per, windows);
    float *part = (float *)a.ws + (int64_t)split * rows * a.R;
    const int64_t slab = (int64_t)blockIdx.x * kTile, row0 = m0 + slab;
    for_each_adapter(id, (uint32_t)id < (uint32_t)a.L, turn, turns, [&](int ad, uint64_t mask) {
        const int rank = rank_of(a, ad);
        if (j0 >= rank) return;
        gather_rows(mask, list);
        const int cnt = __popcll(mask);
        if (cnt <= 16) shrink_group<X, W, P, 1, RT>(a, row0, slab, ad, rank, j0, cnt, list, w0, w1, part, red);
        else if (cnt <= 32) shrink_group<X, W, P, 2, RT>(a, row0, slab, ad, rank, j0, cnt, list, w0, w1, part, red);
        else shrink_group<X, W, P, 4, RT>(a, row0, slab, ad, rank, j0, cnt, list, w0, w1, part, red);
    });
}

// ------------------------------------------------------------------ expand
// v beside weights of type W: bf16 parts as above (P of them), or two fp16 parts of the scaled row.
template <typename W, int P>
struct Held {
    static constexpr bool kScaled = std::is_same<W, _Float16>::value;
    static constexpr int kParts = kScaled ? 2 : P;
};

// Columns: a wave's step is NT matrix tiles of 16 columns, dealt so that a lane's four rows of every tile are NT * 4
// columns in a row (32 bytes of output): tile q, matrix row 4 g + i is column 4 NT g + 4 q + i.
template <typename T>
constexpr int tiles_of() {
    return sizeof(T) == 4 ? 2 : 4;
}

template <typename W, typename T, int P, int KS, int TT>
__device__ __forceinline__ void expand_group(const LoraArgs &a, int64_t row0, int id, int rank, int cnt, const uint8_t *list,
                                             const Eight<W> *vp, const float *undo, int64_t n0, int64_t n1) {
    constexpr int NT = tiles_of<T>(), kStep = 16 * NT, kParts = Held<W, P>::kParts;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, col = lane % 16, g = lane / 16;
    const float scale = a.scale ? a.scale[id] : 1.0f;
    const W *pb = (const W *)a.B + (int64_t)id * a.N * a.R + 8 * g;
    const T *base[TT];
    T *out[TT];
    float f[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int i = t * 16 + col;
        const int64_t row = row0 + list[i < cnt ? i : 0];
        base[t] = (const T *)a.base + row * a.ldb;
        out[t] = (T *)a.out + row * a.ldo;
        f[t] = Held<W, P>::kScaled ? scale * undo[i < cnt ? i : 0] : scale;
    }
    for (int64_t n = n0 + wave * kStep; n < n1; n += kWaves * kStep) {
        const bool whole = n + kStep <= a.N;
        const int64_t c = n + 4 * NT * g;  // the lane's columns c .. c + 4 NT - 1
        typedef T tq __attribute__((ext_vector_type(4 * NT), aligned(sizeof(T))));
        tq have[TT];
        if (whole) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
                if (t * 16 + col < cnt) have[t] = *reinterpret_cast<const tq *>(base[t] + c);
        }
        f4 acc[TT][NT] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks * 32 >= rank) break;
            Eight<W> fb[NT];
            const int rest = rank - ks * 32 - 8 * g;  // ranks from this lane's eight on
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                const int64_t nn = n + 4 * NT * (col / 4) + 4 * q + col % 4;
                fb[q] = rest > 0 ? load8(pb + (nn < a.N ? nn : a.N - 1) * a.R + ks * 32) : zero8<W>();
            }
            if (rank & 7) {  // ranks past the adapter's own, whatever they hold
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e) fb[q][e] = e < rest ? fb[q][e] : (W)0.0f;
            }
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const Eight<W> fv = vp[((p * KS + ks) * kTile + t * 16 + col) * 4 + g];
#pragma unroll
                    for (int q = 0; q < NT; ++q) acc[t][q] = mfma(fb[q], fv, acc[t][q]);
                }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (t * 16 + col >= cnt) continue;
            if (whole) {
                tq o;
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[4 * q + i] = (T)((float)have[t][4 * q + i] + f[t] * acc[t][q][i]);
                *reinterpret_cast<tq *>(out[t] + c) = o;
            } else {
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + 4 * q + i < a.N)
                            out[t][c + 4 * q + i] = (T)((float)base[t][c + 4 * q + i] + f[t] * acc[t][q][i]);
            }
        }
    }
}

// The rows of v of a group in LDS, as the matrix instruction's columns: vp[part][ks][token][g], 8 ranks each.
template <typename W, int P, int KS>
__device__ __forceinline__ void stage_v(const LoraArgs &a, int64_t slab, int rank, int cnt, const uint8_t *list, int rows,
                                        int splits, Eight<W> *vp, float *undo, uint32_t *top) {
    constexpr int kParts = Held<W, P>::kParts;
    const int t = threadIdx.x, eights = KS * 4, tokens = (cnt + 15) / 16 * 16;
    const auto sum = [&](int i, int j, float (&v)[8]) {  // ranks j .. j + 7 of token i
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        if (i >= cnt || j >= rank) return;
        const float *p = (const float *)a.ws + (slab + list[i]) * a.R + j;
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const Eight<float> x = load8(p + (int64_t)s * rows * a.R);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += x[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = j + e < rank ? v[e] : 0.0f;
    };
    if constexpr (Held<W, P>::kScaled) {
        // the largest finite entry of each row goes to [2^14, 2^15): two fp16 parts then hold 22 bits of it, and
        // of smaller entries all that lies above 2^-38 of it
        if (t < kTile) top[t] = 0;
        __syncthreads();
        for (int u = t; u < tokens * eights; u += kThreads) {
            const int i = u / eights, j = u % eights * 8;
            float v[8];
            sum(i, j, v);
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = __builtin_isfinite(v[e]) ? fmaxf(m, fabsf(v[e])) : m;
            if (m > 0.0f) atomicMax(&top[i], __builtin_bit_cast(uint32_t, m));
            // fp32 in the place of the parts until the row's scale is known: 32 bytes for two parts of 16
            vp[(j / 32 * kTile + i) * 4 + j % 32 / 8] = __builtin_bit_cast(Eight<W>, f4{v[0], v[1], v[2], v[3]});
            vp[((KS + j / 32) * kTile + i) * 4 + j % 32 / 8] = __builtin_bit_cast(Eight<W>, f4{v[4], v[5], v[6], v[7]});
        }
        __syncthreads();
        for (int u = t; u < tokens * eights; u += kThreads) {
            const int i = u / eights, j = u % eights * 8;
            const int at0 = (j / 32 * kTile + i) * 4 + j % 32 / 8, at1 = ((KS + j / 32) * kTile + i) * 4 + j % 32 / 8;
            const f4 lo = __builtin_bit_cast(f4, vp[at0]), hi = __builtin_bit_cast(f4, vp[at1]);
            const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            const int shift = top[i] ? 14 - ((int)(top[i] >> 23) - 127) : 0;  // subnormal rows count as 2^-127
            Eight<W> p0, p1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = ldexpf(v[e], shift);
                p0[e] = (W)s;
                p1[e] = (W)(__builtin_isfinite(s) ? s - (float)p0[e] : 0.0f);
            }
            vp[at0] = p0;
            vp[at1] = p1;
            if (j == 0) undo[i] = ldexpf(1.0f, -shift);
        }
    } else {
        for (int u = t; u < tokens * eights; u += kThreads) {
            const int i = u / eights, j = u % eights * 8;
            float v[8];
            sum(i, j, v);
            bf8 part[kParts];
            split<kParts>(v, part);
#pragma unroll
            for (int p = 0; p < kParts; ++p) vp[((p * KS + j / 32) * kTile + i) * 4 + j % 32 / 8] = part[p];
        }
    }
    __syncthreads();
}

template <typename T>
__device__ __forceinline__ void copy_rows(const LoraArgs &a, int64_t row0, uint64_t mask, int64_t n0, int64_t n1) {
    for (; mask; mask &= mask - 1) {
        const int64_t row = row0 + __builtin_ctzll(mask);
        for (int64_t n = n0 + threadIdx.x; n < n1; n += kThreads)
            ((T *)a.out)[row * a.ldo + n] = ((const T *)a.base)[row * a.ldb + n];
    }
}

template <typename W, typename T, int P, int KS>
__global__ __launch_bounds__(kThreads) void lora_expand_kernel(const LoraArgs a, int64_t m0, int rows, int turns, int splits,
                                                               int chunk) {
    __shared__ Eight<W> vp[Held<W, P>::kParts * KS * kTile * 4];
    __shared__ float undo[kTile];
    __shared__ uint32_t top[kTile];
    __shared__ uint8_t list[kTile];
    const int turn = blockIdx.z;
    const int row = blockIdx.x * kTile + threadIdx.x % kWave;
    const int id = row < rows ? a.row_adapter[m0 + row] : -1;
    const bool valid = (uint32_t)id < (uint32_t)a.L;
    const int64_t slab = (int64_t)blockIdx.x * kTile, row0 = m0 + slab;
    const int64_t n0 = (int64_t)blockIdx.y * chunk, n1 = n0 + chunk < a.N ? n0 + chunk : a.N;
    const bool copies = a.base != a.out;
    for_each_adapter(id, valid, turn, turns, [&](int ad, uint64_t mask) {
        const int rank = rank_of(a, ad);
        if (rank == 0) {
            if (copies) copy_rows<T>(a, row0, mask, n0, n1);
            return;
        }
        gather_rows(mask, list);
        const int cnt = __popcll(mask);
        stage_v<W, P, KS>(a, slab, rank, cnt, list, rows, splits, vp, undo, top);
        if (cnt <= 16) expand_group<W, T, P, KS, 1>(a, row0, ad, rank, cnt, list, vp, undo, n0, n1);
        else if (cnt <= 32) expand_group<W, T, P, KS, 2>(a, row0, ad, rank, cnt, list, vp, undo, n0, n1);
        else expand_group<W, T, P, KS, 4>(a, row0, ad, rank, cnt, list, vp, undo, n0, n1);
    });
    if (copies && turn == 0) copy_rows<T>(a, row0, __ballot(row < rows && !valid), n0, n1);
}

// ------------------------------------------------------------------ launches
struct Plan {
    int turns, splits, per;  // workgroups that share a tile's adapters; ranges of k, and windows of each
};
Plan plan_of(int64_t rows, int64_t K, int32_t L, int32_t R) {
    const int64_t tiles = (rows + kTile - 1) / kTile, windows = (K + kWindow - 1) / kWindow;
    Plan p;
    p.turns = (int)std::max<int64_t>(1, std::min<int64_t>({kTile, rows, L, 1024 / tiles}));
    const int64_t blocks = tiles * p.turns * ((R + 63) / 64);
    const int64_t splits = std::min((512 + blocks - 1) / blocks, (windows + kWaves - 1) / kWaves);
    p.per = (int)((windows + splits - 1) / splits);
    p.splits = (int)((windows + p.per - 1) / p.per);
    return p;
}

template <typename X, typename W, int P>
void shrink(const LoraArgs &a, int64_t m0, int rows, const Plan &p, hipStream_t stream) {
    const int rt = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;
    const dim3 grid((rows + kTile - 1) / kTile, p.turns * p.splits, (a.R + rt * 16 - 1) / (rt * 16));
#define W4A8_SHRINK(RT) lora_shrink_kernel<X, W, P, RT><<<grid, kThreads, 0, stream>>>(a, m0, rows, p.turns, p.per)
    if (rt == 1) W4A8_SHRINK(1);
    else if (rt == 2) W4A8_SHRINK(2);
    else W4A8_SHRINK(4);
#undef W4A8_SHRINK
}

template <typename W, typename T, int P>
void expand(const LoraArgs &a, int64_t m0, int rows, const Plan &p, hipStream_t stream) {
    const int64_t tiles = (rows + kTile - 1) / kTile;
    const int step = kWaves * 16 * tiles_of<T>();
    const int64_t blocks = tiles * p.turns;
    int64_t chunk = step;
    while (chunk < 4 * step && blocks * ((a.N + chunk - 1) / chunk) > 2048) chunk *= 2;
    while (blocks * ((a.N + chunk - 1) / chunk) > 1 << 22) chunk *= 2;  // fewer than 2^32 threads
    const dim3 grid((uint32_t)tiles, (uint32_t)((a.N + chunk - 1) / chunk), p.turns);
#define W4A8_EXPAND(KS) \
    lora_expand_kernel<W, T, P, KS><<<grid, kThreads, 0, stream>>>(a, m0, rows, p.turns, p.splits, (int)chunk)
    if (a.R <= 32) W4A8_EXPAND(1);
    else if (a.R <= 64) W4A8_EXPAND(2);
    else if (a.R <= 128) W4A8_EXPAND(4);
    else W4A8_EXPAND(8);
#undef W4A8_EXPAND
}

template <typename W, int P>
hipError_t launch_w(const LoraArgs &a, hipStream_t stream) {
    for (int64_t m0 = 0; m0 < a.M; m0 += kSlab) {
        const int rows = (int)std::min(a.M - m0, kSlab);
        const Plan p = plan_of(rows, a.K, a.L, a.R);
        if (a.x_type == W4A8_F32) shrink<float, W, P>(a, m0, rows, p, stream);
        else if (a.x_type == W4A8_F16) shrink<_Float16, W, 2>(a, m0, rows, p, stream);
        else shrink<__bf16, W, 2>(a, m0, rows, p, stream);
        if (a.out_type == W4A8_F32) expand<W, float, 3>(a, m0, rows, p, stream);
        else if (a.out_type == W4A8_F16) expand<W, _Float16, 2>(a, m0, rows, p, stream);
        else expand<W, __bf16, 2>(a, m0, rows, p, stream);
        if (hipError_t err = hipGetLastError(); err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

namespace w4a8 {

int64_t lora_ws_bytes(int64_t M, int64_t K, int32_t L, int32_t R) {
    if (M == 0) return 0;
    // the first slab is the largest, a last and shorter one may have more ranges of k
    const int64_t first = std::min(M, kSlab), last = M % kSlab;
    int64_t need = plan_of(first, K, L, R).splits * first;
    if (last) need = std::max(need, plan_of(last, K, L, R).splits * last);
    return need * R * 4;
}

hipError_t launch_lora_add(const LoraArgs &a, hipStream_t stream) {
    // an fp32 output is held by three parts of fp32 operands, a 16-bit one by two
    const bool wide = a.out_type == W4A8_F32;
    if (a.ab_type == W4A8_F16) return wide ? launch_w<_Float16, 3>(a, stream) : launch_w<_Float16, 2>(a, stream);
    return wide ? launch_w<__bf16, 3>(a, stream) : launch_w<__bf16, 2>(a, stream);
}

}  // namespace w4a8
