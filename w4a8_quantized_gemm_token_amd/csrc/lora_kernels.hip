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
// A tile's groups: its distinct valid adapters in the order of their first rows.  Each call takes the next one off
// `left` (the valid lanes that no group has taken yet) and gives the mask of its lanes.
__device__ __forceinline__ uint64_t next_group(int id, uint64_t &left, int &adapter) {
    adapter = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t mask = __ballot(id == adapter) & left;
    left &= ~mask;
    return mask;
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

// The workspace: each tile's number of groups, and behind them the parts of v [splits][rows][R].
constexpr int kCounts = kSlab / kTile;

template <typename X, typename W, int P, int RT>
__global__ __launch_bounds__(kThreads) void lora_shrink_kernel(const LoraArgs a, int64_t m0, int rows, int turns, int per) {
    __shared__ f4 red[kWaves][RT][kWave];
    __shared__ uint8_t list[kTile];
    const int split = blockIdx.y / turns, turn = blockIdx.y % turns, j0 = blockIdx.z * RT * 16;
    const int row = blockIdx.x * kTile + threadIdx.x % kWave;
    const int id = row < rows ? a.row_adapter[m0 + row] : -1;
    const int windows = (int)((a.K + kWindow - 1) / kWindow);
    const int w0 = split * per, w1 = min(w0 + per, windows);
    float *part = (float *)a.ws + kCounts + (int64_t)split * rows * a.R;
    const int64_t slab = (int64_t)blockIdx.x * kTile, row0 = m0 + slab;
    uint64_t left = __ballot((uint32_t)id < (uint32_t)a.L);
    const bool bare = __ballot(row < rows) != left;
    int groups = 0;
    for (; left; ++groups) {
        int ad;
        const uint64_t mask = next_group(id, left, ad);
        if (groups % turns != turn) continue;
        const int rank = rank_of(a, ad);
        if (j0 >= rank) continue;
        gather_rows(mask, list);
        const int cnt = __popcll(mask);
        if (cnt <= 16) shrink_group<X, W, P, 1, RT>(a, row0, slab, ad, rank, j0, cnt, list, w0, w1, part, red);
        else if (cnt <= 32) shrink_group<X, W, P, 2, RT>(a, row0, slab, ad, rank, j0, cnt, list, w0, w1, part, red);
        else shrink_group<X, W, P, 4, RT>(a, row0, slab, ad, rank, j0, cnt, list, w0, w1, part, red);
    }
    // rows without an adapter are a last group where they are copied
    if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0)
        ((int *)a.ws)[blockIdx.x] = groups + (bare && a.base != a.out ? 1 : 0);
}

// ------------------------------------------------------------------ expand
// v beside weights of type W: bf16 parts as above (P of them), or two fp16 parts of the scaled row.
template <typename W, int P>
struct Held {
    static constexpr bool kScaled = std::is_same<W, _Float16>::value;
    static constexpr int kParts = kScaled ? 2 : P;
};

constexpr int kExpandBlocks = 3;  // workgroups a CU
constexpr int kUnit = 128;  // columns that a workgroup's share of a group is counted in

// Columns of a wave's step of NT matrix tiles, dealt so that a lane has 16 bytes of output columns in a row: piece p of the
// step is the columns VW (4 p + g) .. + VW - 1 of lane group g, with VW = 4 of fp32 (a tile) or 8 of 16 bits (two tiles).
template <typename T, int NT>
struct Columns {
    static constexpr int VW = 16 / sizeof(T), kPieces = NT * 4 / VW, kStep = 16 * NT;
    static_assert(kUnit % kStep == 0 && NT % 2 == 0, "a step lies in one unit");
    typedef T V __attribute__((ext_vector_type(16 / sizeof(T))));
    typedef T VU __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
    // column of tile q, matrix row r, within a step
    static __device__ __forceinline__ int of(int q, int r) {
        return sizeof(T) == 4 ? 16 * q + r : 32 * (q / 2) + 8 * (r / 4) + 4 * (q % 2) + r % 4;
    }
};

// Columns [n0, n1) of a group's rows; n0 is a multiple of kUnit, n1 too or N.
template <typename W, typename T, int P, int KS, int TT>
__device__ __forceinline__ void expand_group(const LoraArgs &a, int64_t row0, int id, int rank, int cnt, const uint8_t *list,
                                             const Eight<W> *vp, const float *undo, int64_t n0, int64_t n1) {
    // the fewer rows and ranks, the more columns a step, for loads under way
    constexpr int NT = TT * KS <= 1 ? 8 : TT * KS <= 2 ? 4 : 2, kParts = Held<W, P>::kParts;
    using C = Columns<T, NT>;
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
        base[t] = (const T *)a.base + row * a.ldb + C::VW * g;
        out[t] = (T *)a.out + row * a.ldo + C::VW * g;
        f[t] = Held<W, P>::kScaled ? scale * undo[i < cnt ? i : 0] : scale;
    }
    for (int64_t n = n0 + wave * C::kStep; n < n1; n += kWaves * C::kStep) {
        const bool whole = n + C::kStep <= a.N;
        typename C::V have[TT][C::kPieces];
        if (whole) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
                if (t * 16 + col < cnt) {
#pragma unroll
                    for (int p = 0; p < C::kPieces; ++p)
                        have[t][p] = *reinterpret_cast<const typename C::VU *>(base[t] + n + 4 * C::VW * p);
                }
        }
        Eight<W> fb[KS][NT];
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            const int64_t nn = n + C::of(q, col);
            const W *p = pb + (nn < a.N ? nn : a.N - 1) * a.R;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) fb[ks][q] = ks * 32 + 8 * g < rank ? load8(p + ks * 32) : zero8<W>();
        }
        if (rank & 7) {  // ranks past the adapter's own, whatever they hold
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int q = 0; q < NT; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e) fb[ks][q][e] = ks * 32 + 8 * g + e < rank ? fb[ks][q][e] : (W)0.0f;
        }
        f4 acc[TT][NT] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks * 32 >= rank) break;
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const Eight<W> fv = vp[((p * KS + ks) * kTile + t * 16 + col) * 4 + g];
#pragma unroll
                    for (int q = 0; q < NT; ++q) acc[t][q] = mfma(fb[ks][q], fv, acc[t][q]);
                }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            if (t * 16 + col >= cnt) continue;
            if (whole) {
#pragma unroll
                for (int p = 0; p < C::kPieces; ++p) {
                    typename C::V o;
#pragma unroll
                    for (int i = 0; i < C::VW; ++i)
                        o[i] = (T)((float)have[t][p][i] + f[t] * acc[t][(p * C::VW + i) / 4][i % 4]);
                    *reinterpret_cast<typename C::VU *>(out[t] + n + 4 * C::VW * p) = o;
                }
            } else {
#pragma unroll
                for (int p = 0; p < C::kPieces; ++p)
#pragma unroll
                    for (int i = 0; i < C::VW; ++i) {
                        const int64_t c = n + 4 * C::VW * p + i;
                        if (c + C::VW * g < a.N) out[t][c] = (T)((float)base[t][c] + f[t] * acc[t][(p * C::VW + i) / 4][i % 4]);
                    }
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
        const float *p = (const float *)a.ws + kCounts + (slab + list[i]) * a.R + j;
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

// Columns [n0, n1) of cnt rows in list, from base to out, 16 bytes a thread.
template <typename T>
__device__ __forceinline__ void copy_rows(const LoraArgs &a, int64_t row0, int cnt, const uint8_t *list, int64_t n0, int64_t n1) {
    constexpr int VW = 16 / sizeof(T);
    typedef T VU __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
    const int pieces = (int)((n1 - n0 + VW - 1) / VW);
#pragma unroll 4
    for (int u = threadIdx.x; u < cnt * pieces; u += kThreads) {
        const int64_t row = row0 + list[u / pieces], n = n0 + (int64_t)(u % pieces) * VW;
        const T *p = (const T *)a.base + row * a.ldb + n;
        T *o = (T *)a.out + row * a.ldo + n;
        if (n + VW <= n1) {
            *reinterpret_cast<VU *>(o) = *reinterpret_cast<const VU *>(p);
        } else {
            for (int i = 0; n + i < n1; ++i) o[i] = p[i];
        }
    }
}

// A fixed grid walks the units in equal runs: unit (group, kUnit columns), columns fastest, so that a workgroup stages
// a group's v once for all its columns, and tiles of few and of many groups cost what their work costs.
template <typename W, typename T, int P, int KS>
__global__ __launch_bounds__(kThreads, KS > 4 ? 1 : kExpandBlocks) void lora_expand_kernel(const LoraArgs a, int64_t m0, int rows, int splits) {
    __shared__ Eight<W> vp[Held<W, P>::kParts * KS * kTile * 4];
    __shared__ float undo[kTile];
    __shared__ uint32_t top[kTile];
    __shared__ uint8_t list[kTile];
    const int lane = threadIdx.x % kWave, tiles = (rows + kTile - 1) / kTile;
    // groups before each lane's tiles; a lane has kCounts / 64 tiles at most
    const int mine = (tiles + kWave - 1) / kWave;
    const int *counts = (const int *)a.ws;
    int upto = 0;
    for (int i = 0; i < mine; ++i)
        if (lane * mine + i < tiles) upto += counts[lane * mine + i];
    for (int o = 1; o < kWave; o <<= 1) {
        const int v = __shfl_up(upto, o, kWave);
        if (lane >= o) upto += v;
    }
    const int64_t per = (a.N + kUnit - 1) / kUnit, total = per * __builtin_amdgcn_readlane(upto, kWave - 1);
    const int64_t u1 = total * (blockIdx.x + 1) / gridDim.x;
    for (int64_t u = total * blockIdx.x / gridDim.x; u < u1;) {
        const int group = (int)(u / per);
        const int64_t first = u - group * per, last = first + (u1 - u) < per ? first + (u1 - u) : per;
        u += last - first;
        const int64_t n0 = first * kUnit, n1 = last * kUnit < a.N ? last * kUnit : a.N;
        // the group's tile, and its number there
        const int l = __builtin_ctzll(__ballot(upto > group));
        int k = group - (l ? __builtin_amdgcn_readlane(upto, l - 1) : 0), tile = l * mine;
        while (k >= counts[tile]) k -= counts[tile++];
        const int row = tile * kTile + lane;
        const int id = row < rows ? a.row_adapter[m0 + row] : -1;
        const int64_t slab = (int64_t)tile * kTile, row0 = m0 + slab;
        uint64_t left = __ballot((uint32_t)id < (uint32_t)a.L), mask = __ballot(row < rows) & ~left;
        int ad = -1, rank = 0;
        if (left) {
            const uint64_t bare = mask;
            for (; k >= 0 && left; --k) mask = next_group(id, left, ad);
            if (k < 0) rank = rank_of(a, ad);
            else mask = bare;
        }
        if (rank == 0 && a.base == a.out) continue;
        gather_rows(mask, list);
        const int cnt = __popcll(mask);
        if (rank == 0) {
            copy_rows<T>(a, row0, cnt, list, n0, n1);
            continue;
        }
        stage_v<W, P, KS>(a, slab, rank, cnt, list, rows, splits, vp, undo, top);
        if (cnt <= 16) expand_group<W, T, P, KS, 1>(a, row0, ad, rank, cnt, list, vp, undo, n0, n1);
        else if (cnt <= 32) expand_group<W, T, P, KS, 2>(a, row0, ad, rank, cnt, list, vp, undo, n0, n1);
        else expand_group<W, T, P, KS, 4>(a, row0, ad, rank, cnt, list, vp, undo, n0, n1);
    }
}

// ------------------------------------------------------------------ launches
struct Plan {
    int turns, splits, per;  // workgroups that share a tile's adapters; ranges of k, and windows of each
};
Plan plan_of(int64_t rows, int64_t K, int32_t L, int32_t R) {
    const int64_t tiles = (rows + kTile - 1) / kTile, windows = (K + kWindow - 1) / kWindow;
    Plan p;
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(1024 / tiles, (windows + kWaves - 1) / kWaves));
    p.per = (int)((windows + splits - 1) / splits);
    p.splits = (int)((windows + p.per - 1) / p.per);
    p.turns = (int)std::max<int64_t>(1, std::min<int64_t>({kTile, rows, L, 2048 / (tiles * p.splits)}));
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
    // no more workgroups than there can be units, or than are resident
    const int64_t most = tiles * std::min<int64_t>({kTile, rows, (int64_t)a.L + 1}) * ((a.N + kUnit - 1) / kUnit);
    const uint32_t grid = (uint32_t)std::min<int64_t>(most, 256 * kExpandBlocks);
#define W4A8_EXPAND(KS) lora_expand_kernel<W, T, P, KS><<<grid, kThreads, 0, stream>>>(a, m0, rows, p.splits)
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
    return (need * R + kCounts) * 4;
}

hipError_t launch_lora_add(const LoraArgs &a, hipStream_t stream) {
    // an fp32 output is held by three parts of fp32 operands, a 16-bit one by two
    const bool wide = a.out_type == W4A8_F32;
    if (a.ab_type == W4A8_F16) return wide ? launch_w<_Float16, 3>(a, stream) : launch_w<_Float16, 2>(a, stream);
    return wide ? launch_w<__bf16, 3>(a, stream) : launch_w<__bf16, 2>(a, stream);
}

}  // namespace w4a8
