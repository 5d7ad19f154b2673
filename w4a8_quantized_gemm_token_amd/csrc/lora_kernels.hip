// lora_kernels.hip -- low-rank adapters of many requests beside a shared projection.
//
// For row m with adapter a: v = A_a x[m] (rank values), out[m] = base[m] + scale_a B_a v.
// Two launches: the shrink product leaves parts of v per range of k in the workspace, the expand product adds them up
// and walks the output.  Both go by tiles of 64 rows as they stand: a wave's lanes hold the 64 adapter ids, the distinct
// ones are found with ballots, and each one's rows (a group) are gathered into 16-row columns of the matrix
// instruction, so rows of one adapter share its loads without being sorted beforehand, and no row can be met
// twice.  The groups stand in a table in the workspace, which a workgroup of the shrink product writes, or a launch of
// its own in front of it above 64 tiles.  Longer calls go by slabs of 32768 rows.
//
// Arithmetic: the matrix cores take 16-bit operands.  fp32 values enter as sums of three bf16 parts, each the rest of the
// ones before it rounded to its 8 bits, which hold all 24 bits whatever the output's type (rows may cancel, and then bits
// that the output's rounding seems to hide are all that is left); an fp16 value beside bf16 is two such parts, exactly.  v
// meets fp16 weights as two fp16 parts after a scaling of its row by a power of two: within 2^-23 of each entry, or 2^-39 of
// the row's largest, below what its own fp32 sum leaves open.  All sums are fp32.
//
// What has to move: x, base and out once, and the A and B of the adapters in use.  Times and bounds stand at the kernels
// for these calls (rows; adapters in use; rank; k; columns): one token (1; 1; 16; 7168; 4096), decode batch (64; 48; 16;
// 8192; 28672), prompts (500; 5; 64; 4096; 14340), prefill (4096; 4; 16; 8192; 8192), long prefill (20011; 3; to 128; 4096;
// 14336).
#include "block_internal.hpp"

#include <algorithm>
#include <type_traits>

using namespace w4a8;
using namespace w4a8dev;

namespace {

constexpr int kShrinkThreads = 512, kShrinkWaves = kShrinkThreads / kWave;
constexpr int kThreads = 256, kWaves = kThreads / kWave;  // of the expand product
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
// The same at a byte offset of the lane from an address that is the wave's: 32 bits a lane instead of 64.
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T *p, uint32_t bytes) {
    return load8((const T *)((const char *)p + bytes));
}
template <typename V, typename T>
__device__ __forceinline__ V &at(T *p, uint32_t bytes) {
    return *(V *)((char *)p + bytes);
}
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }
template <typename T>
__device__ __forceinline__ Eight<T> zero8() {
    Eight<T> z = {};
    return z;
}

__device__ __forceinline__ f4 mfma(bf8 a, bf8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// A barrier for what passes through LDS.  (__syncthreads would also wait for the stores to memory that are under way.)
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// a / b and what is left, for a < 2^22 and b > 0: the fp32 quotient is off by one at most.  (The compiler's own division
// takes some forty instructions, and these stand before everything else that a workgroup does.)
__device__ __forceinline__ int quotient(int a, int b, int &rest) {
    int q = (int)((float)a * __builtin_amdgcn_rcpf((float)b));
    rest = a - q * b;
    if (rest < 0) --q, rest += b;
    if (rest >= b) ++q, rest -= b;
    return q;
}

// ------------------------------------------------------------------ operands in parts
// part[i] = what the parts before it leave of v, rounded to nearest: N parts hold 8 N bits and more.  All but the last stay
// inside bf16's finite range: above it the rounding would give an infinity (and the rest another one of the other sign), and
// an infinity or NaN has to reach one part only, the last, from where it meets the other operand's first part.
template <int N>
__device__ __forceinline__ void split(const float (&v)[8], bf8 (&part)[N]) {
    constexpr float kTop = 0x1.FEp+127f;  // bf16's largest
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (i + 1 == N) {
                part[i][e] = (__bf16)r[e];
            } else {
                part[i][e] = (__bf16)__builtin_amdgcn_fmed3f(r[e], -kTop, kTop);
                r[e] -= (float)part[i][e];
            }
        }
    }
}

// The operand of type T beside one of type U: itself where both are the same 16-bit type, parts otherwise (three for fp32).
template <typename T, typename U>
struct Operand {
    static constexpr int kParts = std::is_same<T, float>::value ? 3 : std::is_same<T, _Float16>::value ? 2 : 1;
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
template <>
struct Operand<_Float16, _Float16> {
    static constexpr int kParts = 1;
    typedef h8 V;
    static __device__ __forceinline__ void of(const Eight<_Float16> &x, V (&part)[1]) { part[0] = x; }
};

// ------------------------------------------------------------------ groups of a tile
// A tile's groups: its distinct valid adapters in the order of their first rows.  A wave finds the first eight one after
// another (46 ns each), and if there are more, all at once by comparing every pair of ids.
constexpr int kInTurn = 8;

// The lanes that hold this lane's id; every lane calls it.  ids: 64 words of LDS, the wave's own.
__device__ __forceinline__ uint64_t lanes_alike(int id, int *ids) {
    const int lane = threadIdx.x % kWave;
    ids[lane] = id;
    __builtin_amdgcn_wave_barrier();
    uint32_t half[2] = {0, 0};
#pragma unroll
    for (int i = kWave - 4; i >= 0; i -= 4) {
        const v4i o = *reinterpret_cast<const v4i *>(ids + i);
#pragma unroll
        for (int e = 3; e >= 0; --e) half[i / 32] = half[i / 32] + half[i / 32] + (o[e] == id ? 1 : 0);
    }
    __builtin_amdgcn_wave_barrier();
    return (uint64_t)half[1] << 32 | half[0];
}

// A tile's valid lanes, and the first lanes of its groups; by whole waves.
struct Tile {
    int id;
    uint64_t valid, leaders;

    __device__ __forceinline__ Tile(int id, int32_t L, int *ids) : id(id), valid(__ballot((uint32_t)id < (uint32_t)L)) {
        uint64_t left = valid;
        leaders = 0;
        for (int n = 0; left && n < kInTurn; ++n) {
            const int first = __builtin_ctzll(left);
            leaders |= 1ull << first;
            left &= ~__ballot(id == __builtin_amdgcn_readlane(id, first));
        }
        if (left) {
            const int lane = threadIdx.x % kWave;
            const uint64_t same = lanes_alike(id, ids);
            leaders = __ballot((valid >> lane & 1) && __builtin_ctzll(same) == lane);
        }
    }
    __device__ __forceinline__ Tile(int id, int32_t L, uint64_t leaders)
        : id(id), valid(__ballot((uint32_t)id < (uint32_t)L)), leaders(leaders) {}
    __device__ __forceinline__ int groups() const { return __popcll(leaders); }
};

__device__ __forceinline__ int rank_of(const LoraArgs &a, int id) {
    const int r = a.ranks ? a.ranks[id] : a.R;
    return r < 0 ? 0 : r > a.R ? a.R : r;
}

// The lanes of mask in a row in list[]; all threads of the workgroup, between barriers.
__device__ __forceinline__ void gather_rows(uint64_t mask, uint8_t *list) {
    lds_barrier();
    if (threadIdx.x < kTile && (mask >> threadIdx.x & 1))
        list[__popcll(mask & ((1ull << threadIdx.x) - 1))] = (uint8_t)threadIdx.x;
    lds_barrier();
}

// The table of all groups, in the order of tiles and first rows, and behind them one entry for each tile that has rows
// without an adapter, where those are copied.  The workspace: the head, the table, the parts of v [splits][rows][R].
struct Group {
    uint64_t mask;  // rows of the tile
    int32_t adapter, rank, tile;
    float scale;
    int32_t pad[2];
};
struct Head {
    int32_t groups, copies, splits, per;  // per: windows of a range of k
    int32_t pad[12];
};
constexpr int kSelf = 64;  // up to this many tiles the shrink product finds the groups for itself

__host__ __device__ constexpr int tiles_in(int rows) { return (rows + kTile - 1) / kTile; }
__host__ __device__ constexpr int64_t parts_at(int rows) {
    return sizeof(Head) + (int64_t)tiles_in(rows) * ((rows < kTile ? rows : kTile) + 1) * sizeof(Group);
}
__device__ __forceinline__ Head *head_of(const LoraArgs &a) { return (Head *)a.ws; }
__device__ __forceinline__ Group *table_of(const LoraArgs &a) { return (Group *)((Head *)a.ws + 1); }
__device__ __forceinline__ float *parts_of(const LoraArgs &a, int rows) { return (float *)((char *)a.ws + parts_at(rows)); }

// Entry k, the same in every lane.  What it holds is cut to the call's sizes: whatever the memory holds, no row, adapter or
// rank outside them is met.
__device__ __forceinline__ Group group_of(const LoraArgs &a, int rows, int k) {
    Group g = table_of(a)[k];
    g.tile = min((uint32_t)__builtin_amdgcn_readfirstlane(g.tile), (uint32_t)tiles_in(rows) - 1);
    g.adapter = __builtin_amdgcn_readfirstlane(g.adapter);
    g.rank = (uint32_t)g.adapter < (uint32_t)a.L ? min((uint32_t)__builtin_amdgcn_readfirstlane(g.rank), (uint32_t)a.R) : 0;
    const int in = rows - g.tile * kTile;
    const uint64_t mask = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(g.mask >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)g.mask);
    g.mask = in < kTile ? mask & ((1ull << in) - 1) : mask;
    return g;
}

// Entries of N tiles, their groups from number at[] on and their rows without an adapter at bare[]; by whole waves.  All
// masks first, then all ranks and scales, then the stores, so that a tile does not wait for the last one's loads.
template <int N>
__device__ __forceinline__ void write_groups(const LoraArgs &a, const Tile (&t)[N], int rows, const int (&tile)[N],
                                             const int (&at)[N], const int (&bare)[N]) {
    const int lane = threadIdx.x % kWave;
    uint64_t mask[N], in[N];
    int rank[N];
    float scale[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        mask[i] = 0;
        in[i] = __ballot(tile[i] * kTile + lane < rows);
        for (uint64_t left = t[i].leaders; left; left &= left - 1) {
            const int first = __builtin_ctzll(left);
            const uint64_t m = __ballot(t[i].id == __builtin_amdgcn_readlane(t[i].id, first)) & t[i].valid;
            mask[i] = lane == first ? m : mask[i];
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int id = t[i].leaders >> lane & 1 ? t[i].id : 0;
        rank[i] = rank_of(a, id);
        scale[i] = a.scale ? a.scale[id] : 1.0f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (t[i].leaders >> lane & 1)
            table_of(a)[at[i] + __popcll(t[i].leaders & ((1ull << lane) - 1))] =
                Group{mask[i], t[i].id, rank[i], tile[i], scale[i], {0, 0}};
        if (a.base != a.out && in[i] != t[i].valid && lane == 0)
            table_of(a)[bare[i]] = Group{in[i] & ~t[i].valid, -1, 0, tile[i], 0.0f, {0, 0}};
    }
}

// Ranges of k, and windows of each.  At least as many as make kFill units (group, block of ranks, range): 978 rows of one
// adapter of rank 120 with k 5160 and 4096 columns take 37 us, 46 without, and 1656 such rows 46 and 53; with 256 units 37
// and 57.  Beyond that up to kTarget units, or four ranges where there are as many units already (so that the last round
// of workgroups is a short one), if the expand product has not to read more than kStaged bytes of parts of v for a group on
// average: with twice that the long prefill takes 564 us instead of 520, with half of it 517, the prompts the same.
// Never more than the workspace has room for.
constexpr int kTarget = 512, kFill = 128, kStaged = 65536;
constexpr int blocks_of(int R) { return R <= 64 ? 1 : (R + 63) / 64; }  // of ranks in the shrink product
__device__ __forceinline__ void set_ranges(Head &h, int rows, int64_t K, int R, int most) {
    const int windows = (int)((K + kWindow - 1) / kWindow);
    const float units = (float)max(1, h.groups * blocks_of(R));
    const float each = __builtin_amdgcn_rcpf(units);
    const int worth = (int)(kStaged / 4 * (float)h.groups * __builtin_amdgcn_rcpf((float)(rows * R)));
    const int more = min(max(4, (int)(kTarget * each)), worth);
    const int wanted = max(1, min(max((int)(kFill * each + 0.99f), more), most));
    int rest;
    h.per = quotient(windows + wanted - 1, wanted, rest);
    h.splits = quotient(windows + h.per - 1, h.per, rest);
}

// Sums of v over the lanes up to each.
__device__ __forceinline__ int sum_upto(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
}

// More tiles: the table by one workgroup, wave w the tiles w, w + 16, ..., all ids and first rows in LDS, from where the
// entries are written once their places are known.  313 tiles take 20 us, in a call of 520 (24 us with 4 KB of LDS and the
// ids read and compared twice); a wave's 20 tiles stand one after another.
constexpr int kTableThreads = 1024, kTableWaves = kTableThreads / kWave, kMaxTiles = kSlab / kTile;
__global__ __launch_bounds__(kTableThreads) void lora_table_kernel(const LoraArgs a, int64_t m0, int rows, int most) {
    __shared__ __attribute__((aligned(16))) int ids[kMaxTiles][kWave];
    __shared__ uint64_t leaders[kMaxTiles];
    __shared__ int counts[kMaxTiles], bare[kMaxTiles];
    const int lane = threadIdx.x % kWave, wave = wave_id(), tiles = tiles_in(rows);
    constexpr int kTogether = 8;  // tiles whose ids are under way together
    for (int t0 = wave; t0 < tiles; t0 += kTogether * kTableWaves) {
        int id[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            const int row = (t0 + i * kTableWaves) * kTile + lane;
            id[i] = row < rows ? a.row_adapter[m0 + row] : -1;
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            const int tile = t0 + i * kTableWaves;
            if (tile >= tiles) break;
            const Tile t(id[i], a.L, ids[tile]);
            const uint64_t in = __ballot(tile * kTile + lane < rows);
            ids[tile][lane] = id[i];
            if (lane == 0) {
                counts[tile] = t.groups();
                bare[tile] = a.base != a.out && in != t.valid ? 1 : 0;
                leaders[tile] = t.leaders;
            }
        }
    }
    lds_barrier();
    if (wave == 0) {
        // counts become the numbers of first groups
        constexpr int kMine = kMaxTiles / kWave;
        int c = 0, b = 0;
        for (int i = 0; i < kMine; ++i)
            if (lane * kMine + i < tiles) c += counts[lane * kMine + i], b += bare[lane * kMine + i];
        const int cs = sum_upto(c), bs = sum_upto(b), groups = __builtin_amdgcn_readlane(cs, kWave - 1);
        int at = cs - c, bat = groups + bs - b;
        for (int i = 0; i < kMine; ++i)
            if (lane * kMine + i < tiles) {
                const int n = counts[lane * kMine + i], f = bare[lane * kMine + i];
                counts[lane * kMine + i] = at;
                bare[lane * kMine + i] = bat;
                at += n;
                bat += f;
            }
        if (lane == kWave - 1) {
            Head h{groups, bs, 0, 0, {}};
            set_ranges(h, rows, a.K, a.R, most);
            *head_of(a) = h;
        }
    }
    lds_barrier();
    for (int t0 = wave; t0 < tiles; t0 += 4 * kTableWaves) {
        int tile[4], at[4], rest[4];
        const auto entry = [&](int i) {
            tile[i] = t0 + i * kTableWaves;
            const bool in = tile[i] < tiles;
            at[i] = in ? counts[tile[i]] : 0;
            rest[i] = in ? bare[tile[i]] : 0;
            return Tile(in ? ids[tile[i]][lane] : -1, a.L, in ? leaders[tile[i]] : 0);
        };
        const Tile t[4] = {entry(0), entry(1), entry(2), entry(3)};
        write_groups<4>(a, t, rows, tile, at, rest);
    }
}

// ------------------------------------------------------------------ shrink
// Matrix tiles of a round of adding the waves' sums up.
template <int RT>
constexpr int kRound = RT == 1 ? 4 : 8;

// v[token][j] over windows [w0, w1) of k for cnt rows in list and 16 RT ranks from j0; waves take windows in turn.
// Matrix rows are ranks, matrix columns tokens.
template <typename X, typename W, int TT, int RT>
__device__ __forceinline__ void shrink_group(const LoraArgs &a, int64_t row0, int64_t slab, int id, int rank, int j0, int cnt,
                                             const uint8_t *list, int w0, int w1, float *part, f4 (*red)[kRound<RT>][kWave]) {
    using OX = Operand<X, W>;
    using OW = Operand<W, X>;
    const int wave = wave_id(), lane = threadIdx.x % kWave, col = lane % 16, g = lane / 16;
    const X *px = (const X *)a.x + row0 * a.ldx;
    const W *pw = (const W *)a.A + (int64_t)id * a.R * a.K;
    uint32_t ox[TT], ow[RT];  // bytes: 64 rows of strides below 2^24, 256 ranks of K up to 2^20
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int i = t * 16 + col;
        ox[t] = (list[i < cnt ? i : 0] * (uint32_t)a.ldx + 16 * g) * (uint32_t)sizeof(X);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int j = j0 + r * 16 + col;
        ow[r] = ((uint32_t)(j < rank ? j : rank - 1) * (uint32_t)a.K + 16 * g) * (uint32_t)sizeof(W);
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
                            // (the third part of x beside the second of an fp16 weight: 2^-27 of the product)
                            if (p + q < 3) acc[t][r] = mfma(fw[r][q], fx[p], acc[t][r]);
            }
        }
    };
    const int whole = (int)(a.K / kWindow);
    for (int w = w0 + wave; w < w1; w += kShrinkWaves) {
        Eight<W> rw[RT][2];
        Eight<X> rx[TT][2];
        const int64_t k = (int64_t)w * kWindow;
        if (w < whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int r = 0; r < RT; ++r) rw[r][h] = load8(pw + k + 8 * h, ow[r]);
#pragma unroll
                for (int t = 0; t < TT; ++t) rx[t][h] = load8(px + k + 8 * h, ox[t]);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = k + 16 * g + 8 * h < a.K;
#pragma unroll
                for (int r = 0; r < RT; ++r) rw[r][h] = in ? load8(pw + k + 8 * h, ow[r]) : zero8<W>();
#pragma unroll
                for (int t = 0; t < TT; ++t) rx[t][h] = in ? load8(px + k + 8 * h, ox[t]) : zero8<X>();
            }
        }
        step(rw, rx);
    }
    // the waves' sums together, a round of matrix tiles at a time and one wave for each, and to the workspace: lane has
    // ranks 4 g .. 4 g + 3 of the tile, token col
    constexpr int kTiles = TT * RT, kStep = kRound<RT> < kTiles ? kRound<RT> : kTiles;
#pragma unroll
    for (int m = 0; m < kTiles; m += kStep) {
        if (m) lds_barrier();
#pragma unroll
        for (int i = 0; i < kStep; ++i) red[wave][i][lane] = acc[(m + i) / RT][(m + i) % RT];
        lds_barrier();
        if (wave < kStep) {
            const int i = (m + wave) / RT * 16 + col, j = j0 + (m + wave) % RT * 16 + 4 * g;
            f4 v[kShrinkWaves];
#pragma unroll
            for (int w = 0; w < kShrinkWaves; ++w) v[w] = red[w][wave][lane];
#pragma unroll
            for (int w = 1; w < kShrinkWaves; ++w) v[0] += v[w];
            if (i < cnt && j < a.R) *reinterpret_cast<f4 *>(part + (slab + list[i]) * a.R + j) = v[0];
        }
    }
}

// A fixed grid walks units (group, block of ranks, range of k): 16 to 64 ranks (RT matrix tiles) against 16, 32 or 64
// of the group's rows, eight waves sharing out the range.  One token 5.0 us and decode batch 7.0 us: finding the groups,
// one or two windows' loads and adding the waves' sums up, one after another.  Prefill 23.6 us, 2.8 TB/s.  Prompts 12 us.
// Long prefill 178 us: 1.8 TB/s of x, where a window's loads, the making of parts of its fp32 values and of its fp16
// weights (again for each 64 rows) and the products of parts stand one after another in a wave, the other waves of a CU
// cover only part of that, and the last round of units leaves CUs idle.  Units of 32 rows with twice the waves a CU spilled and were slower; grids of
// 256 to 2048 take the same time.  SELF: every workgroup finds the groups for itself, and the last one writes the table
// for the expand product.
template <typename X, typename W, int RT, bool SELF>
__global__ __launch_bounds__(kShrinkThreads) void lora_shrink_kernel(const LoraArgs a, int64_t m0, int rows, int most) {
    __shared__ f4 red[kShrinkWaves][kRound<RT>][kWave];
    __shared__ __attribute__((aligned(16))) int ids[SELF ? kSelf : 1][kWave];  // of all tiles
    __shared__ uint64_t masks[kSelf];
    __shared__ int counts[2][kSelf];
    __shared__ uint8_t list[kTile];
    const int lane = threadIdx.x % kWave, wave = wave_id(), tiles = tiles_in(rows);
    const int windows = (int)((a.K + kWindow - 1) / kWindow), blocks = blocks_of(a.R);
    Head h;
    int upto = 0;  // groups up to and with tile `lane`
    if (SELF) {
        constexpr int kMine = kSelf / kShrinkWaves;  // a wave's tiles, all their ids under way together
        int id[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int row = (i * kShrinkWaves + wave) * kTile + lane;
            id[i] = row < rows ? a.row_adapter[m0 + row] : -1;
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int tile = i * kShrinkWaves + wave;
            if (tile >= tiles) break;
            const Tile t(id[i], a.L, ids[tile]);
            const uint64_t in = __ballot(tile * kTile + lane < rows);
            ids[tile][lane] = id[i];
            if (lane == 0) {
                counts[0][tile] = t.groups();
                counts[1][tile] = a.base != a.out && in != t.valid ? 1 : 0;
                masks[tile] = t.leaders;
            }
        }
        lds_barrier();
        const int c = lane < tiles ? counts[0][lane] : 0, b = lane < tiles ? counts[1][lane] : 0;
        const int bs = sum_upto(b);
        upto = sum_upto(c);
        h.groups = __builtin_amdgcn_readlane(upto, kWave - 1);
        h.copies = __builtin_amdgcn_readlane(bs, kWave - 1);
        set_ranges(h, rows, a.K, a.R, most);
        if (blockIdx.x == gridDim.x - 1) {
            if (threadIdx.x == 0) *head_of(a) = Head{h.groups, h.copies, h.splits, h.per, {}};
            for (int tile = wave; tile < tiles; tile += kShrinkWaves) {
                const Tile t[1] = {Tile(ids[tile][lane], a.L, masks[tile])};
                write_groups<1>(a, t, rows, {tile}, {__builtin_amdgcn_readlane(upto - c, tile)},
                                {h.groups + __builtin_amdgcn_readlane(bs - b, tile)});
            }
        }
    } else {
        h.groups = min((uint32_t)head_of(a)->groups, (uint32_t)tiles * kTile);
        h.splits = min((uint32_t)head_of(a)->splits, (uint32_t)most);
        h.per = head_of(a)->per;
    }
    for (int u = blockIdx.x; u < h.groups * blocks * h.splits; u += gridDim.x) {
        int split, block;
        int k = quotient(quotient(u, h.splits, split), blocks, block);
        const int j0 = block * 16 * RT;
        Group g;
        if (SELF) {
            g.tile = __builtin_ctzll(__ballot(upto > k));
            if (g.tile) k -= __builtin_amdgcn_readlane(upto, g.tile - 1);
            const uint64_t leaders = masks[g.tile];
            const int mine = ids[g.tile][lane];
            const int first =
                __builtin_ctzll(__ballot((leaders >> lane & 1) && __popcll(leaders & ((1ull << lane) - 1)) == k));
            g.adapter = __builtin_amdgcn_readlane(mine, first);
            g.mask = __ballot(mine == g.adapter);
            g.rank = (uint32_t)g.adapter < (uint32_t)a.L ? rank_of(a, g.adapter) : 0;
        } else {
            g = group_of(a, rows, k);
        }
        if (j0 >= g.rank || !g.mask) continue;
        gather_rows(g.mask, list);
        const int cnt = __popcll(g.mask);
        const int64_t slab = (int64_t)g.tile * kTile, row0 = m0 + slab;
        const int w0 = split * h.per, w1 = min(w0 + h.per, windows);
        float *part = parts_of(a, rows) + (int64_t)split * rows * a.R;
        if (cnt <= 16) shrink_group<X, W, 1, RT>(a, row0, slab, g.adapter, g.rank, j0, cnt, list, w0, w1, part, red);
        else if (cnt <= 32) shrink_group<X, W, 2, RT>(a, row0, slab, g.adapter, g.rank, j0, cnt, list, w0, w1, part, red);
        else shrink_group<X, W, 4, RT>(a, row0, slab, g.adapter, g.rank, j0, cnt, list, w0, w1, part, red);
    }
}

// ------------------------------------------------------------------ expand
// v beside weights of type W: bf16 parts as above, or two fp16 parts of the scaled row.
template <typename W>
struct Held {
    static constexpr bool kScaled = std::is_same<W, _Float16>::value;
    static constexpr int kParts = kScaled ? 2 : 3;
};

// Entries from the n-th on become 0: ranks past the adapter's own, whatever they hold.
template <typename W>
__device__ __forceinline__ void cut(Eight<W> &x, int n) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = e < n ? x[e] : (W)0.0f;
}

// Workgroups a CU: three, one of ranks above 128.  Threads that share out the ranges of k in staging: all, but half of them
// beside bf16 weights of 65 to 128 ranks, whose three parts leave LDS for three workgroups only then (500 rows of rank 128, k
// 4096, 8192 columns: 30.1 us, with all threads and two workgroups 37.9; 8000 rows 148 against 167; one row the same).
constexpr int kExpandBlocks = 3;
template <int KS>
constexpr int kResident = KS > 4 ? 1 : kExpandBlocks;
template <typename W, int KS>
constexpr int kSharing = KS == 4 && Held<W>::kParts == 3 ? kThreads / 2 : kThreads;
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

// Columns [n0, n1) of a group's rows; n0 is a multiple of kUnit, n1 too or N.  stage() puts the group's v into vp and undo.
template <typename W, typename T, int KS, int TT, typename Stage>
__device__ __forceinline__ void expand_group(const LoraArgs &a, int64_t row0, int id, int rank, float scale, int cnt, const uint8_t *list,
                                             const Eight<W> *vp, const float *undo, int64_t n0, int64_t n1, Stage &&stage) {
    // the fewer rows and ranks, the more columns a step, for loads under way
    constexpr int NT = TT * KS <= 2 ? 4 : 2, kParts = Held<W>::kParts;
    using C = Columns<T, NT>;
    const int wave = wave_id(), lane = threadIdx.x % kWave, col = lane % 16, g = lane / 16;
    const W *pb = (const W *)a.B + (int64_t)id * a.N * a.R;
    const T *base = (const T *)a.base + row0 * a.ldb;
    T *out = (T *)a.out + row0 * a.ldo;
    uint32_t ob[TT], oo[TT], ow[NT];  // bytes: 64 rows of strides below 2^24, 128 columns of 256 ranks
    float back[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int i = t * 16 + col;
        const uint32_t row = list[i < cnt ? i : 0];
        ob[t] = (row * (uint32_t)a.ldb + C::VW * g) * (uint32_t)sizeof(T);
        oo[t] = (row * (uint32_t)a.ldo + C::VW * g) * (uint32_t)sizeof(T);
    }
#pragma unroll
    for (int q = 0; q < NT; ++q) ow[q] = (C::of(q, col) * a.R + 8 * g) * (uint32_t)sizeof(W);
    // the row's power of two is taken back before the adapter's scale comes in: their product may leave fp32's range, or its
    // normal numbers, where the term is an ordinary one
    const auto term = [](float sum, float back) { return Held<W>::kScaled ? sum * back : sum; };
    typename C::V have[TT][C::kPieces];
    Eight<W> fb[KS][NT];
    const auto load = [&](int64_t n) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
            if (t * 16 + col < cnt) {
#pragma unroll
                for (int p = 0; p < C::kPieces; ++p) have[t][p] = at<const typename C::VU>(base + n + 4 * C::VW * p, ob[t]);
            }
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                fb[ks][q] = ks * 32 + 8 * g < rank ? load8(pb + n * a.R + ks * 32, ow[q]) : zero8<W>();
    };
    const int64_t whole = n0 + (n1 - n0) / C::kStep * C::kStep;  // n1 but for the columns at N's end
    int64_t n = n0 + wave * C::kStep;
    // the first step's loads are under way while v is staged, where the registers last
    if (TT < 4 && n < whole) load(n);
    stage();
    if (TT == 4 && n < whole) load(n);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int i = t * 16 + col;
        back[t] = Held<W>::kScaled ? undo[i < cnt ? i : 0] : 1.0f;
    }
    for (; n < whole; n += kWaves * C::kStep) {
        if (rank & 7) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int q = 0; q < NT; ++q) cut(fb[ks][q], rank - ks * 32 - 8 * g);
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
        for (int t = 0; t < TT; ++t)
            if (t * 16 + col < cnt) {
#pragma unroll
                for (int p = 0; p < C::kPieces; ++p) {
                    typename C::V o;
#pragma unroll
                    for (int i = 0; i < C::VW; ++i)
                        o[i] = (T)((float)have[t][p][i] + scale * term(acc[t][(p * C::VW + i) / 4][i % 4], back[t]));
                    at<typename C::VU>(out + n + 4 * C::VW * p, oo[t]) = o;
                }
            }
        if (n + kWaves * C::kStep < whole) load(n + kWaves * C::kStep);
    }
    // the columns at N's end: 16 at a time, element by element, 16 rows a wave, all loads before the products
    for (int u = wave; whole + u / TT * 16 < n1; u += kWaves) {
        const int i = u % TT * 16 + col;
        const int64_t c = whole + u / TT * 16, nn = c + col < n1 ? c + col : n1 - 1;
        const int64_t row = list[i < cnt ? i : 0];
        Eight<W> b[KS];
        T old[4];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) b[ks] = ks * 32 + 8 * g < rank ? load8(pb + nn * a.R + 8 * g + ks * 32) : zero8<W>();
#pragma unroll
        for (int e = 0; e < 4; ++e) old[e] = base[row * a.ldb + (c + 4 * g + e < n1 ? c + 4 * g + e : n1 - 1)];
        f4 acc = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks * 32 >= rank) break;
            cut(b[ks], rank - ks * 32 - 8 * g);
#pragma unroll
            for (int p = 0; p < kParts; ++p) acc = mfma(b[ks], vp[((p * KS + ks) * kTile + i) * 4 + g], acc);
        }
        const float one = Held<W>::kScaled ? undo[i] : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i < cnt && c + 4 * g + e < n1) out[row * a.ldo + c + 4 * g + e] = (T)((float)old[e] + scale * term(acc[e], one));
    }
}

// The rows of v of a group in LDS, as the matrix instruction's columns: vp[part][ks][token][g], 8 ranks each.  Where the
// group has fewer eights of ranks than there are threads, the ranges of k are shared out over threads too and meet in
// `some`, so that few rows wait for one or two loads and not for one after another.
template <typename W, int KS>
__device__ __forceinline__ void stage_v(const LoraArgs &a, int64_t slab, int rank, int cnt, const uint8_t *list, int rows,
                                        int splits, Eight<W> *vp, float *undo, uint32_t *top, Eight<float> *some) {
    constexpr int kParts = Held<W>::kParts;
    const int t = threadIdx.x, tokens = (cnt + 15) / 16 * 16, eights = (rank + 7) / 8;
    constexpr int all = KS * 4;  // eights of a token, those past the rank 0
    const float *parts = parts_of(a, rows) + slab * a.R;
    const int64_t range = (int64_t)rows * a.R;
    if constexpr (Held<W>::kScaled) {
        if (t < kTile) top[t] = 0;
        lds_barrier();
    }
    // entry u of tokens * all: the token, and its eight of ranks
    const auto put = [&](int u, const Eight<float> &sum) {
        const int i = u / all, j = u % all;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = i < cnt && j * 8 + e < rank ? sum[e] : 0.0f;
        if constexpr (Held<W>::kScaled) {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = __builtin_isfinite(v[e]) ? fmaxf(m, fabsf(v[e])) : m;
            if (m > 0.0f) atomicMax(&top[i], __builtin_bit_cast(uint32_t, m));
            // fp32 in the place of the parts until the row's scale is known: 32 bytes for two parts of 16
            vp[(j / 4 * kTile + i) * 4 + j % 4] = __builtin_bit_cast(Eight<W>, f4{v[0], v[1], v[2], v[3]});
            vp[((KS + j / 4) * kTile + i) * 4 + j % 4] = __builtin_bit_cast(Eight<W>, f4{v[4], v[5], v[6], v[7]});
        } else {
            bf8 part[kParts];
            split<kParts>(v, part);
#pragma unroll
            for (int p = 0; p < kParts; ++p) vp[((p * KS + j / 4) * kTile + i) * 4 + j % 4] = part[p];
        }
    };
    const auto add = [&](int u, int first, int step) {
        const int i = u / all, j = u % all;
        Eight<float> v = {};
        if (i < cnt && j < eights) {
            const float *p = parts + list[i] * a.R + j * 8;
#pragma unroll 8
            for (int s = first; s < splits; s += step) v += load8(p + s * range);
        }
        return v;
    };
    const int entries = tokens * all, bits = 32 - __builtin_clz(cnt * all - 1), wide = 1 << bits;  // cnt * all and more
    int share = 1;
    while (share < splits && 2 * share * wide <= kSharing<W, KS>) share *= 2;
    if (share > 1) {
        if (t < share * wide) some[t] = add(t % wide, t >> bits, share);
        lds_barrier();
        if (t < entries) {
            Eight<float> v = {};
            if (t < wide)
#pragma unroll 4
                for (int p = 0; p < share; ++p) v += some[p * wide + t];
            put(t, v);
        }
#pragma unroll 1
        for (int u = t + kThreads; u < entries; u += kThreads) put(u, Eight<float>{});
    } else {
#pragma unroll 1
        for (int u = t; u < entries; u += kThreads) put(u, add(u, 0, 1));
    }
    if constexpr (Held<W>::kScaled) {
        // the largest finite entry of each row goes to [2^14, 2^15): two fp16 parts then hold 22 bits of it, and
        // of smaller entries all that lies above 2^-38 of it
        lds_barrier();
#pragma unroll 1
        for (int u = t; u < entries; u += kThreads) {
            const int i = u / all, j = u % all;
            const int at0 = (j / 4 * kTile + i) * 4 + j % 4, at1 = ((KS + j / 4) * kTile + i) * 4 + j % 4;
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
    }
    lds_barrier();
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

// A fixed grid walks units (group, kUnit columns) in runs, columns fastest, so that a workgroup stages a group's v once
// for all its columns, and tiles of few and of many groups cost what their work costs.  Prefill 62 us, 4.4 TB/s of base and
// output.  Long prefill 338 us, which is 3.4 TB/s: each of some nine workgroups a group adds up and parts the same 64 rows of
// 128 ranks in front of its run.  Prompts 22 us: the same by some 54 workgroups a group.  Decode batch 18 us (3.2 TB/s) and one
// token 6 us are latency: the table, the parts of v, then steps whose loads (base and B) stand behind the last step's stores
// and right in front of the products that need them, so that only the CU's other waves, eleven at most, cover them.  Ranks
// above 128 leave one workgroup a CU: 4096 rows of rank 256, k 4096, 8192 columns 186 us with fp16 adapters and 16-bit
// outputs, of rank 136 127 us, of rank 128 100 us.
template <typename W, typename T, int KS>
__global__ __launch_bounds__(kThreads, (kResident<KS>)) void lora_expand_kernel(const LoraArgs a, int64_t m0,
                                                                                                int rows, int most) {
    __shared__ Eight<W> vp[Held<W>::kParts * KS * kTile * 4];
    __shared__ float undo[kTile];
    __shared__ uint32_t top[kTile];
    __shared__ Eight<float> some[kSharing<W, KS>];
    __shared__ uint8_t list[kTile];
    const Head *h = head_of(a);
    // (cut to what the workspace holds, as the table's entries are)
    const int splits = min((uint32_t)__builtin_amdgcn_readfirstlane(h->splits), (uint32_t)most);
    const int groups = min((uint32_t)__builtin_amdgcn_readfirstlane(h->groups + h->copies),
                           (uint32_t)tiles_in(rows) * (min(rows, kTile) + 1));
    if (groups == 0) return;
    // Up to as many groups as workgroups: as many workgroups for each, which meet one group only.  Otherwise runs over all
    // units; fewer than 2^32, as N <= 2^23 and 512 tiles have 65 groups each at most.
    const uint32_t per = (uint32_t)((a.N + kUnit - 1) / kUnit);
    uint32_t u, u1;
    int k;
    if ((uint32_t)groups <= gridDim.x) {
        int rest, part, more;
        const int share = min(quotient(gridDim.x, groups, rest), (int)per);
        k = quotient(blockIdx.x, share, part);
        if (k >= groups) return;
        const int each = quotient(per, share, more);
        u = (uint32_t)k * per + each * part + min(part, more);
        u1 = u + each + (part < more ? 1 : 0);
    } else {
        const uint32_t total = per * groups, each = total / gridDim.x, more = total % gridDim.x;
        u = each * blockIdx.x + min(blockIdx.x, more);
        u1 = u + each + (blockIdx.x < more ? 1 : 0);
        k = (int)(u / per);
    }
    for (; u < u1; ++k) {
        const uint32_t start = u - (uint32_t)k * per;
        const int64_t first = start, last = start + min(u1 - u, per - start);
        u += (uint32_t)(last - first);
        const int64_t n0 = first * kUnit, n1 = last * kUnit < a.N ? last * kUnit : a.N;
        const Group g = group_of(a, rows, k);
        const int ad = g.adapter, rank = g.rank, cnt = __popcll(g.mask);
        const int64_t slab = (int64_t)g.tile * kTile, row0 = m0 + slab;
        if (!g.mask || (rank == 0 && a.base == a.out)) continue;
        gather_rows(g.mask, list);
        if (rank == 0) {
            copy_rows<T>(a, row0, cnt, list, n0, n1);
            continue;
        }
        const auto stage = [&] { stage_v<W, KS>(a, slab, rank, cnt, list, rows, splits, vp, undo, top, some); };
        if (cnt <= 16) expand_group<W, T, KS, 1>(a, row0, ad, rank, g.scale, cnt, list, vp, undo, n0, n1, stage);
        else if (cnt <= 32) expand_group<W, T, KS, 2>(a, row0, ad, rank, g.scale, cnt, list, vp, undo, n0, n1, stage);
        else expand_group<W, T, KS, 4>(a, row0, ad, rank, g.scale, cnt, list, vp, undo, n0, n1, stage);
    }
}

// ------------------------------------------------------------------ launches
// the most ranges of k that the parts of v have room for: with one group a tile, and a window a wave or more
int most_splits(int64_t rows, int64_t K) {
    const int64_t tiles = (rows + kTile - 1) / kTile, windows = (K + kWindow - 1) / kWindow;
    return (int)std::max<int64_t>(1, std::min(std::max<int64_t>(4, kTarget / tiles), windows / kShrinkWaves));
}

template <typename X, typename W>
void shrink(const LoraArgs &a, int64_t m0, int rows, hipStream_t stream) {
    const int rt = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4, most = most_splits(rows, a.K);
    const int64_t tiles = (rows + kTile - 1) / kTile;
    const int64_t units = tiles * std::min<int64_t>({kTile, rows, a.L}) * blocks_of(a.R) * most;
    const uint32_t grid = (uint32_t)std::min<int64_t>(units, kTarget);
#define W4A8_SHRINK(RT)                                                                                            \
    (tiles > kSelf ? lora_shrink_kernel<X, W, RT, false><<<grid, kShrinkThreads, 0, stream>>>(a, m0, rows, most) \
                   : lora_shrink_kernel<X, W, RT, true><<<grid, kShrinkThreads, 0, stream>>>(a, m0, rows, most))
    if (rt == 1) W4A8_SHRINK(1);
    else if (rt == 2) W4A8_SHRINK(2);
    else W4A8_SHRINK(4);
#undef W4A8_SHRINK
}

template <typename W, typename T>
void expand(const LoraArgs &a, int64_t m0, int rows, hipStream_t stream) {
    const int64_t tiles = (rows + kTile - 1) / kTile;
    // no more workgroups than there can be units; as many as are resident, or where those would have long runs each, more
    // of shorter ones (long prefill 569 us with 46 units each, 520 with 12, 542 with 3; prefill 84 with 5 units each, 89 with 3)
    const int64_t units = tiles * std::min<int64_t>({kTile, rows, (int64_t)a.L + 1}) * ((a.N + kUnit - 1) / kUnit);
    const int64_t runs = tiles * ((a.N + kUnit - 1) / kUnit) / 12;
    const uint32_t grid = (uint32_t)std::min<int64_t>(units, std::max<int64_t>(256 * kExpandBlocks, std::min<int64_t>(runs, 1 << 20)));
#define W4A8_EXPAND(KS) lora_expand_kernel<W, T, KS><<<grid, kThreads, 0, stream>>>(a, m0, rows, most_splits(rows, a.K))
    if (a.R <= 32) W4A8_EXPAND(1);
    else if (a.R <= 64) W4A8_EXPAND(2);
    else if (a.R <= 128) W4A8_EXPAND(4);
    else W4A8_EXPAND(8);
#undef W4A8_EXPAND
}

template <typename W>
hipError_t launch_w(const LoraArgs &a, hipStream_t stream) {
    for (int64_t m0 = 0; m0 < a.M; m0 += kSlab) {
        const int rows = (int)std::min(a.M - m0, kSlab);
        if (tiles_in(rows) > kSelf)
            lora_table_kernel<<<1, kTableThreads, 0, stream>>>(a, m0, rows, most_splits(rows, a.K));
        if (a.x_type == W4A8_F32) shrink<float, W>(a, m0, rows, stream);
        else if (a.x_type == W4A8_F16) shrink<_Float16, W>(a, m0, rows, stream);
        else shrink<__bf16, W>(a, m0, rows, stream);
        if (a.out_type == W4A8_F32) expand<W, float>(a, m0, rows, stream);
        else if (a.out_type == W4A8_F16) expand<W, _Float16>(a, m0, rows, stream);
        else expand<W, __bf16>(a, m0, rows, stream);
        if (hipError_t err = hipGetLastError(); err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace

namespace w4a8 {

// Room for the first slab, which is the largest.  The parts of v of `rows` rows are most_splits(rows) * rows * R, and that falls
// here and there as rows grow, so that a smaller batch can have more of them; the room is for the least bound that does not:
// rows * kTarget / tiles <= kTile * kTarget, and 4 * rows (most_splits' two terms), of as many ranges as there are windows for.
int64_t lora_ws_bytes(int64_t M, int64_t K, int32_t, int32_t R) {
    if (M == 0) return 0;
    const int64_t rows = std::min(M, kSlab), windows = (K + kWindow - 1) / kWindow;
    const int64_t held = std::min(std::max<int64_t>(1, windows / kShrinkWaves) * rows, std::max<int64_t>(kTile * kTarget, 4 * rows));
    return parts_at((int)rows) + held * R * 4;
}

hipError_t launch_lora_add(const LoraArgs &a, hipStream_t stream) {
    return a.ab_type == W4A8_F16 ? launch_w<_Float16>(a, stream) : launch_w<__bf16>(a, stream);
}

}  // namespace w4a8
