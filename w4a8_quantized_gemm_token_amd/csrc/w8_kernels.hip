// w8_kernels.hip -- the W8A8 product on gfx950 (CDNA4) matrix cores: INT8 activations with a
// scale per token, INT8 weights with a scale per output channel.
//
//     isum[m][n] = sum_k qa[m][k] qw[n][k]                         (int32, exact: K < 2^17)
//     out[m][n]  = T(fp32(isum) * a_scale[m] * w_scale[n] + bias[n])
//
// The same product runs dense, and per expert over the slot lists of the router.  The sums are
// integers, so neither the order of k nor a split of it changes a result: every loop gives the
// same bytes.
//
// Two loops.  Up to 16 rows (slice_walk) the weights are read once and are the whole cost: 235 MB
// in 39.7 us (K 8192, N 28672, one row), 5.9 TB/s, where a large copy moves 5.1 TB/s.  More rows go
// through LDS tiles (tile_unit): 4096 x 8192 x 8192 in 199-218 us among other passes on different
// boxes, 2.5-2.8 POPS, and from 203 us up to 239 in the median of 20 launches in a row, as the clock
// falls under the load; the matrix pipes alone, fed from registers, run at 3.9 POPS with random codes
// and at 4.8 with zeros.
#include <algorithm>
#include <type_traits>

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
// m, four neighbouring output channels per block.  The weight rows are dealt to the blocks so that
// G blocks (16 bytes of outputs; see wrow) make 4 G neighbours of a lane and 16 G of a row's four
// lanes: a store instruction writes 64-byte pieces.
// Both operands go straight from memory into LDS (16 bytes per lane), 128 bytes of k per stage,
// NST stages.  LDS rows are 128 bytes; the 16-byte chunk c of row r sits at chunk c ^ key(r), so
// that the 16 rows of a fragment read fall in distinct banks.
// A stage is computed in two halves of 64 k.  The fragments of a half are read while the half
// before it is multiplied, so the one barrier per stage stands between the halves of stage g:
// there every wave holds the fragments of its second half in registers (the stage's buffer is
// free for stage g + NST) and stage g + 1 has landed (its first half may be read).
// 256 x 256 at M 4096, K = N 8192: MFMA busy 77% of the CUs' busy cycles, no LDS bank conflicts, 20% of
// the L2 reads miss.  The other forms take 249 us there (128 x 256), 320 (128 x 128), 447 (64 x 64) and
// 598 (32 x 64), this one 214.
typedef __attribute__((address_space(3))) void *lds_ptr_t;
typedef const __attribute__((address_space(1))) void *glb_ptr_t;

// s_waitcnt immediate: at most vm memory loads and lgkm LDS accesses outstanding
constexpr int waitcnt(int vm, int lgkm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8); }

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)0xFFFFFFFF, 0x00020000);
}

// A value that every lane holds alike, for the scalar registers (a resource descriptor that the
// compiler cannot prove uniform costs a loop over its values at every load).
__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)v), hi = __builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
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
    static __device__ int key_a(int r) { return (r >> 1) & 7; }
};

// G column blocks whose outputs of one lane are neighbours; their weight rows and LDS keys.
template <int G>
struct Deal {
    // the fragment row i (0..15) of a wave's column block cb is its weight row wrow(i, cb)
    static __device__ int wrow(int i, int cb) { return 16 * G * (cb / G) + 4 * G * (i >> 2) + 4 * (cb % G) + (i & 3); }
    // chunk key of LDS row r: distinct over a fragment's 8 rows of one parity, the same for all blocks
    static __device__ int key(int r) { return ((r >> 1) & 1) | (((r / (4 * G)) & 3) << 1); }
};

// src_row(r), r < rows: activation row of the tile's row r, or -1 (computed as row 0, not stored).
// WIDE: rows may lie 2^32 bytes or more behind qa.  (Its loads take 64-bit addresses, and the compiler
// counts those as able to touch LDS by themselves: it then waits for every access in flight where
// it would wait for some.)
template <typename C, bool WIDE, typename T, typename SrcRow>
__device__ __forceinline__ void tile_unit(uint8_t *lds, const int8_t *__restrict__ qa,
                                          const float *__restrict__ a_scale, SrcRow src_row, int64_t slot0, int rows,
                                          int64_t K, const int8_t *__restrict__ qw,
                                          const float *__restrict__ w_scale, int64_t N, int64_t n0,
                                          const float *__restrict__ bias, T *__restrict__ out, int64_t ldo) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int full = (int)(K >> 7), steps = (int)((K + 127) >> 7);  // whole stages, all stages
    const int tail = (int)(K & 127) >> 4;                          // chunks of a last part stage

    constexpr int V4 = 4 / (int)sizeof(T), G = C::CB >= V4 ? V4 : C::CB;  // blocks of a 16-byte store
    using D = Deal<G>;
    constexpr int kReads = C::RB + C::CB, kMul = C::RB * C::CB, kLoads = C::LA + C::LB;

    // ---- loads: lane L of load j fills chunk L & 7 of row 8 (L? wave + j) + (L >> 3)
    const int8_t *aptr[WIDE ? C::LA : 1];
    uint32_t aoff[C::LA], boff[C::LB];
    int ach[C::LA], bch[C::LB];
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(qa);
#pragma unroll
    for (int j = 0; j < C::LA; ++j) {
        const int r = 8 * (C::LA * wave + j) + (lane >> 3);
        int64_t src = src_row(r < rows ? r : rows - 1);
        if (src < 0) src = 0;
        ach[j] = (lane & 7) ^ C::key_a(r);
        if constexpr (WIDE) aptr[j] = qa + src * K + 16 * ach[j];
        else aoff[j] = (uint32_t)src * (uint32_t)K + 16u * (uint32_t)ach[j];
    }
    const __amdgpu_buffer_rsrc_t rb = make_rsrc((const void *)uniform((int64_t)(qw + n0 * K)));
#pragma unroll
    for (int j = 0; j < C::LB; ++j) {
        const int r = 8 * (C::LB * wave + j) + (lane >> 3);
        const int64_t c = n0 + r < N ? r : N - 1 - n0;
        bch[j] = (lane & 7) ^ D::key(r);
        boff[j] = (uint32_t)(c * K) + 16u * (uint32_t)bch[j];
    }
    auto load_one = [&](int g, int st, int j) {  // load j of a whole stage
        if (j < C::LB) {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rb, (lds_ptr_t)(lds + st * C::kStage + C::kStageA + 1024 * (C::LB * wave + j)), 16, (int)boff[j % C::LB],
                g * 128, 0, 0);
        } else {
            const int i = (j - C::LB) % C::LA;
            const lds_ptr_t to = (lds_ptr_t)(lds + st * C::kStage + 1024 * (C::LA * wave + i));
            if constexpr (WIDE)
                __builtin_amdgcn_global_load_lds((glb_ptr_t)(aptr[i] + (int64_t)g * 128), to, 16, 0, 0);
            else __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to, 16, (int)aoff[i], g * 128, 0, 0);
        }
    };
    auto issue = [&](int g, int st) {
        if (g < full) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) load_one(g, st, j);
        } else {
            // the part stage: chunks past K are not loaded; on the activations' side they are zeros,
            // so whatever the weights' side of the buffer holds there counts for nothing
#pragma unroll
            for (int j = 0; j < C::LB; ++j)
                if (bch[j] < tail) load_one(g, st, j);
#pragma unroll
            for (int j = 0; j < C::LA; ++j) {
                if (ach[j] < tail) load_one(g, st, C::LB + j);
                else
                    *reinterpret_cast<v4i *>(lds + st * C::kStage + 1024 * (C::LA * wave + j) + 16 * lane) =
                        v4i{0, 0, 0, 0};
            }
        }
        // the counted waits need the stages' loads in order
        __asm__ volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- fragments: lane l takes row (l & 15) of a block, chunk 4 ks + (l >> 4)
    const int fr = lane & 15, qd = lane >> 4;
    int aofs[2], bofs[2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const int ra = wm * C::RB * 16 + fr, rw = wn * C::CB * 16 + D::wrow(fr, 0);
        aofs[ks] = ra * 128 + (((4 * ks + qd) ^ C::key_a(ra)) << 4);
        bofs[ks] = C::kStageA + rw * 128 + (((4 * ks + qd) ^ D::key(rw)) << 4);
    }
    struct Frags {
        v4i a[C::RB], b[C::CB];
    };
    auto read_one = [&](Frags &f, int st, int ks, int r) {
        const uint8_t *base = lds + st * C::kStage;
        if (r < C::CB) f.b[r % C::CB] = *reinterpret_cast<const v4i *>(base + bofs[ks] + 128 * D::wrow(0, r));
        else f.a[(r - C::CB) % C::RB] = *reinterpret_cast<const v4i *>(base + aofs[ks] + 2048 * (r - C::CB));
    };
    v4i acc[C::RB][C::CB] = {};
    // Products of the half in `now`; after each of them one fragment of the half after it (stage st,
    // half ks, if rd) and after every second one a load of stage g into the buffer sti (if ld), in
    // just this order: the reads are then back long before the half ends, and no burst of loads
    // holds up the products.  (The compiler's own order put the reads behind the loads, at the end:
    // 225 us against 211 at M 4096, K = N 8192.)
    auto half = [&](const Frags &now, auto rd, Frags &then, int st, int ks, auto ld, int g, int sti) {
        // read r and load d follow these products (a small tile has fewer products than reads or loads)
        constexpr auto read_at = [](int r) { return kMul > kReads + 2 ? r + 2 : r * kMul / kReads; };
        constexpr auto load_at = [](int d) { return kMul >= 2 * kLoads ? 2 * d + 1 : d * kMul / kLoads; };
        int r = 0, d = 0;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < kMul; ++m) {
            const int i = m / C::CB, j = m % C::CB;
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(now.b[j], now.a[i], acc[i][j], 0, 0, 0);
            if constexpr (decltype(rd)::value)
                for (; r < kReads && read_at(r) <= m; ++r) read_one(then, st, ks, r);
            if constexpr (decltype(ld)::value)
                for (; d < kLoads && load_at(d) <= m; ++d) load_one(g, sti, d);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    // a barrier that leaves `vm` loads in flight, with every LDS access done
    auto stage_barrier = [&](auto vm) {
        __asm__ volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(waitcnt(decltype(vm)::value, 0));
        __builtin_amdgcn_s_barrier();
        __asm__ volatile("" ::: "memory");
    };
    using Ahead = std::integral_constant<int, (C::NST - 2) * kLoads>;  // the stages behind the next one
    using None = std::integral_constant<int, 0>;

    // ---- prologue: NST stages on their way, stage 0's first half into registers
#pragma unroll
    for (int g = 0; g < C::NST; ++g)
        if (g < steps) issue(g, g);
    if (C::NST <= full) {
        using First = std::integral_constant<int, (C::NST - 1) * kLoads>;
        stage_barrier(First{});
    } else {
        stage_barrier(None{});
    }
    Frags f0, f1;
#pragma unroll
    for (int r = 0; r < kReads; ++r) read_one(f0, 0, 0, r);
    int st = 0, g = 0;
    auto lds_wait = [&]() {  // f0 is back (or nearly) before new reads are issued behind it
        __builtin_amdgcn_s_waitcnt(waitcnt(63, 0));
    };
    for (; g + C::NST < full; ++g) {
        lds_wait();
        half(f0, Yes{}, f1, st, 1, No{}, 0, 0);
        stage_barrier(Ahead{});
        const int sti = st;
        st = st + 1 == C::NST ? 0 : st + 1;
        half(f1, Yes{}, f0, st, 0, Yes{}, g + C::NST, sti);
    }
    // the last stages: fewer loads in flight, or a part stage's: every wait is for all of them
    for (; g < steps - 1; ++g) {
        lds_wait();
        half(f0, Yes{}, f1, st, 1, No{}, 0, 0);
        stage_barrier(None{});
        if (g + C::NST < steps) issue(g + C::NST, st);
        st = st + 1 == C::NST ? 0 : st + 1;
        half(f1, Yes{}, f0, st, 0, No{}, 0, 0);
    }
    lds_wait();
    half(f0, Yes{}, f1, st, 1, No{}, 0, 0);
    half(f1, No{}, f0, st, 0, No{}, 0, 0);

    // ---- epilogue: lane l holds row 16 i + (l & 15) and, of block j, weight rows wrow(4 (l >> 4) + r, j)
    constexpr int V = 4 * G, kPieces = C::CB / G;
    typedef T vt __attribute__((ext_vector_type(V), aligned(sizeof(T))));
    const int64_t nb = n0 + wn * C::CB * 16 + V * qd;
    float ws[kPieces][V], bv[kPieces][V];
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const int64_t n = nb + 4 * V * p + c < N ? nb + 4 * V * p + c : N - 1;
            ws[p][c] = w_scale[n];
            bv[p][c] = bias ? bias[n] : 0.0f;
        }
#pragma unroll
    for (int i = 0; i < C::RB; ++i) {
        const int m = wm * C::RB * 16 + 16 * i + fr;
        const int64_t row = m < rows ? src_row(m) : -1;
        if (row < 0) continue;
        const float as = a_scale[row];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int64_t n = nb + 4 * V * p;
            T *o = out + (slot0 + m) * ldo + n;
            vt v;
#pragma unroll
            for (int c = 0; c < V; ++c)
                v[c] = finish<T>(acc[i][G * p + (c >> 2)][c & 3], as, ws[p][c], bv[p][c], bias != nullptr);
            if (n + V <= N) *reinterpret_cast<vt *>(o) = v;  // any alignment
            else {
#pragma unroll
                for (int c = 0; c < V; ++c)
                    if (n + c < N) o[c] = v[c];
            }
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

// (256 threads: two waves per SIMD are asked for, or the compiler spreads over 512 registers and moves
// accumulators about.)
template <typename C, typename T>
__global__ __launch_bounds__(C::kThreads, C::kThreads == 256 ? 2 : 1) void gemm_w8a8_tile_kernel(const int8_t *__restrict__ qa,
                                                                     const float *__restrict__ a_scale, int64_t M,
                                                                     int64_t K, const int8_t *__restrict__ qw,
                                                                     const float *__restrict__ w_scale, int64_t N,
                                                                     const float *__restrict__ bias,
                                                                     T *__restrict__ out, int64_t ldo) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
    const int64_t mt = (M + C::BM - 1) / C::BM, nt = (N + C::BN - 1) / C::BN;
    int64_t tm, tn;
    panel_tile<4>(blockIdx.x, mt, nt, tm, tn);
    const int64_t m0 = tm * C::BM;
    const int rows = (int)((M - m0) < C::BM ? (M - m0) : C::BM);
    tile_unit<C, false, T>(lds, qa + m0 * K, a_scale + m0, [](int r) { return (int64_t)r; }, m0, rows, K, qw, w_scale, N,
                           tn * C::BN, bias, out, ldo);
}

// ------------------------------------------------------------------ few rows
// Up to 16 rows: the weights are the whole cost, and each byte of them is used once.  A
// workgroup's waves share out k in 128-byte windows (wave w has the windows w + W i, i < NW, of
// a pass of W NW windows; one pass where K allows) and walk the same run of 16-channel tiles, so
// a wave keeps its slice of the activations in registers for the whole run and does nothing but
// stream weights through a ring of registers (D tiles deep).  The waves' int32 partial sums of a
// tile meet in LDS, and one wave after the other ends a tile.
// A load instruction covers whole 128-byte lines: lane L of load j reads channel 8 j + (L & 7),
// chunk L >> 3 of the window.  The product wants lane l to hold channel l & 15 and, in its two
// steps, the chunks 2 (l >> 4) and 2 (l >> 4) + 1: for channels 0-7 the one is the lane's own and
// the other lane l + 8's, for channels 8-15 the other way round -- a rotation by 8 of each 16
// lanes, written to half of them.
// Channels past N and bytes past the array read as 0 (the descriptor ends with the array); k past
// K and the windows that a wave has no share of are zeros on the activations' side.
// K 8192, N 28672: one row 39.7 us, 16 rows 42.6 (49.5 and 76 with the rows read from the caches per
// window and one tile per workgroup).
template <int BANKS>
__device__ __forceinline__ v4i ror8_into(v4i old, v4i src) {
    v4i r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_update_dpp(old[i], src[i], 0x128, 0xF, BANKS, false);
    return r;
}

constexpr int kMaxSliceWaves = 16;

// Walk: the tiles of a workgroup's run, one after the other: w and bytes (the weights of the
// tile's first channel, and from there to the end of the array's or the expert's last row), n0
// (the first channel), block (the rows stay in registers while it stays), next(), and rows(f),
// which calls f(src_row, slot0, rows, w_scale).  ONE: a single pass.
template <int NW, bool ONE, typename T, typename Walk>
__device__ __forceinline__ void slice_walk(v4i (*red)[kMaxSliceWaves][64], Walk to_load, int64_t tiles,
                                           const int8_t *__restrict__ qa, const float *__restrict__ a_scale, int64_t K,
                                           int passes, int64_t N, const float *__restrict__ bias, T *__restrict__ out,
                                           int64_t ldo) {
    constexpr int D = 4 / NW > 0 ? 4 / NW : 1;  // tiles in the ring: about 4 windows, 8 KB a wave
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int W = blockDim.x >> 6;
    const int qd = lane >> 4;
    const int windows = (int)((K + 127) >> 7);
    const uint32_t lofs = (uint32_t)(lane & 7) * (uint32_t)K + 16u * (uint32_t)(lane >> 3), row8 = 8u * (uint32_t)K;
    Walk now = to_load;  // the tile of the products; to_load is D steps ahead

    v4i a[NW][2], ring[D][NW][2];
    int64_t loaded = 0;
    int load_pass = 0;
    auto load = [&](v4i (&x)[NW][2], int i) {  // window i of the next tile (or pass) to load
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            (void *)to_load.w, (short)0, (int)(uint32_t)(to_load.bytes < 0xFFFFFFFFll ? to_load.bytes : 0xFFFFFFFFll),
            0x00020000);
        int w = (load_pass * NW + i) * W + wave;
        w = w < windows ? w : wave < windows ? wave : 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            x[i][j] = __builtin_bit_cast(
                v4i, __builtin_amdgcn_raw_buffer_load_b128(rs, lofs + (uint32_t)w * 128u + j * row8, 0, 2));
        // past the run's end its last tile is loaded again: the waits always count the same loads
        if (i < NW - 1) return;
        if (!ONE && ++load_pass < passes) return;
        load_pass = 0;
        if (++loaded < tiles) to_load.next();
    };
    float as = 0.0f;
    auto load_rows = [&](int pass) {
        now.rows([&](auto src_row, int64_t, int rows, const float *) {
            int64_t src = src_row((lane & 15) < rows ? lane & 15 : rows - 1);
            src = src < 0 ? 0 : src;
            as = a_scale[src];
            const int8_t *p = qa + src * K;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const int w = (pass * NW + i) * W + wave;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const int64_t k = (int64_t)w * 128 + 32 * qd + 16 * s;
                    const v4i v = *reinterpret_cast<const v4i *>(p + (k < K ? k : 0));
                    a[i][s] = k < K ? v : v4i{0, 0, 0, 0};
                }
            }
        });
    };
    int64_t block = now.block;
    if (ONE) load_rows(0);
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            load(ring[d], i);
        }
    __builtin_amdgcn_sched_barrier(0);
    v4i acc = {};
    int turn = 0, pass = 0, mine = 0;  // mine: the wave that ends the tile
    for (int64_t left = tiles; left > 0;) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (left > 0) {
                if (!ONE) {
                    load_rows(pass);
                } else if (now.block != block) {
                    load_rows(0);
                    block = now.block;
                }
                if (ONE || pass == 0) acc = v4i{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < NW; ++i) {
                    const v4i w0 = ror8_into<0xC>(ring[d][i][0], ring[d][i][1]);
                    const v4i w1 = ror8_into<0x3>(ring[d][i][1], ring[d][i][0]);
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w0, a[i][0], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w1, a[i][1], acc, 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    load(ring[d], i);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (ONE || ++pass == passes) {
                    pass = 0;
                    red[turn][wave][lane] = acc;
                    // LDS done, the weights stay in flight; the other half of red was read before this
                    // barrier by the wave that ended the tile before
                    __asm__ volatile("" ::: "memory");
                    __builtin_amdgcn_s_waitcnt(waitcnt(63, 0));
                    __builtin_amdgcn_s_barrier();
                    __asm__ volatile("" ::: "memory");
                    if (mine == wave)
                        now.rows([&](auto src_row, int64_t slot0, int rows, const float *w_scale) {
                            v4i s = red[turn][0][lane];
                            for (int w = 1; w < W; ++w) s += red[turn][w][lane];
                            // lane l: row l & 15, channels 4 (l >> 4) + r
                            const int m = lane & 15;
                            if (m >= rows || src_row(m) < 0) return;
                            const int64_t nb = now.n0 + 4 * qd;
                            T *o = out + (slot0 + m) * ldo + nb;
                            typedef T vt __attribute__((ext_vector_type(4), aligned(sizeof(T))));
                            vt v;
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int64_t n = nb + r < N ? nb + r : N - 1;
                                v[r] = finish<T>(s[r], as, w_scale[n], bias ? bias[n] : 0.0f, bias != nullptr);
                            }
                            if (nb + 4 <= N) *reinterpret_cast<vt *>(o) = v;  // any alignment
                            else {
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    if (nb + r < N) o[r] = v[r];
                            }
                        });
                    mine = mine + 1 == W ? 0 : mine + 1;
                    turn ^= 1;
                    --left;
                    if (left > 0) now.next();
                }
            }
        }
    }
}

// Workgroup b of g takes the tiles [begin(b), begin(b + 1)) of n: equal runs, the first ones longer.
__device__ __forceinline__ int64_t run_begin(int64_t b, int64_t g, int64_t n) {
    return n / g * b + (b < n % g ? b : n % g);
}

struct DenseWalk {
    const int8_t *w;
    int64_t bytes, n0, step, block;  // step: bytes of a tile
    int rows_;
    const float *w_scale;
    __device__ void next() {
        w += step;
        bytes -= step;
        n0 += 16;
    }
    template <typename F>
    __device__ void rows(F f) const {
        f([](int r) { return (int64_t)r; }, (int64_t)0, rows_, w_scale);
    }
};

template <int NW, bool ONE, typename T>
__global__ __launch_bounds__(64 * kMaxSliceWaves) void gemm_w8a8_slice_kernel(
    const int8_t *__restrict__ qa, const float *__restrict__ a_scale, int64_t M, int64_t K, int passes,
    const int8_t *__restrict__ qw, const float *__restrict__ w_scale, int64_t N, const float *__restrict__ bias,
    T *__restrict__ out, int64_t ldo) {
    __shared__ v4i red[2][kMaxSliceWaves][64];
    const int64_t nt = (N + 15) / 16, u0 = run_begin(blockIdx.x, gridDim.x, nt);
    const DenseWalk walk{qw + u0 * 16 * K, (N - u0 * 16) * K, u0 * 16, 16 * K, 0, (int)M, w_scale};
    slice_walk<NW, ONE, T>(red, walk, run_begin(blockIdx.x + 1, gridDim.x, nt) - u0, qa, a_scale, K, passes, N,
                               bias, out, ldo);
}

// ------------------------------------------------------------------ per expert
constexpr int kMaxE = 1024;

// Activation row of a unit's row r: row_index of its slot (or the slot), -1 outside [0, R).
struct SlotRows {
    const int32_t *row_index;
    int64_t slot0, R;
    __device__ int64_t operator()(int r) const {
        const int64_t row = row_index ? (int64_t)row_index[slot0 + r] : slot0 + r;
        return row >= 0 && row < R ? row : -1;
    }
};

// Work units of the experts with lo < slots <= hi: ceil(slots / bm) row blocks each, times nt column
// tiles.  pfx[0 .. E] receives the exclusive prefix of the row blocks over experts (whole
// workgroup; E <= 1024), cut off at the most there can be of ascending offsets, so that offsets that
// are not ascending cost no more work than others; pfx[kMaxE + 1 ..] is scratch.
constexpr int kPfx = kMaxE + 1 + 2 * 16 + 1;
__device__ __forceinline__ void block_prefix(int32_t *pfx, const int32_t *__restrict__ offsets, int32_t E,
                                             int64_t max_slots, int lo, int hi, int bm) {
    int64_t *part = reinterpret_cast<int64_t *>(pfx + kMaxE + 2);  // 8-byte aligned, as pfx is
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
    const int per = (E + blockDim.x - 1) / blockDim.x;  // <= 16 experts per thread
    const int64_t most = E + max_slots / bm;            // < 2^31
    auto blocks = [&](int e) -> int64_t {
        const int64_t c = clamp_slots(offsets[e + 1], max_slots) - clamp_slots(offsets[e], max_slots);
        return c > lo && c <= hi ? (c + bm - 1) / bm : 0;
    };
    const int e0 = tid * per, e1 = e0 + per < E ? e0 + per : E;
    int64_t own = 0;
    for (int e = e0; e < e1; ++e) own += blocks(e);
    int64_t incl = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t o = __shfl_up(incl, off, 64);
        if (lane >= off) incl += o;
    }
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    int64_t run = incl - own;
    for (int w = 0; w < wave; ++w) run += part[w];
    for (int e = e0; e < e1; ++e) {
        pfx[e] = (int32_t)(run < most ? run : most);
        run += blocks(e);
    }
    if (tid == 0) {
        int64_t total = 0;
        for (int w = 0; w < nw; ++w) total += part[w];
        pfx[E] = (int32_t)(total < most ? total : most);
    }
    __syncthreads();
}

// the expert of row block u: the last e with pfx[e] <= u
__device__ __forceinline__ int find_expert(const int32_t *pfx, int32_t E, int32_t u) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pfx[mid] <= u) lo = mid;
        else hi = mid;
    }
    return __builtin_amdgcn_readfirstlane(lo);  // u is the same for the whole workgroup
}

struct ExpertWalk {
    const int8_t *w;
    int64_t bytes, n0, block;
    int64_t e, K, N, R, max_slots;
    int32_t E;
    const int8_t *qw;
    const float *w_scale;
    const int32_t *pfx, *offsets, *row_index;
    __device__ void at(int64_t b, int64_t n) {
        block = b;
        n0 = n;
        e = find_expert(pfx, E, (int32_t)b);
        w = qw + (e * N + n) * K;
        bytes = (N - n) * K;
    }
    __device__ void next() {
        n0 += 16;
        w += 16 * K;
        bytes -= 16 * K;
        if (n0 >= N) at(block + 1, 0);
    }
    template <typename F>
    __device__ void rows(F f) const {
        const int64_t s0 = clamp_slots(offsets[e], max_slots) + 16 * (block - pfx[e]);
        const int64_t left = clamp_slots(offsets[e + 1], max_slots) - s0;
        f(SlotRows{row_index, s0, R}, s0, left < 16 ? (int)left : 16, w_scale + e * N);
    }
};

// Experts of up to 16 slots: a workgroup's run of tiles goes through one expert after the other.
// Bound by the weights: 64 tokens, top 8 of 384, K 7168, N 4096 (212-220 experts, 6.2-6.5 GB) 0.96 ms here
// (1.69 ms when every 16-channel tile read its rows and shared out k by itself); one token 45 us.
template <int NW, bool ONE>
__global__ __launch_bounds__(64 * kMaxSliceWaves) void grouped_w8a8_slice_kernel(
    const int8_t *__restrict__ qa, const float *__restrict__ a_scale, int64_t R, const int32_t *__restrict__ row_index,
    const int32_t *__restrict__ offsets, int32_t E, int64_t K, int passes, const int8_t *__restrict__ qw,
    const float *__restrict__ w_scale, int64_t N, int64_t max_slots, int hi, float *__restrict__ out) {
    __shared__ v4i red[2][kMaxSliceWaves][64];
    __shared__ __attribute__((aligned(8))) int32_t pfx[kPfx];
    block_prefix(pfx, offsets, E, max_slots, 0, hi, 16);
    const int64_t nt = (N + 15) / 16, units = uniform(pfx[E]) * nt;
    const int64_t u0 = run_begin(blockIdx.x, gridDim.x, units), u1 = run_begin(blockIdx.x + 1, gridDim.x, units);
    if (u0 >= u1) return;
    ExpertWalk walk{nullptr, 0, 0, 0, 0, K, N, R, max_slots, E, qw, w_scale, pfx, offsets, row_index};
    const int64_t b = uniform(u0 / nt);
    walk.at(b, uniform((u0 - b * nt) * 16));
    slice_walk<NW, ONE, float>(red, walk, u1 - u0, qa, a_scale, K, passes, N, nullptr, out, N);
}

// Experts with more than lo slots on C's tiles: a persistent grid over (row block, column tile)
// units, an expert's row blocks next to each other on one XCD, so that its weights come
// through one L2.  4096 tokens, top 8 of 384, K 7168, N 4096 (some 335 experts here, 10 GB) 2.13 ms: 4.9
// TB/s of weights, MFMA busy 42% of the CUs' busy cycles.  A 64 x 256 form for 17-64 slots and this one
// for the rest took as long (0.91 + 1.23 ms) with a launch more, 256 x 256 above 128 slots 5% longer, two
// stages instead of three 12%.
template <typename C>
__global__ __launch_bounds__(C::kThreads) void grouped_w8a8_tile_kernel(
    const int8_t *__restrict__ qa, const float *__restrict__ a_scale, int64_t R, const int32_t *__restrict__ row_index,
    const int32_t *__restrict__ offsets, int32_t E, int64_t K, const int8_t *__restrict__ qw,
    const float *__restrict__ w_scale, int64_t N, int64_t max_slots, int lo, float *__restrict__ out) {
    // one LDS object: with several, the compiler tells the loads into LDS and the reads apart by
    // object and puts a wait for every load in flight before the reads of the stages
    __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds + kPfx * 4];
    int32_t *pfx = reinterpret_cast<int32_t *>(lds + C::kLds);
    block_prefix(pfx, offsets, E, max_slots, lo, 0x7FFFFFFF, C::BM);
    const int64_t nt = (N + C::BN - 1) / C::BN, units = pfx[E] * nt;
    const int64_t per = gridDim.x / 8;  // the grid is a multiple of 8
    for (int64_t u = blockIdx.x % 8 * per + blockIdx.x / 8; u < units; u += gridDim.x) {
        // unit order: expert, column tile, row block
        const int e = find_expert(pfx, E, (int32_t)(u / nt));
        const int64_t p0 = pfx[e], nb = pfx[e + 1] - p0;
        const int64_t b = (u - p0 * nt) % nb, tn = (u - p0 * nt) / nb;
        const int64_t s0 = clamp_slots(offsets[e], max_slots) + C::BM * b;
        const int64_t left = clamp_slots(offsets[e + 1], max_slots) - s0;
        tile_unit<C, true, float>(lds, qa, a_scale, SlotRows{row_index, s0, R}, s0, left < C::BM ? (int)left : C::BM, K,
                            qw + e * N * K, w_scale + e * N, N, tn * C::BN, nullptr, out, N);
        __syncthreads();  // the LDS stages are taken again by the next unit
    }
}

using Tile256 = Tile<256, 256, 2, 4, 2>;
using Tile128 = Tile<128, 256, 2, 4, 3>;
using Tile128n = Tile<128, 128, 2, 4, 4>;
using Tile64 = Tile<64, 64, 2, 2, 4>;  // two workgroups per CU, as the next
using Tile32 = Tile<32, 64, 2, 2, 6>;
constexpr int kCus = 256;

}  // namespace

namespace w4a8 {

template <typename C, typename T>
static hipError_t launch_tile(const int8_t *qa, const float *a_scale, int64_t M, int64_t K, const int8_t *qw,
                              const float *w_scale, int64_t N, const float *bias, T *out, int64_t ldo, hipStream_t stream) {
    const int64_t mt = (M + C::BM - 1) / C::BM, nt = (N + C::BN - 1) / C::BN;
    if (mt * nt * C::kThreads >= 1ll << 32) {
        // a launch has to have fewer than 2^32 threads: two calls, with the longer side halved
        const int64_t m = mt >= nt ? mt / 2 * C::BM : 0, n = mt >= nt ? 0 : nt / 2 * C::BN;
        const hipError_t err = launch_tile<C>(qa, a_scale, mt >= nt ? m : M, K, qw, w_scale, mt >= nt ? N : n, bias, out,
                                              ldo, stream);
        if (err != hipSuccess) return err;
        return launch_tile<C>(qa + m * K, a_scale + m, M - m, K, qw + n * K, w_scale + n, N - n,
                              bias ? bias + n : nullptr, out + m * ldo + n, ldo, stream);
    }
    hipLaunchKernelGGL((gemm_w8a8_tile_kernel<C, T>), dim3((uint32_t)(mt * nt)), dim3(C::kThreads), 0, stream, qa, a_scale,
                       M, K, qw, w_scale, N, bias, out, ldo);
    return hipGetLastError();
}

// How the few-row loop shares out k: waves, windows of each per pass, passes.  The fewest windows
// that no wave needs (they cost cache reads), then the most waves.
struct Slices {
    int waves, nw, passes;
};
static Slices slices_of(int64_t K, int max_waves, int max_nw) {
    const int64_t windows = (K + 127) / 128;
    const int passes = (int)((windows + max_waves * max_nw - 1) / (max_waves * max_nw));
    const int per = (int)((windows + passes - 1) / passes);
    Slices best{1, max_nw, passes};
    int waste = 1 << 30;
    // several passes have one form, of max_nw windows
    for (int nw = passes > 1 ? max_nw : 1; nw <= max_nw; ++nw) {
        const int waves = (per + nw - 1) / nw;
        if (waves <= max_waves && waves * nw - per < waste) {
            waste = waves * nw - per;
            best = Slices{waves, nw, passes};
        }
    }
    return best;
}

template <typename T>
static hipError_t launch_slice(const int8_t *qa, const float *a_scale, int64_t M, int64_t K, const int8_t *qw,
                               const float *w_scale, int64_t N, const float *bias, T *out, int64_t ldo, hipStream_t stream) {
    const Slices s = slices_of(K, kMaxSliceWaves, 4);
    const int64_t grid = std::min<int64_t>((N + 15) / 16, kCus * (kMaxSliceWaves / s.waves));
#define W4A8_SLICE(NN, ONE)                                                                                         \
    hipLaunchKernelGGL((gemm_w8a8_slice_kernel<NN, ONE, T>), dim3((uint32_t)grid), dim3(64 * s.waves), 0, stream, \
                       qa, a_scale, M, K, s.passes, qw, w_scale, N, bias, out, ldo)
    if (s.passes > 1) W4A8_SLICE(4, false);
    else if (s.nw == 1) W4A8_SLICE(1, true);
    else if (s.nw == 2) W4A8_SLICE(2, true);
    else if (s.nw == 3) W4A8_SLICE(3, true);
    else W4A8_SLICE(4, true);
#undef W4A8_SLICE
    return hipGetLastError();
}

template <typename T>
static hipError_t gemm_w8a8_typed(const int8_t *qa, const float *a_scale, int64_t M, int64_t K, const int8_t *qw,
                                  const float *w_scale, int64_t N, const float *bias, T *out, int64_t ldo,
                                  hipStream_t stream) {
    // Few rows and a long k, or runs of at least four 16-channel tiles for every workgroup: k shared
    // out within the workgroup.  us with weights from memory, this loop / 32 x 64 tiles, one row: K 8192,
    // N 28672 40.4 / 43.8; K 8192, N 16384 26.2 / 29.6; K 16384, N 4096 19.1 / 24.6; on the tiles' side
    // K 8192, N 8192 17.2 / 16.3 and K 4096, N 14336 17.3 / 15.0.  The border follows N and K one at a
    // time and is not the best everywhere: N from 16384 on with K up to 2048 would be faster on tiles (K
    // 2048, N 28672 19.3 / 12.9), K 7168 and 8192 with N up to 4096 here (K 8192, N 4096 11.3 / 14.5),
    // and 16 rows of K 16384 from N 6144 on, in two passes, on tiles (N 28672 108 / 86.9).
    if (M <= 16 && (K > 8192 || N >= 16 * 4 * kCus))
        return launch_slice(qa, a_scale, M, K, qw, w_scale, N, bias, out, ldo, stream);
    // Else the tile form of the least expected time.  Per 256 tiles (one for every CU) and K 8192 the
    // forms take about 100 us (256 x 256), 60 (128 x 256), 39 (128 x 128), 15.5 (64 x 64, and 5 once) and
    // 10.7 (32 x 64, and 8 once), part rounds as whole ones: large tiles read less per product, small
    // ones leave fewer CUs idle.  Over 141 sizes of M 17-4096, K 512-8192, N 2048-28672 the form of this
    // rule is within 9% of the fastest one (at short K too, where the constants do not scale with it).
    // us against the other forms: M 512, K = N 8192 128 x 128 43 (128 x 256 60, 64 x 64 71); M 77, K 4112,
    // N 5003 32 x 64 12.5 (64 x 64 13.0, 128 x 128 30); M 256, K 8192, N 28672 128 x 256 76 (128 x 128 90,
    // 256 x 256 110); the widest miss M 192, K = N 8192 64 x 64 39 (128 x 128 36).
    auto cost = [&](int64_t bm, int64_t bn, double round, double once) {
        const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
        return (double)((tiles + kCus - 1) / kCus) * round + once;
    };
    const double c256 = cost(256, 256, 100.0, 0.0), c128 = cost(128, 256, 60.0, 0.0), c128n = cost(128, 128, 39.0, 0.0);
    const double c64 = cost(64, 64, 15.5, 5.0), c32 = cost(32, 64, 10.7, 8.0);
    const double least = std::min({c256, c128, c128n, c64, c32});
#define W4A8_TILE(C) launch_tile<C>(qa, a_scale, M, K, qw, w_scale, N, bias, out, ldo, stream)
    if (c256 == least) return W4A8_TILE(Tile256);
    if (c128 == least) return W4A8_TILE(Tile128);
    if (c128n == least) return W4A8_TILE(Tile128n);
    if (c64 == least) return W4A8_TILE(Tile64);
    return W4A8_TILE(Tile32);
#undef W4A8_TILE
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

template <typename C>
static hipError_t launch_grouped_tile(const int8_t *qa, const float *a_scale, int64_t R, const int32_t *row_index,
                                      const int32_t *offsets, int32_t E, int64_t K, const int8_t *qw,
                                      const float *w_scale, int64_t N, int64_t max_slots, int lo, float *out,
                                      hipStream_t stream) {
    // the most units there can be: every expert of the class has more than lo slots
    const int64_t blocks = std::min<int64_t>((int64_t)E, max_slots / (lo + 1)) + max_slots / C::BM;
    const int64_t units = blocks * ((N + C::BN - 1) / C::BN);
    const int64_t grid = std::min<int64_t>((units + 7) / 8 * 8, kCus);
    hipLaunchKernelGGL((grouped_w8a8_tile_kernel<C>), dim3((uint32_t)grid), dim3(C::kThreads), 0, stream, qa, a_scale, R,
                       row_index, offsets, E, K, qw, w_scale, N, max_slots, lo, out);
    return hipGetLastError();
}

hipError_t launch_grouped_gemm_w8a8(const int8_t *qa, const float *a_scale, int64_t R, const int32_t *row_index,
                                    const int32_t *expert_offsets, int32_t E, int64_t K, const int8_t *qw,
                                    const float *w_scale, int64_t N, int64_t max_slots, float *out,
                                    hipStream_t stream) {
    constexpr int kFewMax = 16;
    const Slices s = slices_of(K, kMaxSliceWaves, 4);
    const int64_t units = std::min<int64_t>(E, max_slots) * ((N + 15) / 16);
    const int64_t grid = std::min<int64_t>(units, kCus * (kMaxSliceWaves / s.waves));
#define W4A8_SLICE(NN, ONE)                                                                                       \
    hipLaunchKernelGGL((grouped_w8a8_slice_kernel<NN, ONE>), dim3((uint32_t)grid), dim3(64 * s.waves), 0, stream, \
                       qa, a_scale, R, row_index, expert_offsets, E, K, s.passes, qw, w_scale, N, max_slots, kFewMax, out)
    if (s.passes > 1) W4A8_SLICE(4, false);
    else if (s.nw == 1) W4A8_SLICE(1, true);
    else if (s.nw == 2) W4A8_SLICE(2, true);
    else if (s.nw == 3) W4A8_SLICE(3, true);
    else W4A8_SLICE(4, true);
#undef W4A8_SLICE
    hipError_t err = hipGetLastError();
    if (err == hipSuccess && max_slots > kFewMax)
        err = launch_grouped_tile<Tile128>(qa, a_scale, R, row_index, expert_offsets, E, K, qw, w_scale, N, max_slots,
                                           kFewMax, out, stream);
    return err;
}

}  // namespace w4a8
