// The tile kernel behind the dense products with more than a few rows, and its
// launch: see tile_gemm.h for the operands.
#pragma once

#include <type_traits>

#include "dense.h"
#include "tile_gemm.h"

namespace moe {
namespace tile {

struct TileArgs {
    // two products: summed over k, side by side in n (b alone has two), or two results
    Operand a, b;
    int64_t M, N, K;     // of one product
    void* out[2];
    int64_t ldo;
    void* gate;
    void* up;
    float* part;         // [splits][products][M][N] partial sums
    int splits;
    int m_tiles, n_tiles;
    int products;
};

enum { kGatedForward, kSumOfTwo, kTwoResults };


// Workgroup -> tile.  Workgroups go round the 8 XCDs by index; each XCD gets a
// consecutive run of tiles, and a run walks kBand tiles of m for one of n after
// the other, so that the tiles an XCD works on at a time share operand rows in
// its L2.
constexpr int kXcds = 8, kBand = 8;
__device__ inline void tile_of(int id, int m_tiles, int n_tiles, int* m, int* n) {
    const int total = m_tiles * n_tiles;
    const int per = total / kXcds, rest = total % kXcds, x = id % kXcds, i = id / kXcds;
    const int t = x * per + min(x, rest) + i;
    const int band = t / (kBand * n_tiles), in = t % (kBand * n_tiles);
    const int rows = min(kBand, m_tiles - band * kBand);
    *m = band * kBand + in % rows;
    *n = in / rows;
}

// (A lambda left as a call would need the arguments it refers to in memory.)
#define TILE_INLINE __attribute__((always_inline))

// WM x WN waves on a BM x BN tile.  kGatedForward: the tile's columns alternate
// 32 of gate and 32 of up, so that a wave holds both of an element.
// FAST: whole k steps are loaded straight into LDS, 16 bytes a lane (lines and
// chunks past the end read the last one; what they make is not stored); the
// last, partial step and everything else go through registers with zeros past
// the end.
// KW > 1: that many groups of WM x WN waves each take a run of the k steps, in
// LDS of their own, and their sums are added in the groups' order at the end.
template <int BM, int BN, int KW = 1> constexpr int tile_lds() { return 2 * (BM + BN) * 128 * KW; }
template <bool BF16, int BM, int BN, int WM, int WN, int ALAY, int BLAY, int MODE, bool FAST, int KW = 1>
__device__ TILE_INLINE void tile_body(const TileArgs& t, int tile, int part, char* lds) {
    typedef TileOf<BF16, BM, ALAY> TA;
    typedef TileOf<BF16, BN, BLAY> TB;
    constexpr int kThreads = WM * WN * 64;
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
    constexpr int BK = TA::BK, E = TA::E;
    constexpr int kStage = TA::kBytes + TB::kBytes;
    const int tid = KW == 1 ? threadIdx.x : threadIdx.x % kThreads;
    const int group = KW == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    lds += group * 2 * kStage;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    int tm, tn;
    tile_of(tile, t.m_tiles, t.n_tiles, &tm, &tn);
    const int64_t m0 = (int64_t)tm * BM;
    const int64_t n0 = (int64_t)tn * (MODE == kGatedForward ? BN / 2 : BN);
    const int which = MODE == kTwoResults ? part & 1 : 0;
    const int split = MODE == kTwoResults ? part >> 1 : part;

    // (the second matrix as a distance: a choice between two of the arguments would
    // be made in memory, on a copy of them all)
    const char *a0 = (const char*)uniform(t.a.p[0]), *b0 = (const char*)uniform(t.b.p[0]);
    const int64_t a_next = (const char*)uniform(t.a.p[1]) - a0, b_next = (const char*)uniform(t.b.p[1]) - b0;
    const int64_t lda = t.a.ld, ldb = t.b.ld;
    const int64_t steps1 = (t.K + BK - 1) / BK;
    const int64_t steps = MODE == kSumOfTwo ? 2 * steps1 : steps1;
    const int64_t part0 = steps * split / t.splits, part1 = steps * (split + 1) / t.splits;
    const int64_t rounds = (part1 - part0 + KW - 1) / KW;  // (the groups meet as often, also one with fewer steps)
    const int64_t s0 = min(part0 + rounds * group, part1), s1 = min(s0 + rounds, part1);

    constexpr int CA = TA::kChunks / kThreads, CB = TB::kChunks / kThreads;
    static_assert(TA::kChunks % kThreads == 0 && TB::kChunks % kThreads == 0, "whole chunks a thread");
    // Through registers: any alignment, zeros past the end.  Where every step
    // comes this way its chunks are loaded together (fetch_step), else (one step of
    // many, copy_step) one after the other, which keeps registers for the rest.
    auto chunk_a = [&](int p, int64_t k0, int i) TILE_INLINE {
        const int q = tid + kThreads * i, line = q / TA::kLineChunks, c = q % TA::kLineChunks;
        const void* a = a0 + (p ? a_next : 0);
        return ALAY == kAlongK ? load_chunk<BF16>(a, lda, m0 + line, k0 + c * E, t.M, t.K)
                               : load_chunk<BF16>(a, lda, k0 + line, m0 + c * E, t.K, t.M);
    };
    auto chunk_b = [&](int p, int64_t k0, int i) TILE_INLINE {
        const int q = tid + kThreads * i, line = q / TB::kLineChunks, c = q % TB::kLineChunks;
        const void* b = b0 + ((MODE == kGatedForward ? line >> 5 & 1 : p) ? b_next : 0);
        const int row = MODE == kGatedForward ? (line >> 6) * 32 + (line & 31) : line;
        return BLAY == kAlongK ? load_chunk<BF16>(b, ldb, n0 + row, k0 + c * E, t.N, t.K)
                               : load_chunk<BF16>(b, ldb, k0 + line, n0 + c * E, t.K, t.N);
    };
    auto place_a = [&](char* l, int i, u32x4 v) TILE_INLINE {
        const int q = tid + kThreads * i;
        *(u32x4*)(l + TA::chunk_at(q / TA::kLineChunks, q % TA::kLineChunks)) = v;
    };
    auto place_b = [&](char* l, int i, u32x4 v) TILE_INLINE {
        const int q = tid + kThreads * i;
        *(u32x4*)(l + TA::kBytes + TB::chunk_at(q / TB::kLineChunks, q % TB::kLineChunks)) = v;
    };
    auto copy_step = [&](int p, int64_t k0, char* l) TILE_INLINE {
#pragma unroll 1
        for (int i = 0; i < CA; i++) place_a(l, i, chunk_a(p, k0, i));
#pragma unroll 1
            for (int i = 0; i < CB; i++) place_b(l, i, chunk_b(p, k0, i));
    };
    // Forward, a step is fetched one ahead of being placed, so that the loads run
    // beside the products (us, fp32 2896 tokens 1926 x 489 124, without 139; bf16
    // 4096 tokens 1999 x 4001 167 and 176).  The backward pass, whose operands
    // across k take more registers, has none left for it (702 and 568).
    constexpr bool kAhead = !FAST && MODE == kGatedForward;
    u32x4 ra[FAST ? 1 : CA], rb[FAST ? 1 : CB];
    auto fetch_step = [&](int64_t s) TILE_INLINE {
        const int p = MODE == kSumOfTwo ? s >= steps1 : which;
        const int64_t k0 = (MODE == kSumOfTwo && s >= steps1 ? s - steps1 : s) * BK;
#pragma unroll
        for (int i = 0; i < CA; i++) ra[i] = chunk_a(p, k0, i);
#pragma unroll
            for (int i = 0; i < CB; i++) rb[i] = chunk_b(p, k0, i);
    };
    auto place_step = [&](char* l) TILE_INLINE {
#pragma unroll
        for (int i = 0; i < CA; i++) place_a(l, i, ra[i]);
#pragma unroll
            for (int i = 0; i < CB; i++) place_b(l, i, rb[i]);
    };
    // Straight into LDS: this thread's byte offsets from the tile's first
    // element of a step.
    constexpr int kBytes = 16 / E;
    uint32_t oa[FAST ? CA : 1], ob[FAST ? CB : 1];
    if constexpr (FAST) {
        // the chunk of a line that lands in LDS position c
        auto source = [&](auto tile, int line, int c) TILE_INLINE {
            typedef decltype(tile) TT;
            return ((TT::chunk_at(line, c) >> 4) - line * TT::kLineChunks);
        };
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int q = tid + kThreads * i, line = q / TA::kLineChunks;
            const int c = source(TA{}, line, q % TA::kLineChunks);
            if (ALAY == kAlongK) oa[i] = (uint32_t)((min(m0 + line, t.M - 1) - m0) * lda + c * E) * kBytes;
            else oa[i] = (uint32_t)(line * lda + (min(m0 + c * E, (t.M - 1) / E * E) - m0)) * kBytes;
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int q = tid + kThreads * i, line = q / TB::kLineChunks;
            const int c = source(TB{}, line, q % TB::kLineChunks);
            const int row = MODE == kGatedForward ? (line >> 6) * 32 + (line & 31) : line;
            if (BLAY == kAlongK) ob[i] = (uint32_t)((min(n0 + row, t.N - 1) - n0) * ldb + c * E) * kBytes;
            else ob[i] = (uint32_t)(line * ldb + (min(n0 + c * E, (t.N - 1) / E * E) - n0)) * kBytes;
        }
    }
    auto load_step = [&](int64_t s, char* l) TILE_INLINE {
        const int p = MODE == kSumOfTwo ? s >= steps1 : which;
        const int64_t k0 = (MODE == kSumOfTwo && s >= steps1 ? s - steps1 : s) * BK;
        if (k0 + BK > t.K) {
            copy_step(p, k0, l);
            return;
        }
        const uint32_t to = lds_address(l) + wave * 1024;
        const char* a = a0 + (p ? a_next : 0) + (ALAY == kAlongK ? m0 * lda + k0 : k0 * lda + m0) * kBytes;
#pragma unroll
        for (int i = 0; i < CA; i++) load_lds16(to + i * kThreads * 16, oa[i], a);
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int bp = MODE == kGatedForward ? ((wave * 64 + kThreads * i) / TB::kLineChunks) >> 5 & 1 : p;
            const char* b = b0 + (bp ? b_next : 0) + (BLAY == kAlongK ? n0 * ldb + k0 : k0 * ldb + n0) * kBytes;
            load_lds16(to + TA::kBytes + i * kThreads * 16, ob[i], b);
        }
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.f;

    // Products steps of 16 columns, operands read one ahead.  The last of a k step
    // comes after the barrier: by then every operand of the step is in registers
    // and the next step has landed, so its first operands are read, and the loads
    // of the step after it start, while these products run.
    constexpr int kSteps = TA::kSteps;
    Fragment<BF16> fa[2][FM], fb[2][FN];
    auto read = [&](const char* l, int kk) TILE_INLINE {
#pragma unroll
        for (int j = 0; j < FN; j++) TB::frag(l + TA::kBytes, wn + 32 * j, kk, lane, fb[kk & 1][j]);
#pragma unroll
        for (int i = 0; i < FM; i++) TA::frag(l, wm + 32 * i, kk, lane, fa[kk & 1][i]);
    };
    constexpr int kReads = FM * TA::kReads + FN * TB::kReads, kProducts = FM * FN * (BF16 ? 1 : 6);
    auto multiply = [&](int kk) TILE_INLINE {
#pragma unroll
        for (int j = 0; j < FN; j++) fb[kk & 1][j].split();
#pragma unroll
        for (int i = 0; i < FM; i++) fa[kk & 1][i].split();
#pragma unroll
        for (int i = 0; i < FM; i++)
#pragma unroll
            for (int j = 0; j < FN; j++) mma(acc[i][j], fb[kk & 1][j], fa[kk & 1][i]);
        if constexpr (BF16) spread_reads<kReads, kProducts>();
    };
    if (rounds > 0) {
        const bool any = KW == 1 || s0 < s1;
        if (any) {
            if constexpr (FAST) load_step(s0, lds);
            else {
                fetch_step(s0);
                place_step(lds);
            }
        }
        wait_loads_and_meet();
        if (s0 + 1 < s1) {
            if constexpr (FAST) load_step(s0 + 1, lds + kStage);
            else fetch_step(s0 + 1);
            if constexpr (!FAST && !kAhead) place_step(lds + kStage);
        }
        if (any) read(lds, 0);
    }
    for (int64_t s = s0; s < s0 + rounds; s++) {
        char* cur = lds + ((s - s0) & 1) * kStage;
        char* next = lds + ((s - s0 + 1) & 1) * kStage;
        const bool any = KW == 1 || s < s1;
        if (any) {
#pragma unroll
            for (int kk = 0; kk < kSteps - 1; kk++) {
                read(cur, kk + 1);
                multiply(kk);
            }
        }
        if constexpr (kAhead)
            if (s + 1 < s1) place_step(next);
        wait_loads_and_meet();
        if (s + 2 < s1) {
            if constexpr (FAST) load_step(s + 2, cur);
            else fetch_step(s + 2);
            if constexpr (!FAST && !kAhead) place_step(cur);
        }
        if (any) {
            read(next, 0);  // (after the last step what lies there, not used)
            multiply(kSteps - 1);
        }
    }
    wait_loads_and_meet();
    if constexpr (KW > 1) {
        static_assert(BM * BN * 4 <= 2 * kStage, "a group's sums fit");
        constexpr int kGroupSums = 2 * kStage / 4;
        float* sums = (float*)lds + wave * (FM * FN * 16 * 64) + lane;
        if (group) {
#pragma unroll
            for (int i = 0; i < FM * FN * 16; i++) sums[i * 64] = acc[i / 16 / FN][i / 16 % FN][i % 16];
        }
        __syncthreads();
        if (group) return;
#pragma unroll
        for (int g = 1; g < KW; g++)
#pragma unroll
            for (int i = 0; i < FM * FN * 16; i++) acc[i / 16 / FN][i / 16 % FN][i % 16] += sums[g * kGroupSums + i * 64];
    }

    // Results through a piece of LDS of the wave's own, 32 rows at a time, so
    // that they leave in rows of 16 bytes a lane.
    constexpr int kOut = MODE == kGatedForward ? FN * 16 : FN * 32;  // columns of a wave's rows
    auto store_rows = [&](int i, void* out, int64_t ldo, auto value, auto elem) TILE_INLINE {
        typedef decltype(elem) O;
        constexpr int OE = 16 / sizeof(O), kPitch = kOut * sizeof(O) + 16;
        char* w = lds + wave * (32 * kPitch);
        static_assert(WM * WN * 32 * kPitch <= 2 * kStage, "the waves' pieces fit");
#pragma unroll
        for (int j = 0; j < kOut / 32; j++)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                typedef O O4 __attribute__((ext_vector_type(4)));
                O4 v;
#pragma unroll
                for (int q = 0; q < 4; q++) v[q] = (O)value(j, e + q);
                *(O4*)(w + (lane & 31) * kPitch + (32 * j + acc_col(lane, e)) * sizeof(O)) = v;
            }
        constexpr int kPerRow = kOut / OE;
#pragma unroll
        for (int v = 0; v < 32 * kPerRow / 64; v++) {
            const int r = (v * 64 + lane) / kPerRow, c = (v * 64 + lane) % kPerRow * OE;
            const u32x4 d = *(const u32x4*)(w + r * kPitch + c * sizeof(O));
            const int64_t m = m0 + wm + 32 * i + r, n = n0 + (MODE == kGatedForward ? wn / 2 : wn) + c;
            if (m >= t.M || n >= t.N) continue;
            O* o = (O*)out + m * ldo + n;
            if (n + OE <= t.N) {
                ((Loose*)o)->v = d;
            } else {
                O x[OE];
                __builtin_memcpy(x, &d, 16);
#pragma unroll
                for (int q = 0; q < OE; q++)
                    if (n + q < t.N) o[q] = x[q];
            }
        }
    };
    typedef typename Elem<BF16>::type T;
    char* out = (char*)uniform(t.out[0]);
    if (which) out += (char*)uniform(t.out[1]) - out;
#pragma unroll
    for (int i = 0; i < FM; i++) {
        if constexpr (MODE == kGatedForward) {
            store_rows(i, t.out[0], t.ldo, [&](int j, int e) {
                const float g = acc[i][2 * j][e];
                return (BF16 ? silu_fast(g) : silu(g)) * acc[i][2 * j + 1][e];
            }, T{});
            if (t.gate) store_rows(i, t.gate, t.ldo, [&](int j, int e) { return acc[i][2 * j][e]; }, T{});
            if (t.up) store_rows(i, t.up, t.ldo, [&](int j, int e) { return acc[i][2 * j + 1][e]; }, T{});
        } else if (t.splits > 1) {
            float* part = t.part + (int64_t)(split * t.products + which) * t.M * t.N;
            store_rows(i, part, t.N, [&](int j, int e) { return acc[i][j][e]; }, float{});
        } else {
            store_rows(i, out, t.ldo, [&](int j, int e) { return acc[i][j][e]; }, T{});
        }
    }
}

template <bool BF16, int BM, int BN, int WM, int WN, int ALAY, int BLAY, int MODE, bool FAST, int KW>
__global__ __launch_bounds__(WM * WN * KW * 64) void tile_kernel(TileArgs t) {
    __shared__ __attribute__((aligned(1024))) char lds[tile_lds<BM, BN, KW>()];
    tile_body<BF16, BM, BN, WM, WN, ALAY, BLAY, MODE, FAST, KW>(t, blockIdx.x, 0, lds);
}

// Whether whole steps may be loaded 16 bytes a lane: aligned lines, and offsets
// within a tile's step that 32 bits hold.
// `length`: of its lines across k (kAcrossK).
inline bool fast_operand(const Operand& o, int layout, int64_t length, bool two, int bf16) {
    const int e = bf16 ? 8 : 4, bytes = bf16 ? 2 : 4;
    if ((uintptr_t)o.p[0] % 16 || (two && (uintptr_t)o.p[1] % 16) || o.ld % e) return false;
    if (layout == kAcrossK && length % e && !o.padded) return false;
    return o.ld <= ((int64_t)1 << 31) / 256 / bytes;
}

template <bool BF16, int BM, int BN, int WM, int WN, int ALAY, int BLAY, int MODE, int KW = 1>
hipError_t launch_shape(TileArgs t, hipStream_t s) {
    constexpr int cols = MODE == kGatedForward ? BN / 2 : BN;
    t.m_tiles = (int)((t.M + BM - 1) / BM);
    t.n_tiles = (int)((t.N + cols - 1) / cols);
    const bool fast = fast_operand(t.a, ALAY, t.M, false, BF16) &&
                      fast_operand(t.b, BLAY, t.N, MODE == kGatedForward, BF16);
    const dim3 grid((unsigned)(t.m_tiles * t.n_tiles)), block(WM * WN * KW * 64);
    if (fast) hipLaunchKernelGGL((tile_kernel<BF16, BM, BN, WM, WN, ALAY, BLAY, MODE, true, KW>), grid, block, 0, s, t);
    else hipLaunchKernelGGL((tile_kernel<BF16, BM, BN, WM, WN, ALAY, BLAY, MODE, false, KW>), grid, block, 0, s, t);
    return hipGetLastError();
}

// Tile shape for a product of M x N with `steps` k steps, by estimated time:
// rounds of workgroups over the CUs, times the steps, times the measured time of
// a step (us, with one workgroup on every CU, and with as many as a CU holds;
// in between by the number there):
//                   bf16         4-bit B      fp32
//   256 x 256       1.7          2.2          -           one a CU (fp32: spills, 5.1)
//   256 x 128       1.2          1.35         3.3         one
//   128 x 128       0.65 - 1.2   1.06 - 1.5   1.5 - 3.2   two
//   64 x 64         0.4 - 1.4    -            0.95 - 3.6  four (4-bit: never the fastest)
//   64 x 64 x 4     0.9          1.3          2.0         one; four steps at a time, and
//                                                         2 us to add the four sums
// The last is for few tiles of many steps, which wait for loads one step after
// the other: fp32 100 tokens 4096 x 512 59 us (64 x 64 107), 4-bit gated 106
// tokens 3360 x 2208 18 (128 x 128 49); but bf16 1000 tokens 1024 x 1024 15 (11.5).
// (The backward pass also splits k into parts over workgroups: they write and
// read partial sums in fp32, 4 MB a us, and cost a launch more, 4 us.)
enum { kShape256, kShape256x128, kShape128, kShapeSmall, kShapeParts, kShapes };
enum { kBf16, kQuant4, kFp32 };
struct TileShape { int bm, bn, per_cu, parts; float one, full; };
constexpr int kTileCus = 256;
static const TileShape kTileShapes[3][kShapes] = {
    {{256, 256, 1, 1, 1.7f, 1.7f}, {256, 128, 1, 1, 1.2f, 1.2f}, {128, 128, 2, 1, 0.65f, 1.2f}, {64, 64, 4, 1, 0.4f, 1.4f}, {64, 64, 1, 4, 0.9f, 0.9f}},
    {{256, 256, 1, 1, 2.2f, 2.2f}, {256, 128, 1, 1, 1.35f, 1.35f}, {128, 128, 2, 1, 1.06f, 1.5f}, {64, 64, 0, 1, 0.f, 0.f}, {64, 64, 1, 4, 1.3f, 1.3f}},
    {{256, 256, 0, 1, 0.f, 0.f}, {256, 128, 1, 1, 3.3f, 3.3f}, {128, 128, 2, 1, 1.5f, 3.2f}, {64, 64, 4, 1, 0.95f, 3.6f}, {64, 64, 1, 4, 2.0f, 2.0f}}};
// `but`: a shape that is not compiled for the caller, because it is never the fastest.
inline int plan_tiles(int kind, int64_t M, int64_t N, int64_t steps, int but, float* estimate) {
    int best = kShape128;
    float best_us = 1e30f;
    for (int h = 0; h < kShapes; h++) {
        const TileShape& c = kTileShapes[kind][h];
        if (!c.per_cu || h == but) continue;
        const int64_t groups = (M + c.bm - 1) / c.bm * ((N + c.bn - 1) / c.bn);
        const int64_t on_cu = (groups + kTileCus - 1) / kTileCus, rounds = (on_cu + c.per_cu - 1) / c.per_cu;
        const float step = rounds > 1 || c.per_cu == 1 ? c.full : c.one + (c.full - c.one) * (float)(on_cu - 1) / (float)(c.per_cu - 1);
        const float us = (float)rounds * ((float)((steps + c.parts - 1) / c.parts) * step + (c.parts > 1 ? 2.f : 0.f));
        if (us < best_us) {
            best = h;
            best_us = us;
        }
    }
    *estimate = best_us;
    return best;
}

inline DensePlan tiles_plan(int kind, int shape, bool gated) {
    const TileShape& c = kTileShapes[kind][shape];
    return {MOE_PLAN_TILES, c.bm, gated ? c.bn / 2 : c.bn, c.parts, 1, 1, shape};
}

template <bool BF16, int ALAY, int BLAY, int MODE>
hipError_t launch_tiles(TileArgs t, int shape, hipStream_t s) {
    t.products = t.splits = 1;
    switch (shape) {
        case kShape256:
            if constexpr (BF16) return launch_shape<BF16, 256, 256, 2, 4, ALAY, BLAY, MODE>(t, s);
            else return hipErrorInvalidValue;
        case kShape256x128:  // (fp32: two of 128 x 128 on a CU take 3.2 us a step, one of these 3.3)
            if constexpr (BF16) return launch_shape<BF16, 256, 128, 4, 2, ALAY, BLAY, MODE>(t, s);
            else return hipErrorInvalidValue;
        case kShapeSmall:  // (gate and up of an element in one wave)
            if constexpr (MODE == kGatedForward) return launch_shape<BF16, 64, 64, 2, 1, ALAY, BLAY, MODE>(t, s);
            else return launch_shape<BF16, 64, 64, 2, 2, ALAY, BLAY, MODE>(t, s);
        case kShapeParts: return launch_shape<BF16, 64, 64, 2, 1, ALAY, BLAY, MODE, 4>(t, s);
        default: return launch_shape<BF16, 128, 128, 2, 2, ALAY, BLAY, MODE>(t, s);
    }
}

}  // namespace tile
}  // namespace moe
