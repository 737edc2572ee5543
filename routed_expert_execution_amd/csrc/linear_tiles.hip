// Many tokens against 4-bit weights: bf16 in, bf16 out, tiles on the matrix cores.
//
//   y[t, n] = sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) x[t, k]
//
// Codes less their zero points are whole numbers of 8 bits at most, exact in
// bf16: the matrix cores sum (q - z) x over a group, or the 64 columns of a step
// where the group is longer, and the vector unit adds s times that to the result
// in fp32.  No weight is rounded.  (Weights s (q - z) rounded to bf16 on the way
// into LDS need no such addition: 2048 tokens 4096 x 4096 took 83 us, this way 84,
// with groups of 32, two additions a step, 103; gated, 1000 tokens 5504 x 2048, 61,
// 71 and 90.  But the result's error against 64 bits grew from its own rounding's
// 0.0017 to 0.0024, gated 0.0029, and a token's with the number of tokens beside
// it.)  Bound by the three units in turn between a step's barriers: of 4800 cycles
// a step (256 x 256) the products are 2050, LDS 2050, the vector unit 2200 on
// unpacking and additions.
#include "quant_codes.h"
#include "tile_kernel.h"

namespace moe {
namespace tile {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct QuantTileArgs {
    Operand x;
    int64_t M;
    int N, K;        // of one matrix
    void* out;
    int64_t ldo;
    QuantView q[2];
    int per_tile, row_groups, col_tiles;  // scales a row has in a tile of 128 columns
    int m_tiles, n_tiles;
};

// WM x WN waves on a BM x BN tile, and KW groups of them along k as in tile_body,
// x the A operand.  Gated, the tile's columns alternate 32 of gate and 32 of up, so
// that a wave holds both of an element.  The packed words of a step go to registers
// two steps ahead and become q - z in LDS one step ahead, each once for all rows of
// x; half of the waves do that before the step's products and half after, so that
// of two waves of a SIMD one unpacks while the other multiplies.  Scales come
// straight from memory a step ahead: a result register holds one column of the
// weights for all of its rows of x, so a lane needs FN of them (two each with
// GROUP32).  Blocks of 16 x 16 results, not 32 x 32, because the sums of a group on
// their way to the result then take 16 registers in place of 32, with which 256 x
// 256 tiles fit (1000 tokens gated 71 us, 256 x 128 84).
template <int BM, int BN, int WM, int WN, bool GATED, bool GROUP32, bool FAST, int KW>
__global__ __launch_bounds__(WM * WN * KW * 64, 2) void quant_tile_kernel(QuantTileArgs t) {
    typedef TileOf<true, BM, kAlongK> TA;
    typedef TileOf<true, BN, kAlongK> TB;
    constexpr int kThreads = WM * WN * 64;
    constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // a wave's blocks of 16 x 16 results
    constexpr int BK = TA::BK, E = TA::E;
    constexpr int kStage = TA::kBytes + TB::kBytes;
    constexpr int S = GROUP32 ? 2 : 1;  // groups of a step
    __shared__ __attribute__((aligned(1024))) char shared[tile_lds<BM, BN, KW>()];
    const int tid = KW == 1 ? threadIdx.x : threadIdx.x % kThreads;
    const int group = KW == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    // (both buffers of an operand side by side, so that one address and constant
    // offsets reach all of it)
    char* lds = shared + group * 2 * kStage;
    char *lds_x = lds, *lds_w = lds + 2 * TA::kBytes;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    int tm, tn;
    tile_of(blockIdx.x, t.m_tiles, t.n_tiles, &tm, &tn);
    const int64_t m0 = (int64_t)tm * BM;
    const int n0 = tn * (GATED ? BN / 2 : BN);

    typedef typename std::conditional<FAST, uint32_t, int64_t>::type Offset;
    const Offset ldx = (Offset)t.x.ld;
    const char* x0 = (const char*)t.x.p[0] + m0 * t.x.ld * 2;
    const int steps = (t.K + BK - 1) / BK;
    const int rounds = (steps + KW - 1) / KW;  // (the groups meet as often, also one with fewer steps)
    const int s0 = min(rounds * group, steps), s1 = min(s0 + rounds, steps);

    // x: straight into LDS if its rows are 16-byte aligned, else through registers
    // a step ahead.  A thread's chunks are one column of lines kThreads / 8 apart.
    // Lines past the last row read the last one, and what they make is not stored;
    // columns past the end, of which only groups of 32 can leave a half step, read
    // the row's last ones, which meet a scale of zero.
    constexpr int CA = TA::kChunks / kThreads;
    static_assert(TA::kChunks % kThreads == 0 && kThreads / 8 % 16 == 0, "whole chunks a thread, all of one column");
    const int line0 = tid / 8, last_line = (int)min(t.M - 1 - m0, (int64_t)BM - 1);
    const int column = FAST ? ((TA::chunk_at(line0, tid % 8) >> 4) - line0 * 8) * E : tid % 8 * E;
    auto source = [&](int s, int i) TILE_INLINE {  // element of the tile's first row
        return (Offset)min(line0 + kThreads / 8 * i, last_line) * ldx + (Offset)min(s * BK + column, t.K - E);
    };
    u32x4 ahead[FAST ? 1 : CA];
    auto fetch_x = [&](int s) TILE_INLINE {
#pragma unroll
        for (int i = 0; i < CA; i++) ahead[i] = ((const Loose*)(x0 + source(s, i) * 2))->v;
    };
    auto place_x = [&](int p) TILE_INLINE {
#pragma unroll
        for (int i = 0; i < CA; i++) *(u32x4*)(lds_x + p * TA::kBytes + TA::chunk_at(line0 + kThreads / 8 * i, tid % 8)) = ahead[i];
    };
    auto load_x = [&](int s, int p) TILE_INLINE {  // (offsets of 32 bits: fast_operand)
        const uint32_t to = lds_address(lds_x) + p * TA::kBytes + wave * 1024;
#pragma unroll
        for (int i = 0; i < CA; i++) load_lds16(to + i * kThreads * 16, (uint32_t)source(s, i) * 2u, x0);
    };

    // Packed words of a step: CQ places of (row group, lane), two words each.
    constexpr int CQ = BN / 16 * 64 / kThreads;
    static_assert(CQ * kThreads == BN * 4, "whole places a thread");
    struct Words {
        u32x2 code[CQ];
        uint8_t zero[CQ][S];
    };
    // Addresses are a wave's own part in scalar registers and a lane's offset in
    // 32 bits: row group r of the tile and step s as a packed tile's number (gated,
    // two row groups of gate and two of up alternate), and the place of group j of
    // the step among the scales (or zero points) of that tile.
    typedef __attribute__((address_space(1))) const char Bytes;
    auto packed_tile = [&](int r, int s) TILE_INLINE {
        const int row_group = (n0 >> 4) + (GATED ? (r >> 2) * 2 + (r & 1) : r);
        return (int64_t)min(row_group, t.row_groups - 1) * t.col_tiles + (s >> 1);
    };
    auto group_at = [&](int64_t p, int s, int j) TILE_INLINE { return p * 16 * t.per_tile + ((2 * (s & 1) + j) * t.per_tile >> 2); };
    const uint32_t code_lane = lane * 16, scale_lane = (lane & 15) * t.per_tile;
    auto load_words = [&](int s, Words& w) TILE_INLINE {
#pragma unroll
        for (int i = 0; i < CQ; i++) {
            const int r = wave + WM * WN * i;
            const QuantView& v = t.q[GATED ? r >> 1 & 1 : 0];
            const int64_t p = packed_tile(r, s);
            w.code[i] = *(__attribute__((address_space(1))) const u32x2*)((Bytes*)v.codes + p * 1024 + (s & 1) * 8 + code_lane);
#pragma unroll
            for (int j = 0; j < S; j++) w.zero[i][j] = v.zeros ? *((Bytes*)v.zeros + group_at(p, s, j) + scale_lane) : 8;
        }
    };
    auto store_words = [&](const Words& w, int p) TILE_INLINE {
#pragma unroll
        for (int i = 0; i < CQ; i++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                *(bf16x8*)(lds_w + p * TB::kBytes + TB::chunk_at(16 * (wave + WM * WN * i) + (lane & 15), 4 * j + (lane >> 4))) =
                    codes_less_zero(j ? w.code[i].y : w.code[i].x, (float)w.zero[i][j % S]);
    };
    struct Scales { uint16_t s[FN][S]; };
    auto load_scales = [&](int s, Scales& v) TILE_INLINE {
#pragma unroll
        for (int j = 0; j < FN; j++) {
            const int r = (wn >> 4) + j;
            typedef __attribute__((address_space(1))) const uint16_t Global;
            Bytes* p = (Bytes*)(GATED && r >> 1 & 1 ? t.q[1] : t.q[0]).scales + group_at(packed_tile(r, s), s, 0) * 2;
#pragma unroll
            for (int i = 0; i < S; i++) v.s[j][i] = *(Global*)(p + i * 2 + scale_lane * 2);
        }
    };

    f32x4 out[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) out[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // A step's products go block by block of 16 x 16 results, rows of blocks one
    // after the other, and beside each the scaling of a block kLate before it.
    // Operands of x are read kAhead rows ahead.  The last kTail rows of a step come
    // after the barrier, when the next step has landed: beside them its first
    // operands are read, those of the weights each after its last use.  (The order
    // is pinned: left to itself the compiler holds as many sums and operands at
    // once as it can.)
    constexpr int kRing = FM == 4 ? 4 : 2, kAhead = kRing / 2, kTail = kAhead, kLate = 3;
    constexpr int kBlocks = FM * FN * S;
    bf16x8 a[kRing][2], b[FN][2];
    f32x4 acc[4];
    auto read = [&](const char* l, int r0, int k) TILE_INLINE {
        return *(const bf16x8*)(l + TA::chunk_at(r0 + (lane & 15), 4 * k + (lane >> 4)));
    };
    auto read_a = [&](int p, int i) TILE_INLINE {
#pragma unroll
        for (int k = 0; k < 2; k++) a[i % kRing][k] = read(lds_x + p * TA::kBytes, wm + 16 * i, k);
    };
    auto read_b = [&](int p, int j) TILE_INLINE {
#pragma unroll
        for (int k = 0; k < 2; k++) b[j][k] = read(lds_w + p * TB::kBytes, wn + 16 * j, k);
    };
    auto add = [&](int n, const Scales& v) TILE_INLINE {
        const int i = n / (FN * S), j = n / S % FN;
        const float s = f16_bits_to_f32(v.s[j][n % S]);
#pragma unroll
        for (int e = 0; e < 4; e++) out[i][j][e] = fmaf(s, acc[n % 4][e], out[i][j][e]);
        asm volatile("" : "+v"(out[i][j]));
    };
    // last: the operands of the weights are replaced, by those of buffer p
    auto multiply_row = [&](int i, bool last, int p, const Scales& v) TILE_INLINE {
#pragma unroll
        for (int j = 0; j < FN; j++) {
#pragma unroll
            for (int g = 0; g < S; g++) {
                const int n = (i * FN + j) * S + g;
                const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                acc[n % 4] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i % kRing][g], b[j][g], zero, 0, 0, 0);
                if constexpr (S == 1) acc[n % 4] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i % kRing][1], b[j][1], acc[n % 4], 0, 0, 0);
                if (n >= kLate) add(n - kLate, v);
            }
            if (last) read_b(p, j);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    Words words;
    Scales scales[2];
    if (s0 < s1) {
        if constexpr (FAST) load_x(s0, 0);
        else {
            fetch_x(s0);
            place_x(0);
        }
        load_words(s0, words);
        load_scales(s0, scales[0]);
        store_words(words, 0);
        if (s0 + 1 < s1) load_words(s0 + 1, words);
    }
    wait_loads_and_meet();
    if (s0 < s1) {
#pragma unroll
        for (int j = 0; j < FN; j++) read_b(0, j);
#pragma unroll
        for (int i = 0; i < kAhead; i++) read_a(0, i);
    }
    if (s0 + 1 < s1) {
        if constexpr (FAST) load_x(s0 + 1, 1);
        else fetch_x(s0 + 1);
    }
    const bool first = wave < WM * WN / 2;
    auto step = [&](auto parity, int s) TILE_INLINE {
        constexpr int p = decltype(parity)::value;
        auto unpack = [&]() TILE_INLINE {
            if (s + 1 < s1) {
                store_words(words, 1 - p);
                if (s + 2 < s1) load_words(s + 2, words);
            }
        };
        if (s + 1 < s1) load_scales(s + 1, scales[1 - p]);
        if (first) unpack();
        if (s < s1) {
#pragma unroll
            for (int i = 0; i < FM - kTail; i++) {
                read_a(p, i + kAhead);
                multiply_row(i, false, 0, scales[p]);
            }
        }
        if (!first) unpack();
        if constexpr (!FAST)
            if (s + 1 < s1) place_x(1 - p);
        wait_loads_and_meet();
        if (s + 2 < s1) {
            if constexpr (FAST) load_x(s + 2, p);
            else fetch_x(s + 2);
        }
        if (s < s1) {
            // (after the last step what lies there is read and not used)
#pragma unroll
            for (int i = 0; i < kTail; i++) {
                read_a(1 - p, i);
                multiply_row(FM - kTail + i, i == kTail - 1, 1 - p, scales[p]);
            }
#pragma unroll
            for (int n = kBlocks - kLate; n < kBlocks; n++) add(n, scales[p]);
        }
    };
    for (int s = s0; s < s0 + rounds; s += 2) {
        step(std::integral_constant<int, 0>{}, s);
        if (s + 1 < s0 + rounds) step(std::integral_constant<int, 1>{}, s + 1);
    }
    wait_loads_and_meet();
    if constexpr (KW > 1) {  // the groups' sums in the groups' order
        static_assert(BM * BN * 4 <= 2 * kStage, "a group's sums fit");
        constexpr int kGroupSums = 2 * kStage / 4;
        float* sums = (float*)lds + wave * (FM * FN * 4 * 64) + lane;
        if (group) {
#pragma unroll
            for (int i = 0; i < FM * FN * 4; i++) sums[i * 64] = out[i / 4 / FN][i / 4 % FN][i % 4];
        }
        __syncthreads();
        if (group) return;
#pragma unroll
        for (int g = 1; g < KW; g++)
#pragma unroll
            for (int i = 0; i < FM * FN * 4; i++) out[i / 4 / FN][i / 4 % FN][i % 4] += sums[g * kGroupSums + i * 64];
    }

    // Results through a piece of LDS of the wave's own, 16 rows at a time, so that
    // they leave in rows of 16 bytes a lane.  Register e of a block is row
    // 4 (lane / 16) + e and column lane % 16.
    constexpr int kOut = GATED ? FN * 8 : FN * 16, kPitch = kOut * 2 + 16, kPerRow = kOut / E;
    static_assert(WM * WN * 16 * kPitch <= 2 * kStage && 16 * kPerRow % 64 == 0, "the waves' pieces fit, in whole waves of chunks");
    char* w = lds + wave * (16 * kPitch);
#pragma unroll
    for (int i = 0; i < FM; i++) {
#pragma unroll
        for (int j = 0; j < kOut / 16; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int of = GATED ? (j >> 1) * 4 + (j & 1) : j;  // gated: its block of gate, up's two further
                const float y = GATED ? silu_fast(out[i][of][e]) * out[i][of + (GATED ? 2 : 0)][e] : out[i][of][e];
                *(__bf16*)(w + (4 * (lane >> 4) + e) * kPitch + (16 * j + (lane & 15)) * 2) = (__bf16)y;
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int v = 0; v < 16 * kPerRow / 64; v++) {
            const int r = (v * 64 + lane) / kPerRow, c = (v * 64 + lane) % kPerRow * E;
            const u32x4 d = *(const u32x4*)(w + r * kPitch + c * 2);
            const int64_t m = m0 + wm + 16 * i + r, n = n0 + (GATED ? wn / 2 : wn) + c;
            if (m >= t.M || n >= t.N) continue;
            uint16_t* o = (uint16_t*)t.out + m * t.ldo + n;
            if (n + E <= t.N) {
                ((Loose*)o)->v = d;
            } else {
                uint16_t h[E];
                __builtin_memcpy(h, &d, 16);
#pragma unroll
                for (int q = 0; q < E; q++)
                    if (n + q < t.N) o[q] = h[q];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <int BM, int BN, int WM, int WN, bool GATED, int KW = 1>
hipError_t launch_quant(QuantTileArgs t, hipStream_t s) {
    constexpr int cols = GATED ? BN / 2 : BN;
    t.m_tiles = (int)((t.M + BM - 1) / BM);
    t.n_tiles = (t.N + cols - 1) / cols;
    const bool fast = fast_operand(t.x, kAlongK, t.M, false, true);
    const dim3 grid((unsigned)(t.m_tiles * t.n_tiles)), block(WM * WN * KW * 64);
    if (t.per_tile == 4) {
        if constexpr (!GATED && KW > 1) return hipErrorInvalidValue;
        else if (fast) hipLaunchKernelGGL((quant_tile_kernel<BM, BN, WM, WN, GATED, true, true, KW>), grid, block, 0, s, t);
        else hipLaunchKernelGGL((quant_tile_kernel<BM, BN, WM, WN, GATED, true, false, KW>), grid, block, 0, s, t);
    } else {
        if (fast) hipLaunchKernelGGL((quant_tile_kernel<BM, BN, WM, WN, GATED, false, true, KW>), grid, block, 0, s, t);
        else hipLaunchKernelGGL((quant_tile_kernel<BM, BN, WM, WN, GATED, false, false, KW>), grid, block, 0, s, t);
    }
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_shape4(const QuantTileArgs& t, int shape, hipStream_t s) {
    switch (shape) {
        case kShape256: return launch_quant<256, 256, 2, 4, GATED>(t, s);
        case kShape256x128: return launch_quant<256, 128, 4, 2, GATED>(t, s);
        case kShapeParts: return launch_quant<64, 64, 2, 1, GATED, 4>(t, s);
        default: return launch_quant<128, 128, 2, 2, GATED>(t, s);
    }
}

}  // namespace
}  // namespace tile

DensePlan linear_tiles_plan(const LinearArgs& a, bool gated, float* us) {
    // (64 x 64 in four parts is the shape of the shared rows' workgroups: with groups
    // of 32, not gated, they are faster at every size)
    const int but = a.group == 32 && !gated ? tile::kShapeParts : tile::kShapes;
    const int shape = tile::plan_tiles(tile::kQuant4, a.T, (int64_t)a.rows * (gated ? 2 : 1), (a.cols + 63) / 64, but, us);
    if (a.group == 32) *us *= 1.25f;  // (two additions a step: 1.2 to 1.28 in every shape)
    return tile::tiles_plan(tile::kQuant4, shape, gated);
}

hipError_t launch_linear_tiles(const LinearArgs& a, bool gated, int shape, hipStream_t s) {
    tile::QuantTileArgs t{};
    t.x = tile::Operand{{a.x, nullptr}, a.ldx, 0};
    t.M = a.T;
    t.N = a.rows;
    t.K = a.cols;
    t.out = a.y;
    t.ldo = a.ldy;
    t.q[0] = a.w[0];
    t.q[1] = a.w[1];
    t.per_tile = 128 / a.group;
    t.row_groups = a.row_groups;
    t.col_tiles = a.col_tiles;
    return gated ? tile::launch_shape4<true>(t, shape, s) : tile::launch_shape4<false>(t, shape, s);
}

}  // namespace moe
