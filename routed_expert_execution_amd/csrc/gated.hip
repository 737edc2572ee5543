// The gated feed-forward block with bf16 or fp32 weights:
//   g = x Wg^T, u = x Wu^T, h = silu(g) u
// and its backward pass
//   dg = dh u s(g) (1 + g (1 - s(g))),  du = dh g s(g),  s the logistic function
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x.
#include <algorithm>

#include "dense.h"
#include "tile_gemm.h"

namespace moe {
namespace {

using namespace tile;

template <bool BF16> __device__ inline float load_elem(const void* p, int64_t i) {
    if (BF16) return bf16_bits_to_f32(((const uint16_t*)p)[i]);
    return ((const float*)p)[i];
}
template <bool BF16> __device__ inline void store_elem(void* p, int64_t i, float v) {
    if (BF16) ((__bf16*)p)[i] = (__bf16)v;
    else ((float*)p)[i] = v;
}

// ---- tiles ------------------------------------------------------------------

struct TileArgs {
    Operand a[2], b[2];  // two products: summed over k, side by side in n, or one after the other in z
    int64_t M, N;        // of one product's result
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

// WM x WN waves on a BM x BN tile.  kGatedForward: the tile's columns alternate
// 32 of gate and 32 of up, so that a wave holds both of an element.
// FAST: whole k steps are loaded straight into LDS, 16 bytes a lane (lines and
// chunks past the end read the last one; what they make is not stored); the
// last, partial step and everything else go through registers with zeros past
// the end.
template <bool BF16, int BM, int BN, int WM, int WN, int ALAY, int BLAY, int MODE, bool FAST>
__global__ __launch_bounds__(WM * WN * 64) void tile_kernel(TileArgs t) {
    typedef TileOf<BF16, BM, ALAY> TA;
    typedef TileOf<BF16, BN, BLAY> TB;
    constexpr int kThreads = WM * WN * 64;
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
    constexpr int BK = TA::BK, E = TA::E;
    constexpr int kStage = TA::kBytes + TB::kBytes;
    __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    int tm, tn;
    tile_of(blockIdx.x, t.m_tiles, t.n_tiles, &tm, &tn);
    const int64_t m0 = (int64_t)tm * BM;
    const int64_t n0 = (int64_t)tn * (MODE == kGatedForward ? BN / 2 : BN);
    const int which = MODE == kTwoResults ? blockIdx.y & 1 : 0;
    const int split = MODE == kTwoResults ? blockIdx.y >> 1 : blockIdx.y;

    const int64_t steps1 = (t.a[0].K + BK - 1) / BK;
    const int64_t steps = MODE == kSumOfTwo ? 2 * steps1 : steps1;
    const int64_t s0 = steps * split / t.splits, s1 = steps * (split + 1) / t.splits;

    constexpr int CA = TA::kChunks / kThreads, CB = TB::kChunks / kThreads;
    static_assert(TA::kChunks % kThreads == 0 && TB::kChunks % kThreads == 0, "whole chunks a thread");
    // Through registers: any alignment, zeros past the end.
    auto copy_step = [&](int p, int64_t k0, char* l) {
        const Operand a = t.a[p];
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int q = threadIdx.x + kThreads * i, line = q / TA::kLineChunks, c = q % TA::kLineChunks;
            *(u32x4*)(l + TA::chunk_at(line, c)) =
                ALAY == kAlongK ? load_chunk<BF16>(a.p, a.ld, m0 + line, k0 + c * E, a.R, a.K)
                                : load_chunk<BF16>(a.p, a.ld, k0 + line, m0 + c * E, a.K, a.R);
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int q = threadIdx.x + kThreads * i, line = q / TB::kLineChunks, c = q % TB::kLineChunks;
            u32x4 v;
            if (MODE == kGatedForward) {
                const Operand b = t.b[line >> 5 & 1];
                v = load_chunk<BF16>(b.p, b.ld, n0 + (line >> 6) * 32 + (line & 31), k0 + c * E, b.R, b.K);
            } else {
                const Operand b = t.b[p];
                v = BLAY == kAlongK ? load_chunk<BF16>(b.p, b.ld, n0 + line, k0 + c * E, b.R, b.K)
                                    : load_chunk<BF16>(b.p, b.ld, k0 + line, n0 + c * E, b.K, b.R);
            }
            *(u32x4*)(l + TA::kBytes + TB::chunk_at(line, c)) = v;
        }
    };
    // Straight into LDS: this thread's byte offsets from the tile's first
    // element of a step.
    constexpr int kBytes = 16 / E;
    uint32_t oa[FAST ? CA : 1], ob[FAST ? CB : 1];
    if constexpr (FAST) {
        // the chunk of a line that lands in LDS position c
        auto source = [&](auto tile, int line, int c) {
            typedef decltype(tile) TT;
            return ((TT::chunk_at(line, c) >> 4) - line * TT::kLineChunks);
        };
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int q = threadIdx.x + kThreads * i, line = q / TA::kLineChunks;
            const int c = source(TA{}, line, q % TA::kLineChunks);
            if (ALAY == kAlongK) oa[i] = (uint32_t)((min(m0 + line, t.M - 1) - m0) * t.a[0].ld + c * E) * kBytes;
            else oa[i] = (uint32_t)(line * t.a[0].ld + (min(m0 + c * E, (t.M - 1) / E * E) - m0)) * kBytes;
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int q = threadIdx.x + kThreads * i, line = q / TB::kLineChunks;
            const int c = source(TB{}, line, q % TB::kLineChunks);
            const int row = MODE == kGatedForward ? (line >> 6) * 32 + (line & 31) : line;
            if (BLAY == kAlongK) ob[i] = (uint32_t)((min(n0 + row, t.N - 1) - n0) * t.b[0].ld + c * E) * kBytes;
            else ob[i] = (uint32_t)(line * t.b[0].ld + (min(n0 + c * E, (t.N - 1) / E * E) - n0)) * kBytes;
        }
    }
    auto load_step = [&](int64_t s, char* l) {
        const int p = MODE == kSumOfTwo ? s >= steps1 : which;
        const int64_t k0 = (MODE == kSumOfTwo && s >= steps1 ? s - steps1 : s) * BK;
        if (!FAST || k0 + BK > t.a[0].K) {
            copy_step(p, k0, l);
            return;
        }
        const uint32_t to = lds_address(l) + wave * 1024;
        const char* a = (const char*)t.a[p].p + (ALAY == kAlongK ? m0 * t.a[0].ld + k0 : k0 * t.a[0].ld + m0) * kBytes;
#pragma unroll
        for (int i = 0; i < CA; i++) load_lds16(to + i * kThreads * 16, oa[i], a);
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int bp = MODE == kGatedForward ? ((wave * 64 + kThreads * i) / TB::kLineChunks) >> 5 & 1 : p;
            const char* b = (const char*)t.b[bp].p + (BLAY == kAlongK ? n0 * t.b[0].ld + k0 : k0 * t.b[0].ld + n0) * kBytes;
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

    if (s0 < s1) load_step(s0, lds);
    for (int64_t s = s0; s < s1; s++) {
        const char* cur = lds + ((s - s0) & 1) * kStage;
        wait_loads_and_meet();
        if (s + 1 < s1) load_step(s + 1, lds + ((s - s0 + 1) & 1) * kStage);
        typedef typename std::conditional<BF16, bf16x8, f32x4>::type Frag;
#pragma unroll
        for (int kk = 0; kk < 4; kk++) {
            Frag fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; i++) TA::frag(cur, wm + 32 * i, kk, lane, fa[i]);
#pragma unroll
            for (int j = 0; j < FN; j++) TB::frag(cur + TA::kBytes, wn + 32 * j, kk, lane, fb[j]);
#pragma unroll
            for (int i = 0; i < FM; i++)
#pragma unroll
                for (int j = 0; j < FN; j++) mma(acc[i][j], fa[i], fb[j]);
        }
    }
    wait_loads_and_meet();

    // Results through a piece of LDS of the wave's own, 32 rows at a time, so
    // that they leave in rows of 16 bytes a lane.
    constexpr int kOut = MODE == kGatedForward ? FN * 16 : FN * 32;  // columns of a wave's rows
    auto store_rows = [&](int i, void* out, int64_t ldo, auto value, auto elem) {
        typedef decltype(elem) O;
        constexpr int OE = 16 / sizeof(O), kPitch = kOut * sizeof(O) + 16;
        char* w = lds + wave * (32 * kPitch);
        static_assert(WM * WN * 32 * kPitch <= 2 * kStage, "the waves' pieces fit");
#pragma unroll
        for (int j = 0; j < kOut / 32; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) *(O*)(w + acc_row(lane, e) * kPitch + (32 * j + (lane & 31)) * sizeof(O)) = (O)value(j, e);
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
#pragma unroll
    for (int i = 0; i < FM; i++) {
        if constexpr (MODE == kGatedForward) {
            store_rows(i, t.out[0], t.ldo, [&](int j, int e) { return silu(acc[i][2 * j][e]) * acc[i][2 * j + 1][e]; }, T{});
            if (t.gate) store_rows(i, t.gate, t.ldo, [&](int j, int e) { return acc[i][2 * j][e]; }, T{});
            if (t.up) store_rows(i, t.up, t.ldo, [&](int j, int e) { return acc[i][2 * j + 1][e]; }, T{});
        } else if (t.splits > 1) {
            float* part = t.part + (int64_t)(split * t.products + which) * t.M * t.N;
            store_rows(i, part, t.N, [&](int j, int e) { return acc[i][j][e]; }, float{});
        } else {
            store_rows(i, t.out[which], t.ldo, [&](int j, int e) { return acc[i][j][e]; }, T{});
        }
    }
}

// Whether whole steps may be loaded 16 bytes a lane: aligned lines, and offsets
// within a tile's step that 32 bits hold.
bool fast_operand(const Operand& o, int layout, int bf16) {
    const int e = bf16 ? 8 : 4, bytes = bf16 ? 2 : 4;
    if ((uintptr_t)o.p % 16 || o.ld % e) return false;
    if (layout == kAcrossK && o.R % e && !o.padded) return false;
    return o.ld <= ((int64_t)1 << 31) / 256 / bytes;
}

template <bool BF16, int BM, int BN, int WM, int WN, int ALAY, int BLAY, int MODE>
hipError_t launch_tiles(TileArgs t, hipStream_t s) {
    constexpr int cols = MODE == kGatedForward ? BN / 2 : BN;
    t.m_tiles = (int)((t.M + BM - 1) / BM);
    t.n_tiles = (int)((t.N + cols - 1) / cols);
    t.products = MODE == kTwoResults ? 2 : 1;
    bool fast = fast_operand(t.a[0], ALAY, BF16) && fast_operand(t.b[0], BLAY, BF16);
    if (MODE != kTwoResults) fast = fast && fast_operand(t.b[1], BLAY, BF16);
    const dim3 grid((unsigned)(t.m_tiles * t.n_tiles), t.products * t.splits), block(WM * WN * 64);
    if (fast) hipLaunchKernelGGL((tile_kernel<BF16, BM, BN, WM, WN, ALAY, BLAY, MODE, true>), grid, block, 0, s, t);
    else hipLaunchKernelGGL((tile_kernel<BF16, BM, BN, WM, WN, ALAY, BLAY, MODE, false>), grid, block, 0, s, t);
    return hipGetLastError();
}

// Partial sums added in split order.
template <bool BF16>
__global__ __launch_bounds__(256) void reduce_kernel(const float* __restrict__ part, int splits, int64_t products,
                                                     int64_t n, void* out0, void* out1) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= products * n) return;
    float s = part[i];
    for (int k = 1; k < splits; k++) s += part[(int64_t)k * products * n + i];
    if (i < n) store_elem<BF16>(out0, i, s);
    else store_elem<BF16>(out1, i - n, s);
}

// dg and du into rows of whole 16-byte chunks (ld >= F), a chunk a thread.  In
// bf16 they are rounded once, as the products that follow take them.
template <bool BF16>
__global__ __launch_bounds__(256) void gate_backward_kernel(const void* __restrict__ dh, int64_t lddh,
                                                            const void* __restrict__ gate, const void* __restrict__ up,
                                                            int64_t T, int F, int64_t ld, void* __restrict__ dg,
                                                            void* __restrict__ du) {
    typedef typename Elem<BF16>::type E;
    constexpr int N = Elem<BF16>::kChunk;
    const int64_t per_row = ld / N, total = T * per_row;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / per_row, f = i % per_row * N;
        E d[N], g[N], u[N], a[N], b[N];
        const u32x4 vd = load_chunk<BF16>(dh, lddh, t, f, T, F), vg = load_chunk<BF16>(gate, F, t, f, T, F),
                    vu = load_chunk<BF16>(up, F, t, f, T, F);
        __builtin_memcpy(d, &vd, 16);
        __builtin_memcpy(g, &vg, 16);
        __builtin_memcpy(u, &vu, 16);
#pragma unroll
        for (int e = 0; e < N; e++) {
            const float gf = (float)g[e], s = 1.0f / (1.0f + expf(-gf)), df = (float)d[e];
            a[e] = (E)(df * (float)u[e] * s * (1.0f + gf * (1.0f - s)));
            b[e] = (E)(df * gf * s);
        }
        __builtin_memcpy((E*)dg + t * ld + f, a, 16);
        __builtin_memcpy((E*)du + t * ld + f, b, 16);
    }
}

template <bool BF16>
hipError_t gated(const GatedArgs& a, hipStream_t s) {
    TileArgs t{};
    t.a[0] = Operand{a.x, a.ldx, a.T, a.d, 0};
    t.b[0] = Operand{a.w_gate, a.d, a.F, a.d, 0};
    t.b[1] = Operand{a.w_up, a.d, a.F, a.d, 0};
    t.M = a.T;
    t.N = a.F;
    t.out[0] = a.h;
    t.ldo = a.F;
    t.gate = a.gate;
    t.up = a.up;
    t.splits = 1;
    if (a.T > 512) return launch_tiles<BF16, 256, 256, 2, 4, kAlongK, kAlongK, kGatedForward>(t, s);
    return launch_tiles<BF16, 128, 128, 2, 2, kAlongK, kAlongK, kGatedForward>(t, s);
}

struct BackwardPlan {
    size_t dg, du, part, total;  // byte offsets in the workspace
    int64_t ld;                  // elements between rows of dg and du: F in whole 16-byte chunks
    int dx_splits, dw_splits;
};
constexpr int kBM = 128, kBN = 128;
int splits_for(int64_t tiles, int64_t steps) {
    // enough workgroups for two on each of 256 CUs, each with at least 4 steps
    int64_t n = 1;
    while (n < 16 && tiles * n * 2 <= 512 && steps / (n * 2) >= 4) n *= 2;
    return (int)n;
}
BackwardPlan backward_plan(int64_t T, int d, int F, int bf16) {
    const size_t e = bf16 ? 2 : 4;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    auto tiles = [](int64_t m, int64_t n) { return (m + kBM - 1) / kBM * ((n + kBN - 1) / kBN); };
    const int bk = bf16 ? 64 : 32;
    BackwardPlan p{};
    p.dx_splits = splits_for(tiles(T, d), 2 * ((F + bk - 1) / bk));
    p.dw_splits = splits_for(2 * tiles(F, d), (T + bk - 1) / bk);
    const size_t dx_part = p.dx_splits > 1 ? (size_t)p.dx_splits * T * d * 4 : 0;
    const size_t dw_part = p.dw_splits > 1 ? (size_t)p.dw_splits * 2 * F * d * 4 : 0;
    p.ld = (F + 16 / e - 1) / (16 / e) * (16 / e);
    p.dg = 0;
    p.du = up((size_t)T * p.ld * e);
    p.part = 2 * p.du;
    p.total = p.part + up(std::max(dx_part, dw_part));
    return p;
}

template <bool BF16>
hipError_t gated_backward(const GatedBackwardArgs& a, hipStream_t s) {
    const BackwardPlan p = backward_plan(a.T, a.d, a.F, a.bf16);
    char* ws = (char*)a.workspace;
    void *dg = ws + p.dg, *du = ws + p.du;
    float* part = (float*)(ws + p.part);
    if (a.T > 0) {
        const int64_t chunks = a.T * (p.ld / Elem<BF16>::kChunk);
        hipLaunchKernelGGL((gate_backward_kernel<BF16>), dim3((unsigned)std::min<int64_t>((chunks + 255) / 256, 1 << 20)),
                           dim3(256), 0, s, a.dh, a.lddh, a.gate, a.up, a.T, a.F, p.ld, dg, du);
        if (hipError_t e = hipGetLastError()) return e;
    }
    if (a.dx && a.T > 0) {
        TileArgs t{};
        t.a[0] = Operand{dg, p.ld, a.T, a.F, 1};
        t.a[1] = Operand{du, p.ld, a.T, a.F, 1};
        t.b[0] = Operand{a.w_gate, a.d, a.d, a.F, 0};
        t.b[1] = Operand{a.w_up, a.d, a.d, a.F, 0};
        t.M = a.T;
        t.N = a.d;
        t.out[0] = a.dx;
        t.ldo = a.d;
        t.part = part;
        t.splits = p.dx_splits;
        if (hipError_t e = a.T > 512 ? launch_tiles<BF16, 128, 256, 2, 4, kAlongK, kAcrossK, kSumOfTwo>(t, s)
                                     : launch_tiles<BF16, 128, 128, 2, 2, kAlongK, kAcrossK, kSumOfTwo>(t, s)) return e;
        if (t.splits > 1) {
            const int64_t n = t.M * t.N;
            hipLaunchKernelGGL((reduce_kernel<BF16>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, part, t.splits,
                               (int64_t)1, n, a.dx, nullptr);
            if (hipError_t e = hipGetLastError()) return e;
        }
    }
    if (a.dw_gate) {
        TileArgs t{};
        t.a[0] = Operand{dg, p.ld, a.F, a.T, 1};
        t.a[1] = Operand{du, p.ld, a.F, a.T, 1};
        t.b[0] = t.b[1] = Operand{a.x, a.ldx, a.d, a.T, 0};
        t.M = a.F;
        t.N = a.d;
        t.out[0] = a.dw_gate;
        t.out[1] = a.dw_up;
        t.ldo = a.d;
        t.part = part;
        t.splits = p.dw_splits;
        if (hipError_t e = a.T > 512 ? launch_tiles<BF16, 256, 256, 2, 4, kAcrossK, kAcrossK, kTwoResults>(t, s)
                                     : launch_tiles<BF16, 128, 128, 2, 2, kAcrossK, kAcrossK, kTwoResults>(t, s)) return e;
        if (t.splits > 1) {
            const int64_t n = t.M * t.N;
            hipLaunchKernelGGL((reduce_kernel<BF16>), dim3((unsigned)((2 * n + 255) / 256)), dim3(256), 0, s, part, t.splits,
                               (int64_t)2, n, a.dw_gate, a.dw_up);
            if (hipError_t e = hipGetLastError()) return e;
        }
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_gated(const GatedArgs& a, hipStream_t s) { return a.bf16 ? gated<true>(a, s) : gated<false>(a, s); }

size_t gated_backward_bytes(int64_t T, int d, int F, int bf16) { return backward_plan(T, d, F, bf16).total; }

hipError_t launch_gated_backward(const GatedBackwardArgs& a, hipStream_t s) {
    return a.bf16 ? gated_backward<true>(a, s) : gated_backward<false>(a, s);
}

}  // namespace moe
