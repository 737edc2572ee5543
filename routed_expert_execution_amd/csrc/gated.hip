// The gated feed-forward block with bf16 or fp32 weights:
//   g = x Wg^T, u = x Wu^T, h = silu(g) u
// and its backward pass
//   dg = dh u s(g) (1 + g (1 - s(g))),  du = dh g s(g),  s the logistic function
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x.
#include <algorithm>

#include "dense.h"
#include "tile_kernel.h"

namespace moe {
namespace {

using namespace tile;

// k steps of a tile
int64_t steps_of(int64_t k, int bf16) { return (k + (bf16 ? 63 : 31)) / (bf16 ? 64 : 32); }

template <bool BF16> __device__ inline void store_elem(void* p, int64_t i, float v) {
    if (BF16) ((__bf16*)p)[i] = (__bf16)v;
    else ((float*)p)[i] = v;
}

// Both products of the backward pass in one launch: the workgroups of dx first
// (a whole number of rounds over the XCDs of them, as tile_of counts from zero),
// then those of dWg and dWu, which fill the CUs that dx leaves.
struct BackwardCounts { int dx_groups, dx_tiles, dw_tiles; };  // dx's workgroups, rounded up; tiles of one part of each
template <bool BF16, int BM, int BN, int WM, int WN, bool FAST>
__global__ __launch_bounds__(WM * WN * 64) void backward_tiles_kernel(TileArgs dx, TileArgs dw, BackwardCounts b) {
    __shared__ __attribute__((aligned(1024))) char lds[tile_lds<BM, BN>()];
    const int id = blockIdx.x;
    if (id < b.dx_groups) {
        if (id < b.dx_tiles * dx.splits)
            tile_body<BF16, BM, BN, WM, WN, kAlongK, kAcrossK, kSumOfTwo, FAST>(dx, id % b.dx_tiles, id / b.dx_tiles, lds);
    } else {
        const int i = id - b.dx_groups;
        tile_body<BF16, BM, BN, WM, WN, kAcrossK, kAcrossK, kTwoResults, FAST>(dw, i % b.dw_tiles, i / b.dw_tiles, lds);
    }
}

// Partial sums added in split order: of dx, then of dWg and dWu.
struct ReduceArgs {
    const float* part[2];
    int splits[2];
    int64_t each[2];    // elements of one part: T d, 2 F d; 0 where nothing is to be added
    void* out[3];       // dx, dWg, dWu
};
template <bool BF16>
__global__ __launch_bounds__(256) void reduce_kernel(ReduceArgs r) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < r.each[0] + r.each[1]; i += (int64_t)gridDim.x * 256) {
        const int w = i >= r.each[0];
        const int64_t k = w ? i - r.each[0] : i;
        const float* p = r.part[w] + k;
        float s = *p;
        for (int n = 1; n < r.splits[w]; n++) s += p[n * r.each[w]];
        if (!w) store_elem<BF16>(r.out[0], k, s);
        else if (k < r.each[1] / 2) store_elem<BF16>(r.out[1], k, s);
        else store_elem<BF16>(r.out[2], k - r.each[1] / 2, s);
    }
}

// dg and du into rows of whole 16-byte chunks (ld >= F), a chunk a thread.  In
// bf16 they are rounded once, as operands of the products that follow and as every
// other tensor of such a block is.  The gradients' error against 64 bits is 0.0023
// by that, where their own rounding makes it 0.0017; two terms of each would save
// the difference at twice the products (4096 tokens 8192 x 2048 533 us, as many
// products as two terms have 1040).
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

// ---- few tokens, forward ----------------------------------------------------

// Up to 16 MT tokens: bound by the bytes of the weights, which go from memory
// straight into the products' B operands, 16 rows of gate and of up a wave, the
// waves of a workgroup taking every blockDim / 64-th tile of columns and adding
// their sums in wave order through LDS.  A lane's 16 bytes of a row are columns
// of one product (bf16) or one column each of four (fp32): the order of the
// columns within a tile does not matter as long as x uses the same.  Four
// tokens at most sit in rows 0, 4, 8, 12 of the products (TI = 1), so that one
// result register holds them.
template <bool BF16, int MT, int TI>
__global__ __launch_bounds__(512) void gated_rows_kernel(GatedArgs a) {
    constexpr int E = Elem<BF16>::kChunk, kCols = 16 * E;  // columns of a tile: 4 chunks for each of 4 lane rows
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    extern __shared__ float red[];  // [2][waves][MT * TI][64]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n = lane & 15, q = lane >> 4;
    const int row0 = blockIdx.x * 16;
    const int64_t t0 = (int64_t)blockIdx.y * (16 * MT);
    const int tiles = (a.d + kCols - 1) / kCols;
    const int64_t row = min(row0 + n, a.F - 1);

    f32x4 acc[2][MT];
#pragma unroll
    for (int b = 0; b < 2; b++)
#pragma unroll
        for (int m = 0; m < MT; m++) acc[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    struct Chunks { u32x4 w[2][4]; };
    // (inside: wave-uniform, whether the whole tile lies before the rows' end)
    auto chunk = [&](const void* p, int64_t ld, int64_t r, int64_t k, bool inside) {
        if (inside) return ((const Loose*)((const typename Elem<BF16>::raw*)p + r * ld + k))->v;
        return load_chunk<BF16>(p, ld, r, k, r + 1, a.d);
    };
    auto load = [&](int kt, Chunks& c) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int64_t k = (int64_t)kt * kCols + (4 * j + q) * E;
            c.w[0][j] = chunk(a.w_gate, a.d, row, k, (kt + 1) * kCols <= a.d);
            c.w[1][j] = chunk(a.w_up, a.d, row, k, (kt + 1) * kCols <= a.d);
        }
    };
    Chunks cur, nxt;
    int kt = wave;
    if (kt < tiles) load(kt, cur);
    for (; kt < tiles; kt += waves) {
        u32x4 x[MT][4];
#pragma unroll
        for (int m = 0; m < MT; m++) {
            const int64_t t = t0 + (TI == 1 ? n / 4 : 16 * m + n);
#pragma unroll
            for (int j = 0; j < 4; j++)  // (rows past the last are computed and not stored)
                x[m][j] = chunk(a.x, a.ldx, t < a.T ? t : a.T - 1, (int64_t)kt * kCols + (4 * j + q) * E, (kt + 1) * kCols <= a.d);
        }
        if (kt + waves < tiles) load(kt + waves, nxt);
#pragma unroll
        for (int j = 0; j < 4; j++) {
#pragma unroll
            for (int b = 0; b < 2; b++) {
                const u32x4 w = cur.w[b][j];
#pragma unroll
                for (int m = 0; m < MT; m++) {
                    const u32x4 v = x[m][j];
                    if constexpr (BF16) {
                        acc[b][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, w),
                                                                            acc[b][m], 0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            acc[b][m] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(v[e]), __uint_as_float(w[e]), acc[b][m], 0, 0, 0);
                    }
                }
            }
        }
        cur = nxt;
    }

    constexpr int V = MT * TI;
#pragma unroll
    for (int b = 0; b < 2; b++)
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int i = 0; i < TI; i++) red[((b * waves + wave) * V + m * TI + i) * 64 + lane] = acc[b][m][i];
    __syncthreads();
    for (int v = threadIdx.x; v < V * 64; v += blockDim.x) {
        float sum[2];
#pragma unroll
        for (int b = 0; b < 2; b++) {
            sum[b] = red[b * waves * V * 64 + v];
            for (int w = 1; w < waves; w++) sum[b] += red[(b * waves + w) * V * 64 + v];
        }
        const int l = v & 63, mi = v >> 6;
        const int64_t t = t0 + (TI == 1 ? l >> 4 : 16 * (mi / TI) + 4 * (l >> 4) + mi % TI);
        const int64_t f = row0 + (l & 15);
        if (t < a.T && f < a.F) {
            store_elem<BF16>(a.h, t * a.F + f, silu(sum[0]) * sum[1]);
            if (a.gate) {
                store_elem<BF16>(a.gate, t * a.F + f, sum[0]);
                store_elem<BF16>(a.up, t * a.F + f, sum[1]);
            }
        }
    }
}

template <bool BF16, int MT, int TI>
hipError_t launch_gated_rows(const GatedArgs& a, int waves, hipStream_t s) {
    const dim3 grid((a.F + 15) / 16, (unsigned)((a.T + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((gated_rows_kernel<BF16, MT, TI>), grid, dim3(64 * waves), 2 * waves * MT * TI * 64 * sizeof(float), s, a);
    return hipGetLastError();
}

// Tokens a workgroup of the rows kernel takes (16 of them: 1, 2 or 4), by
// estimated time: the tiles of columns a wave takes one after the other, times
// what one costs.  In fp32 that is the products, 2 us for each 16 tokens (and
// more precise than the terms of the tiles); in bf16 mostly the wait for loads,
// 2.4 us and 1 for each 16.  Measured, us, 1 or 2, 4, and the tiles: fp32 100
// tokens 4096 x 512 41, 67, 59, 463 tokens 2005 x 350 43, 38, 51; bf16 100
// tokens 4096 x 512 17, 25, 15, 135 tokens 288 x 224 4.4, 6.1, 6.2.
int plan_rows(int64_t T, int d, int F, int bf16, float* us) {
    const int cols = bf16 ? 128 : 64, tiles = (d + cols - 1) / cols;
    int best = 4;
    *us = 1e30f;
    for (int mt = 1; mt <= 4; mt *= 2) {
        const int64_t groups = (int64_t)((F + 15) / 16) * ((T + 16 * mt - 1) / (16 * mt));
        const float t = (float)((tiles + 7) / 8) * (float)((groups + kTileCus - 1) / kTileCus) * (bf16 ? 2.4f + mt : 0.4f + 2.f * mt);
        if (t < *us) {
            best = mt;
            *us = t;
        }
    }
    return best;
}

template <bool BF16>
hipError_t gated(const GatedArgs& a, hipStream_t s) {
    const DensePlan p = gated_plan(a.T, a.d, a.F, BF16);
    if (p.kind == MOE_PLAN_ROWS) {
        if (p.tokens == 4) return launch_gated_rows<BF16, 1, 1>(a, p.parts, s);
        if (p.tokens == 16) return launch_gated_rows<BF16, 1, 4>(a, p.parts, s);
        return p.tokens == 32 ? launch_gated_rows<BF16, 2, 4>(a, p.parts, s) : launch_gated_rows<BF16, 4, 4>(a, p.parts, s);
    }
    TileArgs t{};
    t.a = Operand{{a.x, nullptr}, a.ldx, 0};
    t.b = Operand{{a.w_gate, a.w_up}, a.d, 0};
    t.M = a.T;
    t.N = a.F;
    t.K = a.d;
    t.out[0] = a.h;
    t.ldo = a.F;
    t.gate = a.gate;
    t.up = a.up;
    return launch_tiles<BF16, kAlongK, kAlongK, kGatedForward>(t, p.shape, s);
}

struct BackwardPlan {
    size_t dg, du, dx_part, dw_part, total;  // byte offsets in the workspace
    int64_t ld;                              // elements between rows of dg and du: F in whole 16-byte chunks
    int shape, dx_splits, dw_splits;
};
// One tile shape for both products (one launch) and a number of parts for each,
// by the estimate of plan_tiles; here the CUs share the steps of both, and no
// part may outlast them.
BackwardPlan backward_plan(int64_t T, int d, int F, int bf16) {
    BackwardPlan p{};
    const int64_t dx_steps = 2 * steps_of(F, bf16), dw_steps = steps_of(T, bf16);
    float best = 1e30f;
    for (int h = 0; h < kShapes; h++) {
        const TileShape& c = kTileShapes[bf16 ? kBf16 : kFp32][h];
        if (!c.per_cu || c.parts > 1) continue;
        auto tiles = [&](int64_t m, int64_t n) { return (m + c.bm - 1) / c.bm * ((n + c.bn - 1) / c.bn); };
        const int64_t dx_tiles = tiles(T, d), dw_tiles = 2 * tiles(F, d);
        for (int64_t n = 1; n <= 16 && (n == 1 || dx_steps / n >= 2); n *= 2)
            for (int64_t m = 1; m <= 16 && (m == 1 || dw_steps / m >= 2); m *= 2) {
                const int64_t a = (dx_steps + n - 1) / n, b = (dw_steps + m - 1) / m, most = std::max(a, b);
                const int64_t groups = dx_tiles * n + dw_tiles * m, cap = kTileCus * c.per_cu;
                float us;
                if (groups <= kTileCus) us = (float)most * c.one;
                else us = std::max((float)(dx_tiles * n * a + dw_tiles * m * b) / cap + 0.25f * std::min(a, b), (float)most) * c.full;
                if (n > 1 || m > 1) us += 4.f;
                if (n > 1) us += (float)T * d * (float)(8 * n + 4) / 4e6f;
                if (m > 1) us += 2.f * F * d * (float)(8 * m + 4) / 4e6f;
                if (us < best) {
                    best = us;
                    p.shape = h;
                    p.dx_splits = (int)n;
                    p.dw_splits = (int)m;
                }
            }
    }
    const size_t e = bf16 ? 2 : 4;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    p.ld = (F + 16 / e - 1) / (16 / e) * (16 / e);
    p.dg = 0;
    p.du = up((size_t)T * p.ld * e);
    p.dx_part = 2 * p.du;
    p.dw_part = p.dx_part + (p.dx_splits > 1 ? up((size_t)p.dx_splits * T * d * 4) : 0);
    p.total = p.dw_part + (p.dw_splits > 1 ? up((size_t)p.dw_splits * 2 * F * d * 4) : 0);
    return p;
}

template <bool BF16, int BM, int BN, int WM, int WN>
hipError_t launch_backward_tiles(TileArgs x, TileArgs w, bool dx, bool dw, hipStream_t s) {
    auto tiles = [](TileArgs& t) {
        t.m_tiles = (int)((t.M + BM - 1) / BM);
        t.n_tiles = (int)((t.N + BN - 1) / BN);
        return t.m_tiles * t.n_tiles;
    };
    BackwardCounts b{0, tiles(x), tiles(w)};
    x.products = 1;
    w.products = 2;
    if (dx) b.dx_groups = (b.dx_tiles * x.splits + kXcds - 1) / kXcds * kXcds;
    const bool fast = (!dx || (fast_operand(x.a, kAlongK, x.M, true, BF16) && fast_operand(x.b, kAcrossK, x.N, true, BF16))) &&
                      (!dw || (fast_operand(w.a, kAcrossK, w.M, true, BF16) && fast_operand(w.b, kAcrossK, w.N, false, BF16)));
    const dim3 grid((unsigned)(b.dx_groups + (dw ? 2 * b.dw_tiles * w.splits : 0))), block(WM * WN * 64);
    if (fast) hipLaunchKernelGGL((backward_tiles_kernel<BF16, BM, BN, WM, WN, true>), grid, block, 0, s, x, w, b);
    else hipLaunchKernelGGL((backward_tiles_kernel<BF16, BM, BN, WM, WN, false>), grid, block, 0, s, x, w, b);
    return hipGetLastError();
}

template <bool BF16>
hipError_t gated_backward(const GatedBackwardArgs& a, hipStream_t s) {
    const BackwardPlan p = backward_plan(a.T, a.d, a.F, a.bf16);
    char* ws = (char*)a.workspace;
    void *dg = ws + p.dg, *du = ws + p.du;
    const bool dx = a.dx && a.T > 0, dw = a.dw_gate != nullptr;
    if (!dx && !dw) return hipSuccess;
    if (a.T > 0) {
        const int64_t chunks = a.T * (p.ld / Elem<BF16>::kChunk);
        hipLaunchKernelGGL((gate_backward_kernel<BF16>), dim3((unsigned)std::min<int64_t>((chunks + 255) / 256, 1 << 20)),
                           dim3(256), 0, s, a.dh, a.lddh, a.gate, a.up, a.T, a.F, p.ld, dg, du);
        if (hipError_t e = hipGetLastError()) return e;
    }
    TileArgs x{}, w{};
    x.a = Operand{{dg, du}, p.ld, 1};
    x.b = Operand{{a.w_gate, a.w_up}, a.d, 0};
    x.M = a.T;
    x.N = a.d;
    x.K = a.F;
    x.out[0] = a.dx;
    x.ldo = a.d;
    x.part = (float*)(ws + p.dx_part);
    x.splits = p.dx_splits;
    w.a = Operand{{dg, du}, p.ld, 1};
    w.b = Operand{{a.x, a.x}, a.ldx, 0};
    w.M = a.F;
    w.N = a.d;
    w.K = a.T;
    w.out[0] = a.dw_gate;
    w.out[1] = a.dw_up;
    w.ldo = a.d;
    w.part = (float*)(ws + p.dw_part);
    w.splits = p.dw_splits;
    hipError_t e = hipErrorInvalidValue;
    if (p.shape == kShape256x128) e = launch_backward_tiles<BF16, 256, 128, 4, 2>(x, w, dx, dw, s);
    else if (p.shape == kShape128) e = launch_backward_tiles<BF16, 128, 128, 2, 2>(x, w, dx, dw, s);
    else if (p.shape == kShapeSmall) e = launch_backward_tiles<BF16, 64, 64, 2, 2>(x, w, dx, dw, s);
    else if constexpr (BF16) e = launch_backward_tiles<BF16, 256, 256, 2, 4>(x, w, dx, dw, s);
    if (e) return e;
    ReduceArgs r{{x.part, w.part}, {p.dx_splits, p.dw_splits},
                 {dx && p.dx_splits > 1 ? a.T * a.d : 0, dw && p.dw_splits > 1 ? (int64_t)2 * a.F * a.d : 0},
                 {a.dx, a.dw_gate, a.dw_up}};
    if (const int64_t n = r.each[0] + r.each[1]) {
        hipLaunchKernelGGL((reduce_kernel<BF16>), dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20)), dim3(256), 0, s, r);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace

DensePlan gated_plan(int64_t T, int d, int F, int bf16) {
    int waves = 1;
    while (waves < 8 && waves < (d + (bf16 ? 127 : 63)) / (bf16 ? 128 : 64)) waves *= 2;
    if (T <= 4) return {MOE_PLAN_ROWS, 4, 16, waves, 1, 1, 0};
    if (T <= 16) return {MOE_PLAN_ROWS, 16, 16, waves, 1, 1, 0};
    // (gate and up columns alternate: twice F of them)
    float tiles_us, rows_us;
    const int kind = bf16 ? kBf16 : kFp32, shape = plan_tiles(kind, T, 2 * (int64_t)F, steps_of(d, bf16), bf16 ? kShapes : kShape256x128, &tiles_us);
    const int mt = plan_rows(T, d, F, bf16, &rows_us);
    if (rows_us < tiles_us + 1.5f) return {MOE_PLAN_ROWS, 16 * mt, 16, waves, 1, 1, 0};
    return tiles_plan(kind, shape, true);
}

DensePlan gated_backward_plan(int64_t T, int d, int F, int bf16) {
    const BackwardPlan p = backward_plan(T, d, F, bf16);
    DensePlan plan = tiles_plan(bf16 ? kBf16 : kFp32, p.shape, false);
    plan.dx_parts = p.dx_splits;
    plan.dw_parts = p.dw_splits;
    return plan;
}

hipError_t launch_gated(const GatedArgs& a, hipStream_t s) { return a.bf16 ? gated<true>(a, s) : gated<false>(a, s); }

size_t gated_backward_bytes(int64_t T, int d, int F, int bf16) { return backward_plan(T, d, F, bf16).total; }

hipError_t launch_gated_backward(const GatedBackwardArgs& a, hipStream_t s) {
    return a.bf16 ? gated_backward<true>(a, s) : gated_backward<false>(a, s);
}

}  // namespace moe
