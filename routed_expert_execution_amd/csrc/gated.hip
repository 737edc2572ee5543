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

constexpr int kBM = 128, kBN = 128;

struct TileArgs {
    Operand a[2], b[2];  // two products: summed over k, side by side in n, or one after the other in z
    int64_t M, N;        // of one product's result
    void* out[2];
    int64_t ldo;
    void* gate;
    void* up;
    float* part;         // [splits][products][M][N] partial sums
    int splits;
};

enum { kGatedForward, kSumOfTwo, kTwoResults };

// 4 waves, each 64 x 64 of a 128 x 128 tile.  kGatedForward: the tile's columns
// alternate 32 of gate and 32 of up, so that a wave holds both of an element.
template <bool BF16, int ALAY, int BLAY, int MODE>
__global__ __launch_bounds__(256) void tile_kernel(TileArgs t) {
    typedef TileOf<BF16, kBM, ALAY> TA;
    typedef TileOf<BF16, kBN, BLAY> TB;
    constexpr int BK = TA::BK;
    __shared__ __attribute__((aligned(16))) char lds[2][TA::kBytes + TB::kBytes];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const int64_t m0 = (int64_t)blockIdx.x * kBM;
    const int64_t n0 = (int64_t)blockIdx.y * (MODE == kGatedForward ? kBN / 2 : kBN);
    const int which = MODE == kTwoResults ? blockIdx.z & 1 : 0;
    const int split = MODE == kTwoResults ? blockIdx.z >> 1 : blockIdx.z;

    const int64_t steps1 = (t.a[0].K + BK - 1) / BK;
    const int64_t steps = MODE == kSumOfTwo ? 2 * steps1 : steps1;
    const int64_t s0 = steps * split / t.splits, s1 = steps * (split + 1) / t.splits;

    constexpr int CA = TA::kChunks / 256, CB = TB::kChunks / 256;
    u32x4 ra[CA], rb[CB];
    auto fetch = [&](int64_t s) {
        const int p = MODE == kSumOfTwo ? (s >= steps1) : which;
        const int64_t k0 = (MODE == kSumOfTwo && s >= steps1 ? s - steps1 : s) * BK;
        const Operand a = t.a[p];
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int q = threadIdx.x + 256 * i, line = q / TA::kLineChunks, c = q % TA::kLineChunks;
            ra[i] = ALAY == kAlongK ? load_chunk<BF16>(a.p, a.ld, m0 + line, k0 + c * TA::E, a.R, a.K)
                                    : load_chunk<BF16>(a.p, a.ld, k0 + line, m0 + c * TA::E, a.K, a.R);
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int q = threadIdx.x + 256 * i, line = q / TB::kLineChunks, c = q % TB::kLineChunks;
            if (MODE == kGatedForward) {
                const Operand b = t.b[line >> 5 & 1];
                rb[i] = load_chunk<BF16>(b.p, b.ld, n0 + (line >> 6) * 32 + (line & 31), k0 + c * TB::E, b.R, b.K);
            } else {
                const Operand b = t.b[p];
                rb[i] = BLAY == kAlongK ? load_chunk<BF16>(b.p, b.ld, n0 + line, k0 + c * TB::E, b.R, b.K)
                                        : load_chunk<BF16>(b.p, b.ld, k0 + line, n0 + c * TB::E, b.K, b.R);
            }
        }
    };
    auto stage = [&](char* l) {
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int q = threadIdx.x + 256 * i;
            *(u32x4*)(l + TA::chunk_at(q / TA::kLineChunks, q % TA::kLineChunks)) = ra[i];
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int q = threadIdx.x + 256 * i;
            *(u32x4*)(l + TA::kBytes + TB::chunk_at(q / TB::kLineChunks, q % TB::kLineChunks)) = rb[i];
        }
    };

    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.f;

    if (s0 < s1) {
        fetch(s0);
        stage(lds[0]);
        __syncthreads();
    }
    for (int64_t s = s0; s < s1; s++) {
        const int cur = (int)(s - s0) & 1;
        if (s + 1 < s1) fetch(s + 1);
        typedef typename std::conditional<BF16, bf16x8, f32x4>::type Frag;
#pragma unroll
        for (int kk = 0; kk < 4; kk++) {
            Frag fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                TA::frag(lds[cur], wm + 32 * i, kk, lane, fa[i]);
                TB::frag(lds[cur] + TA::kBytes, wn + 32 * i, kk, lane, fb[i]);
            }
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int j = 0; j < 2; j++) mma(acc[i][j], fa[i], fb[j]);
        }
        if (s + 1 < s1) {
            stage(lds[cur ^ 1]);
            __syncthreads();
        }
    }

#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) {
            const int64_t m = m0 + wm + 32 * i + acc_row(lane, e);
            if (m >= t.M) continue;
            if (MODE == kGatedForward) {
                const int64_t n = n0 + wn / 2 + (lane & 31);
                if (n >= t.N) continue;
                const float g = acc[i][0][e], u = acc[i][1][e];
                store_elem<BF16>(t.out[0], m * t.ldo + n, silu(g) * u);
                if (t.gate) store_elem<BF16>(t.gate, m * t.ldo + n, g);
                if (t.up) store_elem<BF16>(t.up, m * t.ldo + n, u);
            } else {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int64_t n = n0 + wn + 32 * j + (lane & 31);
                    if (n >= t.N) continue;
                    if (t.splits > 1) {
                        const int products = MODE == kTwoResults ? 2 : 1;
                        t.part[((int64_t)(split * products + which) * t.M + m) * t.N + n] = acc[i][j][e];
                    } else {
                        store_elem<BF16>(t.out[which], m * t.ldo + n, acc[i][j][e]);
                    }
                }
            }
        }
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

// dg and du, an element a thread.  In bf16 they are rounded once, as the
// products that follow take them.
template <bool BF16>
__global__ __launch_bounds__(256) void gate_backward_kernel(const void* __restrict__ dh, int64_t lddh,
                                                            const void* __restrict__ gate, const void* __restrict__ up,
                                                            int64_t T, int F, void* __restrict__ dg, void* __restrict__ du) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= T * F) return;
    const float d = load_elem<BF16>(dh, i / F * lddh + i % F), g = load_elem<BF16>(gate, i), u = load_elem<BF16>(up, i);
    const float s = 1.0f / (1.0f + expf(-g));
    store_elem<BF16>(dg, i, d * u * s * (1.0f + g * (1.0f - s)));
    store_elem<BF16>(du, i, d * g * s);
}

template <bool BF16>
hipError_t gated(const GatedArgs& a, hipStream_t s) {
    TileArgs t{};
    t.a[0] = Operand{a.x, a.ldx, a.T, a.d};
    t.b[0] = Operand{a.w_gate, a.d, a.F, a.d};
    t.b[1] = Operand{a.w_up, a.d, a.F, a.d};
    t.M = a.T;
    t.N = a.F;
    t.out[0] = a.h;
    t.ldo = a.F;
    t.gate = a.gate;
    t.up = a.up;
    t.splits = 1;
    const dim3 grid((unsigned)((a.T + kBM - 1) / kBM), (unsigned)((a.F + kBN / 2 - 1) / (kBN / 2)));
    hipLaunchKernelGGL((tile_kernel<BF16, kAlongK, kAlongK, kGatedForward>), grid, dim3(256), 0, s, t);
    return hipGetLastError();
}

struct BackwardPlan {
    size_t dg, du, part, total;  // byte offsets in the workspace
    int dx_splits, dw_splits;
};
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
    p.dg = 0;
    p.du = up((size_t)T * F * e);
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
        hipLaunchKernelGGL((gate_backward_kernel<BF16>), dim3((unsigned)((a.T * a.F + 255) / 256)), dim3(256), 0, s, a.dh,
                           a.lddh, a.gate, a.up, a.T, a.F, dg, du);
        if (hipError_t e = hipGetLastError()) return e;
    }
    if (a.dx && a.T > 0) {
        TileArgs t{};
        t.a[0] = Operand{dg, a.F, a.T, a.F};
        t.a[1] = Operand{du, a.F, a.T, a.F};
        t.b[0] = Operand{a.w_gate, a.d, a.d, a.F};
        t.b[1] = Operand{a.w_up, a.d, a.d, a.F};
        t.M = a.T;
        t.N = a.d;
        t.out[0] = a.dx;
        t.ldo = a.d;
        t.part = part;
        t.splits = p.dx_splits;
        const dim3 grid((unsigned)((t.M + kBM - 1) / kBM), (unsigned)((t.N + kBN - 1) / kBN), t.splits);
        hipLaunchKernelGGL((tile_kernel<BF16, kAlongK, kAcrossK, kSumOfTwo>), grid, dim3(256), 0, s, t);
        if (hipError_t e = hipGetLastError()) return e;
        if (t.splits > 1) {
            const int64_t n = t.M * t.N;
            hipLaunchKernelGGL((reduce_kernel<BF16>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, part, t.splits,
                               (int64_t)1, n, a.dx, nullptr);
            if (hipError_t e = hipGetLastError()) return e;
        }
    }
    if (a.dw_gate) {
        TileArgs t{};
        t.a[0] = Operand{dg, a.F, a.F, a.T};
        t.a[1] = Operand{du, a.F, a.F, a.T};
        t.b[0] = t.b[1] = Operand{a.x, a.ldx, a.d, a.T};
        t.M = a.F;
        t.N = a.d;
        t.out[0] = a.dw_gate;
        t.out[1] = a.dw_up;
        t.ldo = a.d;
        t.part = part;
        t.splits = p.dw_splits;
        const dim3 grid((unsigned)((t.M + kBM - 1) / kBM), (unsigned)((t.N + kBN - 1) / kBN), 2 * t.splits);
        hipLaunchKernelGGL((tile_kernel<BF16, kAcrossK, kAcrossK, kTwoResults>), grid, dim3(256), 0, s, t);
        if (hipError_t e = hipGetLastError()) return e;
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
