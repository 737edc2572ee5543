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

template <bool BF16> __device__ inline float load_elem(const void* p, int64_t i) {
    if (BF16) return bf16_bits_to_f32(((const uint16_t*)p)[i]);
    return ((const float*)p)[i];
}
template <bool BF16> __device__ inline void store_elem(void* p, int64_t i, float v) {
    if (BF16) ((__bf16*)p)[i] = (__bf16)v;
    else ((float*)p)[i] = v;
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
