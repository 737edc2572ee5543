// Products of up to 64 tokens at a time with 4-bit weights and group scales.
//
//   y[t, n] = sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) x[t, k]
//
// Bound by the bytes of the weights, so a weight has to cost few instructions:
// its code goes into the top mantissa bits of a bf16 whose exponent is that of
// 16, which makes the pair of codes in a word two bf16 16 + q in a shift and
// one and-or, and the matrix cores sum (16 + q) x over a group exactly as they
// would sum the weights.  The group's sum of x alone, one more product with a
// matrix of ones shared by every row, turns that into the sum of (q - z) x in
// fp32:   s * (sum (16 + q) x - (16 + z) sum x).   Nothing is rounded to bf16:
// codes and bf16 x are exact in the products, fp32 x enters as three bf16 terms
// (x = a + b + c to 24 bits) with a product each, and scales, zero points and
// sums stay in fp32.  The subtraction costs about two bits of the sum's 24
// (16 + q against q - z).
#pragma once

#include "dense.h"
#include "device_util.h"

namespace moe {
namespace linear {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16-byte loads from addresses aligned to the element only.
struct __attribute__((packed, aligned(2))) Loose16 { u32x4 v; };
struct __attribute__((packed, aligned(4))) Loose16f { f32x4 v; };

// A word's 8 codes as bf16 16 + q, columns in order.
__device__ inline bf16x8 codes_bf16(uint32_t w) {
    const uint32_t mask = 0x00780078u, one = 0x41804180u;
    u32x4 r;
    r[0] = ((w << 3) & mask) | one;
    r[1] = ((w >> 1) & mask) | one;
    r[2] = ((w >> 5) & mask) | one;
    r[3] = ((w >> 9) & mask) | one;
    return __builtin_bit_cast(bf16x8, r);
}

// The A operands of one 32-column step: 8 columns of this lane's token.
template <bool BF16>
struct XOperand;
template <>
struct XOperand<true> {
    static constexpr int kTerms = 1;
    u32x4 raw;
    __device__ void load(const void* x, int64_t at) { raw = ((const Loose16*)((const uint16_t*)x + at))->v; }
    __device__ void terms(bf16x8 (&t)[1]) const { t[0] = __builtin_bit_cast(bf16x8, raw); }
};
template <>
struct XOperand<false> {
    static constexpr int kTerms = 3;
    f32x4 raw[2];
    __device__ void load(const void* x, int64_t at) {
        const float* p = (const float*)x + at;
        raw[0] = ((const Loose16f*)p)->v;
        raw[1] = ((const Loose16f*)(p + 4))->v;
    }
    __device__ void terms(bf16x8 (&t)[3]) const {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float v = raw[i / 4][i % 4];
            t[0][i] = (__bf16)v;
            const float r = v - (float)t[0][i];
            t[1][i] = (__bf16)r;
            t[2][i] = (__bf16)(r - (float)t[1][i]);
        }
    }
};

// MT token tiles of 16, of which TI result registers are used.  A result
// register i of lane l is token row 4 (l / 16) + i, so up to four tokens sit in
// rows 0, 4, 8 and 12 and need register 0 alone (TI = 1).
// A wave takes R row groups (of each matrix) and every blockDim / 64-th column
// tile; the waves' sums are added in wave order through LDS.
template <bool XBF16, int MT, int TI, int R, int S, bool GATED>
__global__ __launch_bounds__(512) void rows_kernel(LinearArgs a) {
    constexpr int NB = GATED ? 2 : 1, RB = R * NB;
    constexpr int kTerms = XOperand<XBF16>::kTerms;
    extern __shared__ float red[];  // [NB][waves][MT * TI][64]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int n = lane & 15, q = lane >> 4;
    const int rg0 = blockIdx.x * R;
    const int64_t t0 = (int64_t)blockIdx.y * (16 * MT);

    int64_t xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; m++) {
        int64_t t = t0 + (TI == 1 ? n / 4 : 16 * m + n);
        xrow[m] = (t < a.T ? t : a.T - 1) * a.ldx;  // (rows past the last are computed and not stored)
    }
    bf16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; i++) ones[i] = (__bf16)1.0f;

    f32x4 out[RB][MT];
#pragma unroll
    for (int r = 0; r < RB; r++)
#pragma unroll
        for (int m = 0; m < MT; m++) out[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    struct Tile {
        uint4 code[RB];
        uint16_t scale[RB][S];
        uint8_t zero[RB][S];
    };
    auto load = [&](int kt, Tile& t) {
#pragma unroll
        for (int r = 0; r < RB; r++) {
            const QuantView& w = a.w[r / R];
            const int rg = min(rg0 + r % R, a.row_groups - 1);
            const int64_t tile = (int64_t)rg * a.col_tiles + kt;
            t.code[r] = w.codes[tile * 64 + lane];
            __builtin_memcpy(t.scale[r], __builtin_assume_aligned(w.scales + (tile * 16 + n) * S, 2 * S), 2 * S);
            if (w.zeros) __builtin_memcpy(t.zero[r], __builtin_assume_aligned(w.zeros + (tile * 16 + n) * S, S), S);
        }
    };
    Tile cur, nxt;
    int kt = wave;
    if (kt < a.col_tiles) load(kt, cur);
    for (; kt < a.col_tiles; kt += waves) {
        XOperand<XBF16> x[4][MT];
        const int steps = min(4, (a.cols - kt * 128) / 32);  // (columns come in whole 32s)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int m = 0; m < MT; m++)
                x[j][m].load(a.x, xrow[m] + kt * 128 + 32 * min(j, steps - 1) + 8 * q);
        if (kt + waves < a.col_tiles) load(kt + waves, nxt);
        f32x4 acc[RB][MT], xs[MT];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j >= steps) break;
            if (j % (4 / S) == 0) {
#pragma unroll
                for (int m = 0; m < MT; m++) {
                    xs[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int r = 0; r < RB; r++) acc[r][m] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            }
            bf16x8 xt[MT][kTerms];
#pragma unroll
            for (int m = 0; m < MT; m++) {
                x[j][m].terms(xt[m]);
#pragma unroll
                for (int c = kTerms - 1; c >= 0; c--)
                    xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xt[m][c], ones, xs[m], 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < RB; r++) {
                const uint32_t word = j == 0 ? cur.code[r].x : j == 1 ? cur.code[r].y : j == 2 ? cur.code[r].z : cur.code[r].w;
                const bf16x8 w = codes_bf16(word);
#pragma unroll
                for (int m = 0; m < MT; m++)
#pragma unroll
                    for (int c = kTerms - 1; c >= 0; c--)
                        acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xt[m][c], w, acc[r][m], 0, 0, 0);
            }
            if (j % (4 / S) == 4 / S - 1 || j == steps - 1) {
#pragma unroll
                for (int r = 0; r < RB; r++) {
                    const float s = f16_bits_to_f32(cur.scale[r][j / (4 / S)]);
                    const float z = a.w[r / R].zeros ? 16.f + (float)cur.zero[r][j / (4 / S)] : 24.f;
#pragma unroll
                    for (int m = 0; m < MT; m++)
#pragma unroll
                        for (int i = 0; i < TI; i++) out[r][m][i] = fmaf(s, fmaf(-z, xs[m][i], acc[r][m][i]), out[r][m][i]);
                }
            }
        }
        cur = nxt;
    }

    constexpr int V = MT * TI;
#pragma unroll
    for (int r = 0; r < R; r++) {
        if (r) __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; b++)
#pragma unroll
            for (int m = 0; m < MT; m++)
#pragma unroll
                for (int i = 0; i < TI; i++) red[((b * waves + wave) * V + m * TI + i) * 64 + lane] = out[b * R + r][m][i];
        __syncthreads();
        for (int v = threadIdx.x; v < V * 64; v += blockDim.x) {
            float sum[NB];
#pragma unroll
            for (int b = 0; b < NB; b++) {
                sum[b] = red[b * waves * V * 64 + v];
                for (int w = 1; w < waves; w++) sum[b] += red[(b * waves + w) * V * 64 + v];
            }
            const int l = v & 63, mi = v >> 6;
            const int64_t t = t0 + (TI == 1 ? l >> 4 : 16 * (mi / TI) + 4 * (l >> 4) + mi % TI);
            const int64_t row = (int64_t)(rg0 + r) * 16 + (l & 15);
            if (t < a.T && row < a.rows) {
                const float y = GATED ? silu(sum[0]) * sum[NB - 1] : sum[0];
                if (a.y_bf16) ((__bf16*)a.y)[t * a.ldy + row] = (__bf16)y;
                else ((float*)a.y)[t * a.ldy + row] = y;
            }
        }
    }
}

template <bool XBF16, int MT, int TI, int R, bool GATED>
hipError_t launch_rows(const LinearArgs& a, int waves, hipStream_t s) {
    const dim3 grid((a.row_groups + R - 1) / R, (unsigned)((a.T + 16 * MT - 1) / (16 * MT)));
    const size_t lds = (size_t)(GATED ? 2 : 1) * waves * MT * TI * 64 * sizeof(float);
    if (a.group == 32) hipLaunchKernelGGL((rows_kernel<XBF16, MT, TI, R, 4, GATED>), grid, dim3(64 * waves), lds, s, a);
    else if (a.group == 64) hipLaunchKernelGGL((rows_kernel<XBF16, MT, TI, R, 2, GATED>), grid, dim3(64 * waves), lds, s, a);
    else hipLaunchKernelGGL((rows_kernel<XBF16, MT, TI, R, 1, GATED>), grid, dim3(64 * waves), lds, s, a);
    return hipGetLastError();
}

template <bool XBF16, bool GATED>
hipError_t launch_rows_t(const LinearArgs& a, hipStream_t s) {
    int waves = 1;
    while (waves < 8 && waves < a.col_tiles) waves *= 2;
    if (a.T <= 4) return launch_rows<XBF16, 1, 1, 1, GATED>(a, waves, s);
    if (a.T <= 16) return launch_rows<XBF16, 1, 4, 1, GATED>(a, waves, s);
    return launch_rows<XBF16, 4, 4, 1, GATED>(a, waves, s);
}

}  // namespace linear

// One translation unit each (linear_bf16.hip, linear_f32.hip).
hipError_t launch_linear_rows_bf16(const LinearArgs& a, bool gated, hipStream_t s);
hipError_t launch_linear_rows_f32(const LinearArgs& a, bool gated, hipStream_t s);

}  // namespace moe
