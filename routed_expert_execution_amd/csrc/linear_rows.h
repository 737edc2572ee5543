// Products of up to 64 tokens at a time with 4-bit weights and group scales.
//
//   y[t, n] = sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) x[t, k]
//
// Bound by the bytes of the weights, so a weight has to cost few instructions.
// bf16 x: a code goes into the top mantissa bits of a bf16 whose exponent is that
// of 16, which makes the pair of codes in a word two bf16 16 + q in a shift and
// one and-or, and the matrix cores sum (16 + q) x over a group exactly as they
// would sum the weights.  The group's sum of x alone, one more product with a
// matrix of ones shared by every row, turns that into the sum of (q - z) x in
// fp32:   s * (sum (16 + q) x - (16 + z) sum x).
// fp32 x enters as three bf16 terms (x = a + b + c to 24 bits) with a product
// each, and there the sums of 16 + q would cost two of the 24 bits: the codes are
// made q - z, exact in bf16, at three times the instructions, which the terms
// outweigh.  Nothing is rounded to bf16: codes and terms are exact in the
// products, and scales and sums stay in fp32.
#pragma once

#include "bf16_terms.h"
#include "dense.h"
#include "device_util.h"
#include "quant_codes.h"

namespace moe {
namespace linear {

typedef bf16x8_t bf16x8;
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
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = raw[i / 4][i % 4];
        bf16_terms(v, t);
    }
};

// Up to 16 tokens, of which TI result registers are used.  A result register i
// of lane l is token row 4 (l / 16) + i, so up to four tokens sit in rows 0, 4,
// 8 and 12 and need register 0 alone (TI = 1).
// A wave takes R row groups (of each matrix) and every blockDim / 64-th column
// tile; the waves' sums are added in wave order through LDS.
template <bool XBF16, int TI, int R, int S, bool GATED>
__global__ __launch_bounds__(512) void rows_kernel(LinearArgs a) {
    constexpr int NB = GATED ? 2 : 1, RB = R * NB;
    constexpr int kTerms = XOperand<XBF16>::kTerms;
    extern __shared__ float red[];  // [NB][waves][TI][64]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n = lane & 15, q = lane >> 4;
    const int rg0 = blockIdx.x * R;
    const int64_t token = TI == 1 ? n / 4 : n;
    const int64_t xrow = (token < a.T ? token : a.T - 1) * a.ldx;  // (rows past the last are computed and not stored)
    bf16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; i++) ones[i] = (__bf16)1.0f;
    f32x4 out[RB];
#pragma unroll
    for (int r = 0; r < RB; r++) out[r] = f32x4{0.f, 0.f, 0.f, 0.f};

    struct Tile {
        uint4 code[RB];
        uint16_t scale[RB][S];
        uint8_t zero[RB][S];
        XOperand<XBF16> x[4];
    };
    auto load = [&](int kt, Tile& t) {
#pragma unroll
        for (int r = 0; r < RB; r++) {
            const QuantView& w = a.w[r / R];
            const int64_t tile = (int64_t)min(rg0 + r % R, a.row_groups - 1) * a.col_tiles + kt;
            t.code[r] = w.codes[tile * 64 + lane];
            __builtin_memcpy(t.scale[r], __builtin_assume_aligned(w.scales + (tile * 16 + n) * S, 2 * S), 2 * S);
            if (w.zeros) __builtin_memcpy(t.zero[r], __builtin_assume_aligned(w.zeros + (tile * 16 + n) * S, S), S);
        }
#pragma unroll
        for (int j = 0; j < 4; j++)  // (past the last column the token's last ones, which meet zero codes and scales)
            t.x[j].load(a.x, xrow + min(kt * 128 + 32 * j + 8 * q, a.cols - 8));
    };
    Tile cur, nxt;
    int kt = wave;
    if (kt < a.col_tiles) load(kt, cur);
    for (; kt < a.col_tiles; kt += waves) {
        if (kt + waves < a.col_tiles) load(kt + waves, nxt);
        f32x4 acc[RB], xs;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j % (4 / S) == 0) {
                xs = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int r = 0; r < RB; r++) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            bf16x8 xt[kTerms];
            cur.x[j].terms(xt);
            if constexpr (XBF16) xs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xt[0], ones, xs, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < RB; r++) {
                const uint4 c4 = cur.code[r];
                const uint32_t word = j == 0 ? c4.x : j == 1 ? c4.y : j == 2 ? c4.z : c4.w;
                const float z = a.w[r / R].zeros ? (float)cur.zero[r][j / (4 / S)] : 8.f;
                const bf16x8 w = XBF16 ? codes_bf16(word) : codes_less_zero(word, z);
#pragma unroll
                for (int c = kTerms - 1; c >= 0; c--) acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xt[c], w, acc[r], 0, 0, 0);
            }
            if (j % (4 / S) == 4 / S - 1) {
#pragma unroll
                for (int r = 0; r < RB; r++) {
                    const float s = f16_bits_to_f32(cur.scale[r][j / (4 / S)]);
                    const float z = a.w[r / R].zeros ? 16.f + (float)cur.zero[r][j / (4 / S)] : 24.f;
#pragma unroll
                    for (int i = 0; i < TI; i++) out[r][i] = fmaf(s, XBF16 ? fmaf(-z, xs[i], acc[r][i]) : acc[r][i], out[r][i]);
                }
            }
        }
        cur = nxt;
    }

#pragma unroll
    for (int r = 0; r < R; r++) {
        if (r) __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; b++)
#pragma unroll
            for (int i = 0; i < TI; i++) red[((b * waves + wave) * TI + i) * 64 + lane] = out[b * R + r][i];
        __syncthreads();
        for (int v = threadIdx.x; v < TI * 64; v += blockDim.x) {
            float sum[NB];
#pragma unroll
            for (int b = 0; b < NB; b++) {
                sum[b] = red[b * waves * TI * 64 + v];
                for (int w = 1; w < waves; w++) sum[b] += red[(b * waves + w) * TI * 64 + v];
            }
            const int l = v & 63, i = v >> 6;
            const int64_t t = TI == 1 ? l >> 4 : 4 * (l >> 4) + i;
            const int64_t row = (int64_t)(rg0 + r) * 16 + (l & 15);
            if (t < a.T && row < a.rows) {
                const float y = GATED ? silu(sum[0]) * sum[NB - 1] : sum[0];
                if (a.y_bf16) ((__bf16*)a.y)[t * a.ldy + row] = (__bf16)y;
                else ((float*)a.y)[t * a.ldy + row] = y;
            }
        }
    }
}

// More tokens, or fp32 x.  There the activations, not the weights, are most of
// what a wave reads and (fp32) converts, so RW waves with a row group each share
// them: the workgroup stages a tile of 128 columns for each of its KW parts of
// the columns in LDS, as bf16 terms, while the tile before is multiplied.  An
// x operand is then 16 bytes a lane from LDS; chunk c of row r sits at
// c ^ r % 16, so that the 16 rows of a read cover all banks.
template <bool XBF16, int MT, int RW, int KW, int S, bool GATED>
__global__ __launch_bounds__(64 * RW * KW) void shared_rows_kernel(LinearArgs a) {
    constexpr int NB = GATED ? 2 : 1, kThreads = 64 * RW * KW, V = MT * 4;
    constexpr int kTerms = XOperand<XBF16>::kTerms;
    constexpr int kRows = 16 * MT;
    constexpr int kPlane = 16 * MT * 256, kPart = kTerms * kPlane;  // LDS bytes of a term's tile, of a part's
    constexpr int kChunks = kRows * 16 * KW, kPer = (kChunks + kThreads - 1) / kThreads;
    constexpr int kRed = NB * RW * KW * V * 256;
    constexpr int kLds = 2 * KW * kPart > kRed ? 2 * KW * kPart : kRed;
    __shared__ __attribute__((aligned(16))) char lds[kLds];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave % RW, kw = wave / RW;
    const int n = lane & 15, q = lane >> 4;
    const int rg = min((int)blockIdx.x * RW + rw, a.row_groups - 1);
    const int64_t t0 = (int64_t)blockIdx.y * kRows;
    const int rounds = (a.col_tiles + KW - 1) / KW;

    // Staging: this thread's chunks of 8 columns, each of one token row and part.
    XOperand<XBF16> x[kPer];
    int64_t xat[kPer];
    int part_of[kPer], col_of[kPer], to[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int c = min((int)threadIdx.x + kThreads * i, kChunks - 1);
        const int part = c / (kRows * 16), r = c / 16 % kRows, k = c % 16;
        xat[i] = min(t0 + r, a.T - 1) * a.ldx;  // (rows past the last are computed and not stored)
        part_of[i] = part;
        col_of[i] = 8 * k;
        to[i] = part * kPart + r * 256 + ((k ^ (r & 15)) << 4);
    }
    auto load_x = [&](int round) {
#pragma unroll
        for (int i = 0; i < kPer; i++)  // (past the last column the token's last ones, which meet zero codes and scales)
            x[i].load(a.x, xat[i] + min((round * KW + part_of[i]) * 128 + col_of[i], a.cols - 8));
    };
    auto stage_x = [&](char* l) {
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            bf16x8 t[kTerms];
            x[i].terms(t);
            if (kChunks % kThreads == 0 || threadIdx.x + kThreads * i < kChunks)
#pragma unroll
                for (int c = 0; c < kTerms; c++) *(bf16x8*)(l + to[i] + c * kPlane) = t[c];
        }
    };

    struct Tile {
        uint4 code[NB];
        uint16_t scale[NB][S];
        uint8_t zero[NB][S];
    };
    auto load_w = [&](int round, Tile& t) {
        const int kt = round * KW + kw;
#pragma unroll
        for (int b = 0; b < NB; b++) {
            const QuantView& w = a.w[b];
            const int64_t tile = (int64_t)rg * a.col_tiles + min(kt, a.col_tiles - 1);
            t.code[b] = w.codes[tile * 64 + lane];
            __builtin_memcpy(t.scale[b], __builtin_assume_aligned(w.scales + (tile * 16 + n) * S, 2 * S), 2 * S);
            if (w.zeros) __builtin_memcpy(t.zero[b], __builtin_assume_aligned(w.zeros + (tile * 16 + n) * S, S), S);
            if (kt >= a.col_tiles) {  // a part past the last tile: scales of zero
#pragma unroll
                for (int g = 0; g < S; g++) t.scale[b][g] = 0;
            }
        }
    };

    bf16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; i++) ones[i] = (__bf16)1.0f;
    f32x4 out[NB][MT];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int m = 0; m < MT; m++) out[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};

    Tile cur, nxt;
    load_x(0);
    load_w(0, cur);
    for (int round = 0; round < rounds; round++) {
        char* l = lds + (round & 1) * (KW * kPart);
        stage_x(l);
        if (round + 1 < rounds) {
            load_x(round + 1);
            load_w(round + 1, nxt);
        }
        lds_barrier();
        const char* mine = l + kw * kPart;
        f32x4 acc[NB][MT], xs[MT];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j % (4 / S) == 0) {
#pragma unroll
                for (int m = 0; m < MT; m++) {
                    xs[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int b = 0; b < NB; b++) acc[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            }
            bf16x8 w[NB];
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const uint4 c = cur.code[b];
                const uint32_t word = j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w;
                const float z = a.w[b].zeros ? (float)cur.zero[b][j / (4 / S)] : 8.f;
                w[b] = XBF16 ? codes_bf16(word) : codes_less_zero(word, z);
            }
#pragma unroll
            for (int c = kTerms - 1; c >= 0; c--)
#pragma unroll
                for (int m = 0; m < MT; m++) {
                    const bf16x8 xt = *(const bf16x8*)(mine + c * kPlane + (16 * m + n) * 256 + (((4 * j + q) ^ n) << 4));
                    if constexpr (XBF16) xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xt, ones, xs[m], 0, 0, 0);
#pragma unroll
                    for (int b = 0; b < NB; b++)
                        acc[b][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xt, w[b], acc[b][m], 0, 0, 0);
                }
            if (j % (4 / S) == 4 / S - 1) {
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const float s = f16_bits_to_f32(cur.scale[b][j / (4 / S)]);
                    const float z = a.w[b].zeros ? 16.f + (float)cur.zero[b][j / (4 / S)] : 24.f;
#pragma unroll
                    for (int m = 0; m < MT; m++)
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            out[b][m][i] = fmaf(s, XBF16 ? fmaf(-z, xs[m][i], acc[b][m][i]) : acc[b][m][i], out[b][m][i]);
                }
            }
        }
        cur = nxt;
    }

    // The parts' sums in part order.
    __syncthreads();
    float* red = (float*)lds;  // [NB][KW][RW][V][64]
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int i = 0; i < 4; i++) red[(((b * KW + kw) * RW + rw) * V + m * 4 + i) * 64 + lane] = out[b][m][i];
    __syncthreads();
    for (int v = threadIdx.x; v < RW * V * 64; v += kThreads) {
        float sum[NB];
#pragma unroll
        for (int b = 0; b < NB; b++) {
            sum[b] = red[b * KW * RW * V * 64 + v];
#pragma unroll
            for (int w = 1; w < KW; w++) sum[b] += red[(b * KW + w) * RW * V * 64 + v];
        }
        const int l = v & 63, mi = v / 64 % V, r = v / (V * 64);
        const int64_t t = t0 + (16 * (mi / 4) + 4 * (l >> 4) + mi % 4);
        const int64_t row = ((int64_t)blockIdx.x * RW + r) * 16 + (l & 15);
        if (t < a.T && row < a.rows) {
            const float y = GATED ? silu(sum[0]) * sum[NB - 1] : sum[0];
            if (a.y_bf16) ((__bf16*)a.y)[t * a.ldy + row] = (__bf16)y;
            else ((float*)a.y)[t * a.ldy + row] = y;
        }
    }
}

template <bool XBF16, int MT, int RW, int KW, bool GATED>
hipError_t launch_shared(const LinearArgs& a, hipStream_t s) {
    constexpr int tokens = 16 * MT;
    const dim3 grid((a.row_groups + RW - 1) / RW, (unsigned)((a.T + tokens - 1) / tokens)), block(64 * RW * KW);
    if (a.group == 32) hipLaunchKernelGGL((shared_rows_kernel<XBF16, MT, RW, KW, 4, GATED>), grid, block, 0, s, a);
    else if (a.group == 64) hipLaunchKernelGGL((shared_rows_kernel<XBF16, MT, RW, KW, 2, GATED>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((shared_rows_kernel<XBF16, MT, RW, KW, 1, GATED>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <bool XBF16, int TI, int R, bool GATED>
hipError_t launch_rows(const LinearArgs& a, int waves, hipStream_t s) {
    const dim3 grid((a.row_groups + R - 1) / R), block(64 * waves);
    const size_t lds = (size_t)(GATED ? 2 : 1) * waves * TI * 64 * sizeof(float);
    if (a.group == 32) hipLaunchKernelGGL((rows_kernel<XBF16, TI, R, 4, GATED>), grid, block, lds, s, a);
    else if (a.group == 64) hipLaunchKernelGGL((rows_kernel<XBF16, TI, R, 2, GATED>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((rows_kernel<XBF16, TI, R, 1, GATED>), grid, block, lds, s, a);
    return hipGetLastError();
}

// Measured (us; bf16 x unless said, 4-bit matrices):
//   one token, 100003 x 4096: two row groups a wave and 4 waves 38.5, one and 8
//     waves 47; 2048 x 2048: 5.2 and 3.8.  Two once the groups fill the GPU
//     16 times over.
//   13 tokens in fp32, 6007 x 5184: two row groups a wave, for one conversion
//     of x, 17, one 22; 3 tokens 4096 x 4096: 12 and 10.
//   24 tokens, gated 10240 x 4096: x shared (4 row groups, 4 parts) 26, a wave
//     for itself 32; 9 tokens, 8192 x 2048: 12 and 8.
//   64 tokens, 4096 x 4096: 2 row groups and 4 parts 15, 4 and 2 23; 37 tokens,
//     gated 10240 x 4096: 50 and 41: fewer parts once the workgroups fill half
//     the CUs.
inline DensePlan rows_plan(const LinearArgs& a) {
    if (a.T <= 16) {
        const bool two = a.x_bf16 ? a.T <= 4 && a.row_groups >= 4096 : a.T > 4 && a.row_groups >= 256;
        const int most = a.x_bf16 && two ? 4 : 8;
        int waves = 1;
        while (waves < most && waves < a.col_tiles) waves *= 2;
        return {MOE_PLAN_ROWS, a.T <= 4 ? 4 : 16, two ? 32 : 16, waves, 1, 1, 0};
    }
    if (!a.x_bf16) return {MOE_PLAN_SHARED_ROWS, 32, 64, 2, 1, 1, 0};
    if (a.T <= 32) return {MOE_PLAN_SHARED_ROWS, 32, 64, 4, 1, 1, 0};
    const bool few = (a.row_groups + 3) / 4 * ((a.T + 63) / 64) <= 128;
    return {MOE_PLAN_SHARED_ROWS, a.T <= 48 ? 48 : 64, few ? 32 : 64, few ? 4 : 2, 1, 1, 0};
}

template <bool XBF16, bool GATED>
hipError_t launch_rows_t(const LinearArgs& a, const DensePlan& p, hipStream_t s) {
    if constexpr (XBF16) {
        if (p.tokens == 4) return p.rows == 32 ? launch_rows<true, 1, 2, GATED>(a, p.parts, s) : launch_rows<true, 1, 1, GATED>(a, p.parts, s);
        if (p.tokens == 16) return launch_rows<true, 4, 1, GATED>(a, p.parts, s);
        if (p.tokens == 32) return launch_shared<true, 2, 4, 4, GATED>(a, s);
        if (p.tokens == 48) return p.rows == 32 ? launch_shared<true, 3, 2, 4, GATED>(a, s) : launch_shared<true, 3, 4, 2, GATED>(a, s);
        return p.rows == 32 ? launch_shared<true, 4, 2, 4, GATED>(a, s) : launch_shared<true, 4, 4, 2, GATED>(a, s);
    } else {
        if (p.tokens == 4) return launch_rows<false, 1, 1, GATED>(a, p.parts, s);
        if (p.tokens == 16) return p.rows == 32 ? launch_rows<false, 4, 2, GATED>(a, p.parts, s) : launch_rows<false, 4, 1, GATED>(a, p.parts, s);
        return launch_shared<false, 2, 4, 2, GATED>(a, s);
    }
}

}  // namespace linear

// One translation unit each (linear_bf16.hip, linear_f32.hip).
hipError_t launch_linear_rows_bf16(const LinearArgs& a, bool gated, const DensePlan& p, hipStream_t s);
hipError_t launch_linear_rows_f32(const LinearArgs& a, bool gated, const DensePlan& p, hipStream_t s);

}  // namespace moe
