// Attention over packed sequences, forward:
//   S = scale Q K^T,  P = softmax of each row over the keys that it sees,  O = P V.
// One pass over the keys with a running maximum and sum.
#pragma once

#include "attention_tiles.h"

namespace moe {
namespace packed {

constexpr int kForwardWaves = 4;
template <bool BF16, int D> struct ForwardShape {
    static constexpr int kWaves = kForwardWaves;
    static constexpr int kRows = 32 * kWaves;              // a wave has 32 rows
    static constexpr int kKeys = BF16 && D <= 128 ? 64 : 32;  // of a tile
    static constexpr int kTileBytes = kKeys * Tile<BF16, D>::kLineBytes;
    static constexpr int kLds = 4 * kTileBytes;            // keys and values, double
};

template <bool BF16, int D>
__global__ __launch_bounds__(kForwardWaves * 64) void attention_kernel(PackedArgs a) {
    typedef ForwardShape<BF16, D> F;
    typedef Tile<BF16, D> T;
    constexpr int kThreads = F::kWaves * 64, BK = F::kKeys, KK = D / 16, DB = D / 32, KB = BK / 32;
    __shared__ __attribute__((aligned(1024))) char lds[F::kLds];
    __shared__ int odd_tile[2];  // the last tile whose values are not all finite, by buffer
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;

    // key heads first, so that workgroups that go to one XCD share keys and values;
    // then the query heads of a key head; a sequence's last tiles, which see most, first
    const int kv_head = blockIdx.x % a.kv_heads, rest = blockIdx.x / a.kv_heads;
    const int head = kv_head * a.per_head + rest % a.per_head;
    if (blockIdx.x == gridDim.x - 1) {
        check_offsets(a.offsets_q, a.n, a.Tq, a.err);
        check_offsets(a.offsets_k, a.n, a.Tk, a.err);
    }
    int seq, local;
    if (!find_tile<F::kRows>(a.offsets_q, a.n, a.Tq, rest / a.per_head, &seq, &local)) return;
    const Sequence s = sequence_of(a, seq);
    const int tiles = (s.rows + F::kRows - 1) / F::kRows;
    if (local >= tiles) return;
    const int row0 = (tiles - 1 - local) * F::kRows, row = row0 + wave * 32 + (lane & 31);
    const bool live = row < s.rows;
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

    Fragment<BF16> q[KK];
    const int64_t line = (int64_t)(s.q0 + row) * a.ldq + (int64_t)head * D;
#pragma unroll
    for (int kk = 0; kk < KK; kk++) {
        along_memory<BF16>(a.q, line, live, kk, lane, q[kk]);
        q[kk].split();
    }
    f32x16 out[DB];
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) out[d][i] = 0;
    float m = -kInf, l = 0;  // of the row: m the largest q.k so far; l this lane's part of the sum

    // keys that any of the workgroup's rows, and of the wave's, sees
    const int last_row = min(row0 + F::kRows, s.rows) - 1;
    const int end = a.causal ? min(s.keys, last_row + s.shift + 1) : s.keys;
    const int begin = a.window ? max(0, row0 + s.shift - a.window + 1) / BK * BK : 0;
    const int wave_first = row0 + wave * 32, wave_last = min(wave_first + 31, s.rows - 1);

    const char* kbase = (const char*)a.k + ((int64_t)s.k0 * a.ldk + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    const char* vbase = (const char*)a.v + ((int64_t)s.k0 * a.ldv + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    auto masked_tile = [&](int k0) {  // for some row of the workgroup
        return k0 + BK > s.keys || (a.causal && k0 + BK - 1 > row0 + s.shift) || (a.window && k0 <= last_row + s.shift - a.window);
    };
    Staged<BF16, D, BK, kThreads> sk, sv;
    auto put = [&](int k0, int buffer) {
        sk.store(lds + 2 * buffer * F::kTileBytes);
        sv.store(lds + (2 * buffer + 1) * F::kTileBytes);
        if (masked_tile(k0) && sv.any_not_finite()) odd_tile[buffer] = k0;
    };
    if (threadIdx.x < 2) odd_tile[threadIdx.x] = -1;
    if (begin < end) {
        sk.load(kbase, a.ldk, begin, s.keys - begin);
        sv.load(vbase, a.ldv, begin, s.keys - begin);
        __syncthreads();
        put(begin, 0);
    }
    __syncthreads();
    int buffer = 0;
    for (int k0 = begin; k0 < end; k0 += BK, buffer ^= 1) {
        const bool more = k0 + BK < end;
        if (more) {
            sk.load(kbase, a.ldk, k0 + BK, s.keys - k0 - BK);
            sv.load(vbase, a.ldv, k0 + BK, s.keys - k0 - BK);
        }
        const char* kt = lds + 2 * buffer * F::kTileBytes;
        const char* vt = kt + F::kTileBytes;
        const bool none = wave_first >= s.rows || (a.causal && k0 > wave_last + s.shift) || (a.window && k0 + BK - 1 <= wave_first + s.shift - a.window);
        if (!none) {
            f32x16 st[KB];
#pragma unroll
            for (int b = 0; b < KB; b++) {
#pragma unroll
                for (int i = 0; i < 16; i++) st[b][i] = 0;
#pragma unroll
                for (int kk = 0; kk < KK; kk++) {
                    Fragment<BF16> f;
                    T::along(kt, 32 * b, kk, lane, f);
                    f.split();
                    mma(st[b], f, q[kk]);
                }
            }
            const bool masked = k0 + BK > s.keys || (a.causal && k0 + BK - 1 > wave_first + s.shift) || (a.window && k0 <= wave_last + s.shift - a.window);
            if (masked) {
#pragma unroll
                for (int b = 0; b < KB; b++)
#pragma unroll
                    for (int i = 0; i < 16; i++)
                        if (!sees(a, s, row, k0 + 32 * b + reg_line(i, h))) st[b][i] = -kInf;
            }
            float top = st[0][0];
#pragma unroll
            for (int b = 0; b < KB; b++)
#pragma unroll
                for (int i = 0; i < 16; i++) top = fmaxf(top, st[b][i]);
            const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
            top = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
            const float before = m;
            m = fmaxf(m, top);
            const float base = m == -kInf ? 0.f : m * a.scale_log2;
            if (__any(m != before)) {
                const float f = __builtin_amdgcn_exp2f(fmaf(before, a.scale_log2, -base));
                l *= f;
#pragma unroll
                for (int d = 0; d < DB; d++) out[d] *= f;
            }
            float sum = 0;
#pragma unroll
            for (int b = 0; b < KB; b++)
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    st[b][i] = __builtin_amdgcn_exp2f(fmaf(st[b][i], a.scale_log2, -base));
                    sum += st[b][i];
                }
            l += sum;
            const bool odd = masked && odd_tile[buffer] == k0;
#pragma unroll
            for (int b = 0; b < KB; b++)
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    float p[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) p[e] = st[b][8 * g + e];
                    Fragment<BF16> pf;
                    operand_of(p, pf);
                    if (odd) {
                        bf16x8 seen;
#pragma unroll
                        for (int e = 0; e < 8; e++) seen[e] = (__bf16)(sees(a, s, row, k0 + 32 * b + reg_line(8 * g + e, h)) ? 1.f : 0.f);
#pragma unroll
                        for (int d = 0; d < DB; d++) {
                            Fragment<BF16> f;
                            T::across(vt, 32 * b + 16 * g, 32 * d, lane, f);
                            mma_seen(out[d], f, pf, seen);
                        }
                    } else {
#pragma unroll
                        for (int d = 0; d < DB; d++) {
                            Fragment<BF16> f;
                            T::across(vt, 32 * b + 16 * g, 32 * d, lane, f);
                            f.split();
                            mma(out[d], f, pf);
                        }
                    }
                }
        }
        if (more) put(k0 + BK, buffer ^ 1);
        __syncthreads();
    }
    if (!live) return;
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    // a row that sees nothing: 0, and minus infinity
    const float nan = __uint_as_float(0x7FC00000u), by = s.bad ? nan : m == -kInf && l == 0.f ? 0.f : 1.0f / l;
    const int64_t o = (int64_t)(s.q0 + row) * a.ldo + (int64_t)head * D;
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) store1<BF16>(a.out, o + 32 * d + 8 * j + 4 * h + e, out[d][4 * j + e] * by);
    if (a.lse && h == 0) a.lse[(int64_t)(s.q0 + row) * a.q_heads + head] = s.bad ? nan : m == -kInf ? -kInf : fmaf(m, a.scale, __builtin_amdgcn_logf(l) * kLn2);
}

template <bool BF16, int D>
hipError_t launch_forward(const PackedArgs& a, hipStream_t s) {
    typedef ForwardShape<BF16, D> F;
    const int64_t groups = tile_slots(a.Tq, F::kRows, a.n) * a.q_heads;
    hipLaunchKernelGGL((attention_kernel<BF16, D>), dim3((unsigned)groups), dim3(F::kWaves * 64), 0, s, a);
    return hipGetLastError();
}
template <bool BF16>
hipError_t launch_forward_by_width(const PackedArgs& a, hipStream_t s) {
    switch (a.D) {
        case 64: return launch_forward<BF16, 64>(a, s);
        case 96: return launch_forward<BF16, 96>(a, s);
        case 128: return launch_forward<BF16, 128>(a, s);
        case 192: return launch_forward<BF16, 192>(a, s);
        default: return launch_forward<BF16, 256>(a, s);
    }
}

}  // namespace packed
}  // namespace moe
