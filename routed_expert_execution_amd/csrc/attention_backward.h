// Attention over packed sequences, backward, from the rows' log sums of
// exponentials L and the outputs O that the forward pass has kept:
//   P = exp(scale Q K^T - L),  dV = P^T dO,  dP = dO V^T,  delta = rowsum(dO O),
//   dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q.
// Two kernels, each with results of its own rows only, so that sums have one order
// and nothing is added in memory: dQ over tiles of queries, dK and dV over tiles of
// keys (with all query heads of the key head).  S and dP are computed in both: seven
// products in place of five.
#pragma once

#include "attention_tiles.h"

namespace moe {
namespace packed {

constexpr int kBackwardWaves = 4;
template <bool BF16, int D> struct BackwardShape {
    static constexpr int kThreads = 64 * kBackwardWaves;
    static constexpr int kRows = 32 * kBackwardWaves;       // of a workgroup's own tile, 32 a wave
    static constexpr int kOther = BF16 && D <= 128 ? 64 : 32;  // of a tile that it passes over
    static constexpr int kTileBytes = kOther * Tile<BF16, D>::kLineBytes;
};

// dQ, and delta for the other kernel.  As the forward kernel: S^T = K Q^T and
// dP^T = V dO^T with a row a lane, dQ^T = K^T dS^T.
template <bool BF16, int D>
__global__ __launch_bounds__(kBackwardWaves * 64) void attention_dq_kernel(PackedArgs a) {
    typedef BackwardShape<BF16, D> B;
    typedef Tile<BF16, D> T;
    constexpr int BK = B::kOther, KK = D / 16, DB = D / 32, KB = BK / 32;
    __shared__ __attribute__((aligned(1024))) char lds[4 * B::kTileBytes];
    __shared__ int odd_tile[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    const int kv_head = blockIdx.x % a.kv_heads, rest = blockIdx.x / a.kv_heads;
    const int head = kv_head * a.per_head + rest % a.per_head;
    if (blockIdx.x == gridDim.x - 1) {
        check_offsets(a.offsets_q, a.n, a.Tq, a.err);
        check_offsets(a.offsets_k, a.n, a.Tk, a.err);
    }
    int seq, local;
    if (!find_tile<B::kRows>(a.offsets_q, a.n, a.Tq, rest / a.per_head, &seq, &local)) return;
    const Sequence s = sequence_of(a, seq);
    const int tiles = (s.rows + B::kRows - 1) / B::kRows;
    if (local >= tiles) return;
    const int row0 = (tiles - 1 - local) * B::kRows, row = row0 + wave * 32 + (lane & 31);
    const bool live = row < s.rows;
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

    Fragment<BF16> q[KK], g[KK];
    const int64_t token = s.q0 + row;
    float delta = 0;
#pragma unroll
    for (int kk = 0; kk < KK; kk++) {
        along_memory<BF16>(a.q, token * a.ldq + (int64_t)head * D, live, kk, lane, q[kk]);
        along_memory<BF16>(a.dout, token * a.lddo + (int64_t)head * D, live, kk, lane, g[kk]);
        Fragment<BF16> o;
        along_memory<BF16>(a.out, token * a.ldo + (int64_t)head * D, live, kk, lane, o);
#pragma unroll
        for (int e = 0; e < 8; e++) delta = fmaf((float)g[kk].raw[e], (float)o.raw[e], delta);
        q[kk].split();
        g[kk].split();
    }
    {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(delta), __float_as_uint(delta), false, false);
        delta = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    float lse = kInf;  // (a row past the last: P = 0)
    if (live) {
        lse = a.lse[token * a.q_heads + head] * kLog2e;
        if (h == 0) a.delta[token * a.q_heads + head] = delta;
    }
    f32x16 out[DB];
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) out[d][i] = 0;

    const int last_row = min(row0 + B::kRows, s.rows) - 1;
    const int end = a.causal ? min(s.keys, last_row + s.shift + 1) : s.keys;
    const int begin = a.window ? max(0, row0 + s.shift - a.window + 1) / BK * BK : 0;
    const int wave_first = row0 + wave * 32, wave_last = min(wave_first + 31, s.rows - 1);
    const char* kbase = (const char*)a.k + ((int64_t)s.k0 * a.ldk + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    const char* vbase = (const char*)a.v + ((int64_t)s.k0 * a.ldv + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    auto masked_tile = [&](int k0) {
        return k0 + BK > s.keys || (a.causal && k0 + BK - 1 > row0 + s.shift) || (a.window && k0 <= last_row + s.shift - a.window);
    };
    Staged<BF16, D, BK, B::kThreads> sk, sv;
    auto put = [&](int k0, int buffer) {
        sk.store(lds + 2 * buffer * B::kTileBytes);
        sv.store(lds + (2 * buffer + 1) * B::kTileBytes);
        if (masked_tile(k0) && sk.any_not_finite()) odd_tile[buffer] = k0;
    };
    if (threadIdx.x < 2) odd_tile[threadIdx.x] = -1;
    if (begin < end) {
        sk.load(kbase, a.ldk, begin, s.keys - begin);
        sv.load(vbase, a.ldv, begin, s.keys - begin);
        __syncthreads();
        put(begin, 0);
    }
    __syncthreads();
    const uint32_t along_lane = T::along_lane(lane), across_lane = T::across_lane(lane);
    int buffer = 0;
    for (int k0 = begin; k0 < end; k0 += BK, buffer ^= 1) {
        const bool more = k0 + BK < end;
        if (more) {
            sk.load(kbase, a.ldk, k0 + BK, s.keys - k0 - BK);
            sv.load(vbase, a.ldv, k0 + BK, s.keys - k0 - BK);
        }
        const char* kt = lds + 2 * buffer * B::kTileBytes;
        const char* vt = kt + B::kTileBytes;
        const uint32_t ka = tile::lds_address(kt) + along_lane, va = tile::lds_address(vt) + along_lane, kx = tile::lds_address(kt) + across_lane;
        const bool none = wave_first >= s.rows || (a.causal && k0 > wave_last + s.shift) || (a.window && k0 + BK - 1 <= wave_first + s.shift - a.window);
        if (!none) {
            const bool masked = k0 + BK > s.keys || (a.causal && k0 + BK - 1 > wave_first + s.shift) || (a.window && k0 <= wave_last + s.shift - a.window);
            const bool odd = masked && odd_tile[buffer] == k0;
            const Span span = keys_seen(a, s, row, k0, h);
#pragma unroll
            for (int b = 0; b < KB; b++) {
                f32x16 st, dp;
#pragma unroll
                for (int i = 0; i < 16; i++) st[i] = dp[i] = 0;
#pragma unroll
                for (int kk = 0; kk < KK; kk++) {
                    Fragment<BF16> f;
                    T::along(ka, 32 * b, kk, f);
                    f.split();
                    mma(st, f, q[kk]);
                    T::along(va, 32 * b, kk, f);
                    f.split();
                    mma(dp, f, g[kk]);
                }
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    const float ds = __builtin_amdgcn_exp2f(fmaf(st[i], a.scale_log2, -lse)) * (dp[i] - delta);
                    st[i] = masked && !span.has(b, i) ? 0.f : ds;
                }
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) v[e] = st[8 * n + e];
                    Fragment<BF16> df;
                    operand_of(v, df);
                    bf16x8 seen;
                    if (odd)
#pragma unroll
                        for (int e = 0; e < 8; e++) seen[e] = (__bf16)(span.has(b, 8 * n + e) ? 1.f : 0.f);
#pragma unroll
                    for (int d = 0; d < DB; d++) {
                        Fragment<BF16> f;
                        T::across(kx, 32 * b + 16 * n, 32 * d, f);
                        if (odd) {
                            mma_seen(out[d], f, df, seen);
                        } else {
                            f.split();
                            mma(out[d], f, df);
                        }
                    }
                }
            }
        }
        if (more) put(k0 + BK, buffer ^ 1);
        __syncthreads();
    }
    if (!live) return;
    const float by = s.bad ? __uint_as_float(0x7FC00000u) : a.scale;
    const int64_t o = token * a.lddq + (int64_t)head * D;
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) store1<BF16>(a.dq, o + 32 * d + 8 * j + 4 * h + e, out[d][4 * j + e] * by);
}

// dK and dV.  A wave has 32 keys as operands in registers and passes over the rows
// that see any of the workgroup's keys, of one query head after the other: S = Q K^T
// and dP = dO V^T with a key a lane, dV^T = dO^T P, dK^T = Q^T dS.
// WHAT: 3 both; 1 dV alone, 2 dK alone (where registers do not hold both).
template <bool BF16, int D, int WHAT>
__global__ __launch_bounds__(kBackwardWaves * 64) void attention_dkv_kernel(PackedArgs a) {
    typedef BackwardShape<BF16, D> B;
    typedef Tile<BF16, D> T;
    constexpr int BQ = B::kOther, KK = D / 16, DB = D / 32, RB = BQ / 32;
    constexpr bool kDv = WHAT & 1, kDk = WHAT & 2;
    __shared__ __attribute__((aligned(1024))) char lds[4 * B::kTileBytes];
    __shared__ __attribute__((aligned(16))) float row_lse[2][BQ], row_delta[2][BQ];
    __shared__ int odd_tile[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    const int kv_head = blockIdx.x % a.kv_heads;
    int seq, local;
    if (!find_tile<B::kRows>(a.offsets_k, a.n, a.Tk, blockIdx.x / a.kv_heads, &seq, &local)) return;
    const Sequence s = sequence_of(a, seq);
    const int key0 = local * B::kRows, wave_key = key0 + wave * 32, key = wave_key + (lane & 31);
    if (key0 >= s.keys) return;
    const bool live = key < s.keys;
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

    Fragment<BF16> k[KK], v[kDk ? KK : 1];
    const int64_t token = s.k0 + key;
#pragma unroll
    for (int kk = 0; kk < KK; kk++) {
        along_memory<BF16>(a.k, token * a.ldk + (int64_t)kv_head * D, live, kk, lane, k[kk]);
        if constexpr (kDk) along_memory<BF16>(a.v, token * a.ldv + (int64_t)kv_head * D, live, kk, lane, v[kk]);
    }
    f32x16 dk[kDk ? DB : 1], dv[kDv ? DB : 1];
#pragma unroll
    for (int i = 0; i < 16; i++) {
#pragma unroll
        for (int d = 0; d < (kDk ? DB : 1); d++) dk[d][i] = 0;
#pragma unroll
        for (int d = 0; d < (kDv ? DB : 1); d++) dv[d][i] = 0;
    }
    // rows that see any of the workgroup's keys
    const int last_key = min(key0 + B::kRows, s.keys) - 1;
    const int begin = a.causal ? max(0, key0 - s.shift) / BQ * BQ : 0;
    const int64_t end_row = a.window ? (int64_t)last_key - s.shift + a.window : s.rows;
    const int end = (int)min((int64_t)s.rows, end_row);
    const int per = end > begin ? (end - begin + BQ - 1) / BQ : 0, total = per * a.per_head;
    const int wave_last_key = min(wave_key + 31, s.keys - 1);
    auto row_of = [&](int t) { return begin + t % per * BQ; };
    auto masked_tile = [&](int r0) {
        return (a.causal && last_key > r0 + s.shift) || (a.window && key0 <= r0 + BQ - 1 + s.shift - a.window);
    };
    Staged<BF16, D, BQ, B::kThreads> sq, sg;
    float s_lse = 0, s_delta = 0;
    auto get = [&](int t) {
        const int r0 = row_of(t), head = kv_head * a.per_head + t / per;
        sq.load((const char*)a.q + ((int64_t)s.q0 * a.ldq + (int64_t)head * D) * (BF16 ? 2 : 4), a.ldq, r0, s.rows - r0);
        sg.load((const char*)a.dout + ((int64_t)s.q0 * a.lddo + (int64_t)head * D) * (BF16 ? 2 : 4), a.lddo, r0, s.rows - r0);
        if (threadIdx.x < BQ) {
            const int r = r0 + threadIdx.x;
            const int64_t at = (int64_t)(s.q0 + r) * a.q_heads + head;
            s_lse = r < s.rows ? a.lse[at] * kLog2e : kInf;  // (past the last row: P = 0)
            s_delta = r < s.rows ? a.delta[at] : 0.f;
        }
    };
    auto put = [&](int t, int buffer) {
        sq.store(lds + 2 * buffer * B::kTileBytes);
        sg.store(lds + (2 * buffer + 1) * B::kTileBytes);
        if (threadIdx.x < BQ) {
            row_lse[buffer][threadIdx.x] = s_lse;
            row_delta[buffer][threadIdx.x] = s_delta;
        }
        if (masked_tile(row_of(t)) && (sq.any_not_finite() || sg.any_not_finite())) odd_tile[buffer] = t;
    };
    if (threadIdx.x < 2) odd_tile[threadIdx.x] = -1;
    if (total) {
        get(0);
        __syncthreads();
        put(0, 0);
    }
    __syncthreads();
    const uint32_t along_lane = T::along_lane(lane), across_lane = T::across_lane(lane);
    for (int t = 0; t < total; t++) {
        const int buffer = t & 1, r0 = row_of(t);
        if (t + 1 < total) get(t + 1);
        const char* qt = lds + 2 * buffer * B::kTileBytes;
        const char* gt = qt + B::kTileBytes;
        const uint32_t qa = tile::lds_address(qt) + along_lane, ga = tile::lds_address(gt) + along_lane;
        const uint32_t qx = tile::lds_address(qt) + across_lane, gx = tile::lds_address(gt) + across_lane;
        const bool none = wave_key >= s.keys || (a.causal && wave_key > r0 + BQ - 1 + s.shift) || (a.window && wave_last_key <= r0 + s.shift - a.window);
        if (!none) {
            const bool masked = (a.causal && wave_last_key > r0 + s.shift) || (a.window && wave_key <= r0 + BQ - 1 + s.shift - a.window);
            const bool odd = masked && odd_tile[buffer] == t;
            const Span span = rows_seeing(a, s, key, r0, h);
#pragma unroll
            for (int b = 0; b < RB; b++) {
                f32x16 st, dp;
#pragma unroll
                for (int i = 0; i < 16; i++) st[i] = dp[i] = 0;
#pragma unroll
                for (int kk = 0; kk < KK; kk++) {
                    Fragment<BF16> f, o;
                    T::along(qa, 32 * b, kk, f);
                    f.split();
                    o = k[kk];
                    o.split();
                    mma(st, f, o);
                    if constexpr (kDk) {
                        T::along(ga, 32 * b, kk, f);
                        f.split();
                        o = v[kk];
                        o.split();
                        mma(dp, f, o);
                    }
                }
                float p[16];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const f32x4 lse = *(const f32x4*)&row_lse[buffer][32 * b + 8 * j + 4 * h], delta = *(const f32x4*)&row_delta[buffer][32 * b + 8 * j + 4 * h];
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int i = 4 * j + e;
                        const bool off = masked && !span.has(b, i);
                        p[i] = __builtin_amdgcn_exp2f(fmaf(st[i], a.scale_log2, -lse[e]));
                        const float ds = p[i] * (dp[i] - delta[e]);
                        p[i] = off ? 0.f : p[i];
                        st[i] = off ? 0.f : ds;
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    Fragment<BF16> pf, df;
                    float x[8];
                    bf16x8 seen;
                    if (odd)
#pragma unroll
                        for (int e = 0; e < 8; e++) seen[e] = (__bf16)(span.has(b, 8 * n + e) ? 1.f : 0.f);
                    if constexpr (kDv) {
#pragma unroll
                        for (int e = 0; e < 8; e++) x[e] = p[8 * n + e];
                        operand_of(x, pf);
                    }
                    if constexpr (kDk) {
#pragma unroll
                        for (int e = 0; e < 8; e++) x[e] = st[8 * n + e];
                        operand_of(x, df);
                    }
#pragma unroll
                    for (int d = 0; d < DB; d++) {
                        Fragment<BF16> f;
                        if constexpr (kDv) {
                            T::across(gx, 32 * b + 16 * n, 32 * d, f);
                            if (odd) {
                                mma_seen(dv[d], f, pf, seen);
                            } else {
                                f.split();
                                mma(dv[d], f, pf);
                            }
                        }
                        if constexpr (kDk) {
                            T::across(qx, 32 * b + 16 * n, 32 * d, f);
                            if (odd) {
                                mma_seen(dk[d], f, df, seen);
                            } else {
                                f.split();
                                mma(dk[d], f, df);
                            }
                        }
                    }
                }
            }
        }
        if (t + 1 < total) put(t + 1, buffer ^ 1);
        __syncthreads();
    }
    if (!live) return;
    const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int at = 32 * d + 8 * j + 4 * h + e;
                if constexpr (kDk) store1<BF16>(a.dk, token * a.lddk + (int64_t)kv_head * D + at, s.bad ? nan : dk[d][4 * j + e] * a.scale);
                if constexpr (kDv) store1<BF16>(a.dv, token * a.lddv + (int64_t)kv_head * D + at, s.bad ? nan : dv[d][4 * j + e]);
            }
}

template <bool BF16, int D>
hipError_t launch_backward(const PackedArgs& a, hipStream_t s) {
    typedef BackwardShape<BF16, D> B;
    const dim3 threads(B::kThreads);
    const int64_t q_groups = tile_slots(a.Tq, B::kRows, a.n) * a.q_heads, k_groups = tile_slots(a.Tk, B::kRows, a.n) * a.kv_heads;
    hipLaunchKernelGGL((attention_dq_kernel<BF16, D>), dim3((unsigned)q_groups), threads, 0, s, a);
    if constexpr (BF16 || D <= 128) {
        hipLaunchKernelGGL((attention_dkv_kernel<BF16, D, 3>), dim3((unsigned)k_groups), threads, 0, s, a);
    } else {
        hipLaunchKernelGGL((attention_dkv_kernel<BF16, D, 1>), dim3((unsigned)k_groups), threads, 0, s, a);
        hipLaunchKernelGGL((attention_dkv_kernel<BF16, D, 2>), dim3((unsigned)k_groups), threads, 0, s, a);
    }
    return hipGetLastError();
}
template <bool BF16>
hipError_t launch_backward_by_width(const PackedArgs& a, hipStream_t s) {
    switch (a.D) {
        case 64: return launch_backward<BF16, 64>(a, s);
        case 96: return launch_backward<BF16, 96>(a, s);
        case 128: return launch_backward<BF16, 128>(a, s);
        case 192: return launch_backward<BF16, 192>(a, s);
        default: return launch_backward<BF16, 256>(a, s);
    }
}

}  // namespace packed
}  // namespace moe
