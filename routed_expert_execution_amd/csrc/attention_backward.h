// Attention over packed sequences, backward, from the rows' log sums of
// exponentials L and the outputs O that the forward pass has kept:
//   P = exp(scale Q K^T - L),  dV = P^T dO,  dP = dO V^T,  delta = rowsum(dO O),
//   dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q.
// In bf16 P and dS are rounded to bf16 for the second products: the gradients are 0.0023 off,
// their own rounding being 0.0017.  Two terms of both, in the steady loops, take 616 us for
// 489 (four sequences of up to 4096 tokens, 16 and 4 heads of 128); who needs them whole
// calls in fp32.
// delta first, then one launch of workgroups with results of their own rows only, so that
// sums have one order and nothing is added in memory: dQ over tiles of queries, dK and dV
// over tiles of keys (with all query heads of the key head).  S and dP are computed in
// each: seven or eight products in place of five.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attention_parts.h"

namespace moe {
namespace packed {

// fp32, and bf16 heads of more than 128 channels, by PartsShape.  Two sequences of 611 and
// 54 tokens, 6 and 3 heads of 96 in fp32: 65 us (one launch after the other, dK and dV
// together: 123), ten steps one after the other, of whose 4 us the products take 1.5.  fp32
// heads of 192 and 256 channels spill (361 and 882 registers), of 96 with ROLES 1 a few (42).
// What the others need of each row: L / ln 2 and delta = rowsum(dO O), by 16 or 32 lanes a
// row.  Bound by bytes: 8532 rows of 16 heads of 128 in bf16 18 us.
constexpr int kRowsThreads = 256;
template <bool BF16, int D>
__global__ __launch_bounds__(kRowsThreads) void attention_rows_kernel(PackedArgs a) {
    constexpr int kLanes = D <= 128 ? 16 : 32, kRows = kRowsThreads / kLanes;
    const int c = threadIdx.x % kLanes;
    // (rows of no sequence are not read)
    const int64_t from = (int64_t)clamp_to(a.offsets_q[0], a.Tq) * a.q_heads, to = (int64_t)clamp_to(a.offsets_q[a.n], a.Tq) * a.q_heads;
    for (int64_t first = from + (int64_t)blockIdx.x * kRows; first < to; first += (int64_t)gridDim.x * kRows) {
        const int64_t at = first + threadIdx.x / kLanes, token = at / a.q_heads;
        const int head = (int)(at - token * a.q_heads);
        float delta = 0;
        if (at < to && c < D / 8) {
            float o[8], g[8];
            load8<BF16>(a.out, token * a.ldo + (int64_t)head * D + 8 * c, o);
            load8<BF16>(a.dout, token * a.lddo + (int64_t)head * D + 8 * c, g);
#pragma unroll
            for (int e = 0; e < 8; e++) delta = fmaf(g[e], o[e], delta);
        }
        delta = seg_sum<kLanes>(delta);
        if (at < to && c == 0) a.rows[(int64_t)head * a.Tq + token] = make_float2(a.lse[at] * kLog2e, delta);
    }
}

// dQ: S^T = K Q^T and dP^T = V dO^T with a row a lane,
// dQ^T = K^T dS^T.
template <bool BF16, int D, bool DIRECT>
__device__ inline void attention_dq_parts(const PackedArgs& a, int group, char* lds, int& odd_tile) {
    typedef PartsShape<BF16, D> B;
    typedef Tile<BF16, D> T;
    constexpr int BK = B::kOther, KK = D / 16, DB = D / 32;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    const int block = wave % B::kBlocks, part = wave / B::kBlocks;
    const int kv_head = group % a.kv_heads, rest = group / a.kv_heads;
    const int head = kv_head * a.per_head + rest % a.per_head;
    int seq, local;
    if (!find_tile<B::kOwn>(a.offsets_q, a.n, a.Tq, rest / a.per_head, &seq, &local)) return;
    const Sequence s = sequence_of(a, seq);
    const int tiles = (s.rows + B::kOwn - 1) / B::kOwn;
    if (local >= tiles) return;
    const int row0 = (tiles - 1 - local) * B::kOwn, wave_first = row0 + block * 32, row = wave_first + (lane & 31);
    const bool live = row < s.rows;
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

    Fragment<BF16> q[KK], g[KK];
    const int64_t token = s.q0 + row;
    float2 of_row = make_float2(kInf, 0.f);  // (a row past the last: P = 0)
    if (live) of_row = a.rows[(int64_t)head * a.Tq + token];
    const float lse = of_row.x, delta = of_row.y;
#pragma unroll
    for (int kk = 0; kk < KK; kk++) {
        along_memory<BF16>(a.q, token * a.ldq + (int64_t)head * D, live, kk, lane, q[kk]);
        along_memory<BF16>(a.dout, token * a.lddo + (int64_t)head * D, live, kk, lane, g[kk]);
        q[kk].split();
        g[kk].split();
    }
    f32x16 out[DB];
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) out[d][i] = 0;

    const int last_row = min(row0 + B::kOwn, s.rows) - 1, wave_last = min(wave_first + 31, s.rows - 1);
    const int end = a.causal ? min(s.keys, last_row + s.shift + 1) : s.keys;
    const int begin = a.window ? max(0, row0 + s.shift - a.window + 1) / 32 * 32 : 0;
    const char* kbase = (const char*)a.k + ((int64_t)s.k0 * a.ldk + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    const char* vbase = (const char*)a.v + ((int64_t)s.k0 * a.ldv + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    char *kt = lds, *vt = lds + B::kTileBytes;
    const uint32_t ka = tile::lds_address(kt) + T::along_lane(lane) + part * 32 * T::kLineBytes, va = ka + B::kTileBytes;
    const uint32_t kx = tile::lds_address(kt) + T::across_lane(lane) + part * 32 * T::kLineBytes;
    if (threadIdx.x == 0) odd_tile = -1;
#pragma unroll 1
    for (int t0 = begin; t0 < end; t0 += BK) {
        __syncthreads();
        bring<BF16, D, BK, DIRECT>(kbase, a.ldk, t0, s.keys - t0, kt);
        bring<BF16, D, BK, DIRECT>(vbase, a.ldv, t0, s.keys - t0, vt);
        meet<DIRECT>();
        if (t0 + BK > s.keys || (a.causal && t0 + BK - 1 > row0 + s.shift) || (a.window && t0 <= last_row + s.shift - a.window)) {
            if (tile_not_finite<BF16, D, BK, kPartsThreads>(kt)) odd_tile = t0;
            __syncthreads();
        }
        const int k0 = t0 + 32 * part;  // this wave's 32 keys
        if (k0 >= s.keys || wave_first >= s.rows || (a.causal && k0 > wave_last + s.shift) || (a.window && k0 + 31 <= wave_first + s.shift - a.window)) continue;
        const bool masked = k0 + 32 > s.keys || (a.causal && k0 + 31 > wave_first + s.shift) || (a.window && k0 <= wave_last + s.shift - a.window);
        const bool odd = masked && odd_tile == t0;
        const Span span = keys_seen(a, s, row, k0, h);
        f32x16 st, dp;
#pragma unroll
        for (int i = 0; i < 16; i++) st[i] = dp[i] = 0;
        in_turn<2 * KK, BF16>([&](int i, Fragment<BF16>& f) { T::along(i & 1 ? va : ka, 0, i / 2, f); },
                              [&](int i, const Fragment<BF16>& f) { mma(i & 1 ? dp : st, f, i & 1 ? g[i / 2] : q[i / 2]); });
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const float ds = __builtin_amdgcn_exp2f(fmaf(st[i], a.scale_log2, -lse)) * (dp[i] - delta);
            st[i] = masked && !span.has(0, i) ? 0.f : ds;
        }
        Fragment<BF16> df[2];
#pragma unroll
        for (int n = 0; n < 2; n++) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; e++) v[e] = st[8 * n + e];
            operand_of(v, df[n]);
        }
        if (!odd) {
            in_turn<2 * DB, BF16>([&](int i, Fragment<BF16>& f) { T::across(kx, 16 * (i / DB), 32 * (i % DB), f); },
                                  [&](int i, const Fragment<BF16>& f) { mma(out[i % DB], f, df[i / DB]); });
            continue;
        }
#pragma unroll
        for (int n = 0; n < 2; n++) {
            bf16x8 seen;
#pragma unroll
            for (int e = 0; e < 8; e++) seen[e] = (__bf16)(span.has(0, 8 * n + e) ? 1.f : 0.f);
#pragma unroll
            for (int d = 0; d < DB; d++) {
                Fragment<BF16> f;
                T::across(kx, 16 * n, 32 * d, f);
                mma_seen(out[d], f, df[n], seen);
                if (!BF16) __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if (!add_parts<DB, B::kParts, B::kBlocks>(out, lds, part, block, lane) || !live) return;
    const float by = s.bad ? __uint_as_float(0x7FC00000u) : a.scale;
    const int64_t o = token * a.lddq + (int64_t)head * D;
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) store1<BF16>(a.dq, o + 32 * d + 8 * j + 4 * h + e, out[d][4 * j + e] * by);
}

// dK and dV: a wave has 32 keys as operands in registers and passes over the rows that
// see any of the workgroup's keys, of one query head after the other: S = Q K^T and
// dP = dO V^T with a key a lane, dV^T = dO^T P, dK^T = Q^T dS.
// WHAT: 3 both; 1 dV alone, 2 dK alone (where registers do not hold both).
template <bool BF16, int D, int WHAT, bool DIRECT>
__device__ inline void attention_dkv_parts(const PackedArgs& a, int group, char* lds, float2* stats, int& odd_tile) {
    typedef PartsShape<BF16, D> B;
    typedef Tile<BF16, D> T;
    constexpr int BQ = B::kOther, KK = D / 16, DB = D / 32;
    constexpr bool kDv = WHAT & 1, kDk = WHAT & 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    const int block = wave % B::kBlocks, part = wave / B::kBlocks;
    const int kv_head = group % a.kv_heads;
    int seq, local;
    if (!find_tile<B::kOwn>(a.offsets_k, a.n, a.Tk, group / a.kv_heads, &seq, &local)) return;
    const Sequence s = sequence_of(a, seq);
    const int key0 = local * B::kOwn, wave_key = key0 + block * 32, key = wave_key + (lane & 31);
    if (key0 >= s.keys) return;
    const bool live = key < s.keys;
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

    Fragment<BF16> k[KK], v[kDk ? KK : 1];
    const int64_t token = s.k0 + key;
#pragma unroll
    for (int kk = 0; kk < KK; kk++) {
        along_memory<BF16>(a.k, token * a.ldk + (int64_t)kv_head * D, live, kk, lane, k[kk]);
        k[kk].split();
        if constexpr (kDk) {
            along_memory<BF16>(a.v, token * a.ldv + (int64_t)kv_head * D, live, kk, lane, v[kk]);
            v[kk].split();
        }
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
    const int last_key = min(key0 + B::kOwn, s.keys) - 1, wave_last_key = min(wave_key + 31, s.keys - 1);
    const int begin = a.causal ? max(0, key0 - s.shift) / 32 * 32 : 0;
    const int end = (int)min((int64_t)s.rows, a.window ? (int64_t)last_key - s.shift + a.window : s.rows);
    char *qt = lds, *gt = lds + B::kTileBytes;
    const uint32_t qa = tile::lds_address(qt) + T::along_lane(lane) + part * 32 * T::kLineBytes, ga = qa + B::kTileBytes;
    const uint32_t qx = tile::lds_address(qt) + T::across_lane(lane) + part * 32 * T::kLineBytes, gx = qx + B::kTileBytes;
    if (threadIdx.x == 0) odd_tile = -1;
    int at = 0;  // a number for each tile
#pragma unroll 1
    for (int head = kv_head * a.per_head; head < (kv_head + 1) * a.per_head; head++)
#pragma unroll 1
        for (int t0 = begin; t0 < end; t0 += BQ, at++) {
            __syncthreads();
            bring<BF16, D, BQ, DIRECT>((const char*)a.q + ((int64_t)s.q0 * a.ldq + (int64_t)head * D) * (BF16 ? 2 : 4), a.ldq, t0, s.rows - t0, qt);
            bring<BF16, D, BQ, DIRECT>((const char*)a.dout + ((int64_t)s.q0 * a.lddo + (int64_t)head * D) * (BF16 ? 2 : 4), a.lddo, t0, s.rows - t0, gt);
            if (threadIdx.x < BQ) {
                const int r = t0 + threadIdx.x;  // (past the last row: P = 0)
                stats[threadIdx.x] = r < s.rows ? a.rows[(int64_t)head * a.Tq + s.q0 + r] : make_float2(kInf, 0.f);
            }
            meet<DIRECT>();
            if (t0 + BQ > s.rows || (a.causal && last_key > t0 + s.shift) || (a.window && key0 <= t0 + BQ - 1 + s.shift - a.window)) {
                const bool bad_q = tile_not_finite<BF16, D, BQ, kPartsThreads>(qt), bad_g = tile_not_finite<BF16, D, BQ, kPartsThreads>(gt);
                if (bad_q || bad_g) odd_tile = at;
                __syncthreads();
            }
            const int r0 = t0 + 32 * part;  // this wave's 32 rows
            if (r0 >= s.rows || wave_key >= s.keys || (a.causal && wave_key > r0 + 31 + s.shift) || (a.window && wave_last_key <= r0 + s.shift - a.window)) continue;
            const bool masked = r0 + 32 > s.rows || (a.causal && wave_last_key > r0 + s.shift) || (a.window && wave_key <= r0 + 31 + s.shift - a.window);
            const bool odd = masked && odd_tile == at;
            const Span span = rows_seeing(a, s, key, r0, h);
            f32x16 st, dp;
#pragma unroll
            for (int i = 0; i < 16; i++) st[i] = dp[i] = 0;
            if constexpr (kDk)
                in_turn<2 * KK, BF16>([&](int i, Fragment<BF16>& f) { T::along(i & 1 ? ga : qa, 0, i / 2, f); },
                                      [&](int i, const Fragment<BF16>& f) { mma(i & 1 ? dp : st, f, i & 1 ? v[i / 2] : k[i / 2]); });
            else
                in_turn<KK, BF16>([&](int i, Fragment<BF16>& f) { T::along(qa, 0, i, f); }, [&](int i, const Fragment<BF16>& f) { mma(st, f, k[i]); });
            float p[16];
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int i = 4 * j + e;
                    const float2 of_row = stats[32 * part + 8 * j + 4 * h + e];
                    const bool off = masked && !span.has(0, i);
                    p[i] = __builtin_amdgcn_exp2f(fmaf(st[i], a.scale_log2, -of_row.x));
                    const float ds = p[i] * (dp[i] - of_row.y);
                    p[i] = off ? 0.f : p[i];
                    st[i] = off ? 0.f : ds;
                }
            Fragment<BF16> pf[2], df[2];
#pragma unroll
            for (int n = 0; n < 2; n++) {
                float x[8];
                if constexpr (kDv) {
#pragma unroll
                    for (int e = 0; e < 8; e++) x[e] = p[8 * n + e];
                    operand_of(x, pf[n]);
                }
                if constexpr (kDk) {
#pragma unroll
                    for (int e = 0; e < 8; e++) x[e] = st[8 * n + e];
                    operand_of(x, df[n]);
                }
            }
            // products i: of dV and dK in turn, or of the one of them
            constexpr int kBoth = kDv && kDk ? 2 : 1;
            auto is_dv = [](int i) { return kBoth == 2 ? i % 2 == 0 : kDv; };
            auto read = [&](int i, Fragment<BF16>& f) { T::across(is_dv(i) ? gx : qx, 16 * (i / kBoth / DB), 32 * (i / kBoth % DB), f); };
            if (!odd) {
                in_turn<2 * DB * kBoth, BF16>(read, [&](int i, const Fragment<BF16>& f) {
                    const int n = i / kBoth / DB, d = i / kBoth % DB;
                    if (is_dv(i)) mma(dv[kDv ? d : 0], f, pf[n]);
                    else mma(dk[kDk ? d : 0], f, df[n]);
                });
                continue;
            }
#pragma unroll
            for (int i = 0; i < 2 * DB * kBoth; i++) {
                const int n = i / kBoth / DB, d = i / kBoth % DB;
                bf16x8 seen;
#pragma unroll
                for (int e = 0; e < 8; e++) seen[e] = (__bf16)(span.has(0, 8 * n + e) ? 1.f : 0.f);
                Fragment<BF16> f;
                read(i, f);
                if (is_dv(i)) mma_seen(dv[kDv ? d : 0], f, pf[n], seen);
                else mma_seen(dk[kDk ? d : 0], f, df[n], seen);
                if (!BF16) __builtin_amdgcn_sched_barrier(0);
            }
        }
    if constexpr (kDk) add_parts<DB, B::kParts, B::kBlocks>(dk, lds, part, block, lane);
    if constexpr (kDv) add_parts<DB, B::kParts, B::kBlocks>(dv, lds, part, block, lane);
    if (part != 0 || !live) return;
    const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int c = 32 * d + 8 * j + 4 * h + e;
                if constexpr (kDk) store1<BF16>(a.dk, token * a.lddk + (int64_t)kv_head * D + c, s.bad ? nan : dk[d][4 * j + e] * a.scale);
                if constexpr (kDv) store1<BF16>(a.dv, token * a.lddv + (int64_t)kv_head * D + c, s.bad ? nan : dv[d][4 * j + e]);
            }
}

// All in one launch, those that take longest first, so that the card is full.  ROLES: 1,
// dK and dV by one workgroup; 2, by one each, five products in place of four: past 96
// channels, where a wave's registers do not hold both sums, the operands and what is on its
// way (with launches of their own, 3548 tokens of 16 and 4 heads of 128 in fp32 1.4 ms with 1,
// 1.1 ms with 2; of 256 in bf16 1.8 and 0.8 ms), and where there are few workgroups (of 96 channels, 1 and 2: 665
// tokens of 6 and 3 heads, 198 of them, 103 and 79 us; 1000 of 16 and 4, 640, 255 and 193;
// four times 700 of 6 and 3, 819, 169 and 182; 2000 of 16 and 4, 1260, 498 and 559).
template <bool BF16, int D, int ROLES, bool DIRECT>
__global__ __launch_bounds__(kPartsThreads) void attention_parts_kernel(PackedArgs a, int dkv_groups) {
    typedef PartsShape<BF16, D> B;
    __shared__ __attribute__((aligned(1024))) char lds[2 * B::kTileBytes];
    __shared__ __attribute__((aligned(16))) float2 stats[B::kOther];
    __shared__ int odd_tile;
    int group = blockIdx.y * gridDim.x + blockIdx.x;
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) {
        check_offsets(a.offsets_q, a.n, a.Tq, a.err);
        check_offsets(a.offsets_k, a.n, a.Tk, a.err);
    }
    if (group >= ROLES * dkv_groups) {
        attention_dq_parts<BF16, D, DIRECT>(a, group - ROLES * dkv_groups, lds, odd_tile);
    } else if constexpr (ROLES == 1) {
        attention_dkv_parts<BF16, D, 3, DIRECT>(a, group, lds, stats, odd_tile);
    } else {
        if (group < dkv_groups) attention_dkv_parts<BF16, D, 2, DIRECT>(a, group, lds, stats, odd_tile);
        else attention_dkv_parts<BF16, D, 1, DIRECT>(a, group - dkv_groups, lds, stats, odd_tile);
    }
}

// The same for bf16 heads of up to 128 channels, where registers hold two
// blocks' scores: the products of the next block's S and dP run beside this block's
// exponentials, and the products with them follow, so that the matrix cores wait
// neither for the vector unit nor for LDS.  A block is 32 keys (dQ) or 32 rows a wave
// (dK, dV).
// DIRECT: tiles go straight from memory into LDS; 18 registers are spilled there at 128
// channels, none in the steady loops (149 where lines go through registers).
// Four sequences of up to 4096 tokens, 16 query and 4 key heads of 128, causal: 511 us (dQ
// and dK, dV in launches of their own 193 and 360; 3548 tokens 230 for 190, 665 tokens 72
// for 50), the matrix cores busy for 0.45 of it; what is left is the vector unit's work,
// reads of LDS behind a step's barrier, and the eight products in place of five.
constexpr int kAhead = 2;  // products between an operand's read and its use

constexpr int kBesideThreads = 512;
// dQ: a workgroup has 256 rows, a wave 32 of them.
template <int D> struct DqShape {
    static constexpr int kBytes = 32 * Tile<true, D>::kLineBytes, kLds = 8 * kBytes;  // keys and values, four blocks (three would do: their number's low bits say where)
};
template <int D, bool DIRECT>
__device__ inline void attention_dq_beside(const PackedArgs& a, int group, char* lds, int* odd_block) {
    typedef Tile<true, D> T;
    constexpr int kThreads = kBesideThreads, kRows = kThreads / 2, KK = D / 16, DB = D / 32, kBytes = DqShape<D>::kBytes;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    const int kv_head = group % a.kv_heads, rest = group / a.kv_heads;
    const int head = kv_head * a.per_head + rest % a.per_head;
    int seq, local;
    if (!find_tile<kRows>(a.offsets_q, a.n, a.Tq, rest / a.per_head, &seq, &local)) return;
    const Sequence s = sequence_of(a, seq);
    const int tiles = (s.rows + kRows - 1) / kRows;
    if (local >= tiles) return;
    const int row0 = (tiles - 1 - local) * kRows, wave_first = row0 + wave * 32, row = wave_first + (lane & 31);
    const bool live = row < s.rows;
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

    Fragment<true> q[KK], g[KK];
    const int64_t token = s.q0 + row;
    float2 of_row = make_float2(kInf, 0.f);  // (a row past the last: P = 0)
    if (live) of_row = a.rows[(int64_t)head * a.Tq + token];
    const float lse = of_row.x, delta = of_row.y;
#pragma unroll
    for (int kk = 0; kk < KK; kk++) {
        along_memory<true>(a.q, token * a.ldq + (int64_t)head * D, live, kk, lane, q[kk]);
        along_memory<true>(a.dout, token * a.lddo + (int64_t)head * D, live, kk, lane, g[kk]);
    }
    f32x16 out[DB], st, dp, st_next, dp_next;
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) out[d][i] = 0;

    const int last_row = min(row0 + kRows, s.rows) - 1, wave_last = min(wave_first + 31, s.rows - 1);
    const int end = a.causal ? min(s.keys, last_row + s.shift + 1) : s.keys;
    const int begin = a.window ? max(0, row0 + s.shift - a.window + 1) / 32 * 32 : 0;
    const int total = end > begin ? (end - begin + 31) / 32 : 0;
    // a block whose keys all the workgroup's rows see begins with one of these keys
    const int clear_from = a.window ? last_row + s.shift - a.window + 1 : INT32_MIN;
    const int clear_to = min(s.keys - 32, a.causal ? row0 + s.shift - 31 : INT32_MAX);
    auto masked_block = [&](int t) {
        const int k0 = begin + 32 * t;
        return k0 < clear_from || k0 > clear_to;
    };
    auto in_range = [&](int t) {  // for some row of the wave
        const int k0 = begin + 32 * t;
        return t >= 0 && t < total && wave_first < s.rows && !(a.causal && k0 > wave_last + s.shift) && !(a.window && k0 + 31 <= wave_first + s.shift - a.window);
    };
    Pipe<true, D, 32, kThreads, false> pk, pv;
    LinesToLds<D, 32, kThreads> to_k, to_v;
    auto keys_at = [&](int t) { return lds + (t & 3) * 2 * kBytes; };
    auto values_at = [&](int t) { return lds + (t & 3) * 2 * kBytes + kBytes; };
    // what is fetched next
    int fetch_key = begin;
    const char* k_at = (const char*)a.k + (((int64_t)s.k0 + begin) * a.ldk + (int64_t)kv_head * D) * 2;
    const char* v_at = (const char*)a.v + (((int64_t)s.k0 + begin) * a.ldv + (int64_t)kv_head * D) * 2;
    auto places = [&](int keys) __attribute__((always_inline)) {
        to_k.places(a.ldk, keys);
        to_v.places(a.ldv, keys);
    };
    if (DIRECT && total) places(s.keys - begin);
    auto fetch = [&](int t) __attribute__((always_inline)) {
        if constexpr (DIRECT) {
            if (t > 0 && fetch_key + 32 > s.keys) places(s.keys - fetch_key);
            to_k.fetch(k_at, tile::lds_address(keys_at(t)), wave);
            to_v.fetch(v_at, tile::lds_address(values_at(t)), wave);
        } else {
            pk.fetch(k_at, a.ldk, 0, s.keys - fetch_key, nullptr);
            pv.fetch(v_at, a.ldv, 0, s.keys - fetch_key, nullptr);
        }
        fetch_key += 32;
        k_at += 64 * a.ldk;
        v_at += 64 * a.ldv;
    };
    // Block t + 1 has arrived and t + 2 is fetched.
    auto advance = [&](int t, bool check) __attribute__((always_inline)) {
        if (!DIRECT && t + 1 < total) {
            pk.arrive(keys_at(t + 1));
            pv.arrive(values_at(t + 1));
        }
        meet<DIRECT>();
        if (check && t >= 0 && masked_block(t)) {
            if (tile_not_finite<true, D, 32, kThreads>(keys_at(t))) odd_block[t & 3] = t;
            __syncthreads();
        }
        if (t + 2 < total) fetch(t + 2);
    };
    if (threadIdx.x < 4) odd_block[threadIdx.x] = -1;
    const uint32_t along_lane = T::along_lane(lane), across_lane = T::across_lane(lane);
    if (total) fetch(0);
    int t = -1;
    while (t < total) {
#pragma unroll 1
        while (t >= 0 && t + 1 < total && !masked_block(t)) {
            advance(t, false);
            const uint32_t ka = tile::lds_address(keys_at(t + 1)) + along_lane, va = tile::lds_address(values_at(t + 1)) + along_lane;
            const uint32_t kx = tile::lds_address(keys_at(t)) + across_lane;
            constexpr int kScores = 2 * KK, kSums = 2 * DB, kPairs = 8;
            Fragment<true> f[kAhead + 1], df[2];
            auto read = [&](int i) __attribute__((always_inline)) {
                if (i < kScores) T::along(i & 1 ? va : ka, 0, i / 2, f[i % (kAhead + 1)]);
                else if (i < kScores + kSums) T::across(kx, 16 * ((i - kScores) / DB), 32 * ((i - kScores) % DB), f[i % (kAhead + 1)]);
            };
#pragma unroll
            for (int i = 0; i < kAhead; i++) read(i);
#pragma unroll
            for (int i = 0; i < 16; i++) st_next[i] = dp_next[i] = 0;
#pragma unroll
            for (int i = 0; i < kScores; i++) {
                read(i + kAhead);
                if (i & 1) mma(dp_next, f[i % (kAhead + 1)], g[i / 2]);
                else mma(st_next, f[i % (kAhead + 1)], q[i / 2]);
#pragma unroll
                for (int p = (i * kPairs + kScores - 1) / kScores; p < ((i + 1) * kPairs + kScores - 1) / kScores; p++)
#pragma unroll
                    for (int e = 2 * p; e < 2 * p + 2; e++)
                        df[e / 8].raw[e % 8] = (__bf16)(__builtin_amdgcn_exp2f(fmaf(st[e], a.scale_log2, -lse)) * (dp[e] - delta));
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < kSums; i++) {
                read(kScores + i + kAhead);
                mma(out[i % DB], f[(kScores + i) % (kAhead + 1)], df[i / DB]);
                __builtin_amdgcn_sched_barrier(0);
            }
            st = st_next;
            dp = dp_next;
            t++;
        }
        advance(t, true);
        if (in_range(t)) {
            const uint32_t kx = tile::lds_address(keys_at(t)) + across_lane;
            const bool odd = odd_block[t & 3] == t;
            const Span span = keys_seen(a, s, row, begin + 32 * t, h);
#pragma unroll
            for (int n = 0; n < 2; n++) {
                Fragment<true> df;
                bf16x8 seen;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const bool on = span.has(0, 8 * n + e);
                    const float ds = __builtin_amdgcn_exp2f(fmaf(st[8 * n + e], a.scale_log2, -lse)) * (dp[8 * n + e] - delta);
                    df.raw[e] = (__bf16)(on ? ds : 0.f);
                    seen[e] = (__bf16)(on ? 1.f : 0.f);
                }
#pragma unroll
                for (int d = 0; d < DB; d++) {
                    Fragment<true> f;
                    T::across(kx, 16 * n, 32 * d, f);
                    if (odd) mma_seen(out[d], f, df, seen);
                    else mma(out[d], f, df);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        if (in_range(t + 1)) {
            const uint32_t ka = tile::lds_address(keys_at(t + 1)) + along_lane, va = tile::lds_address(values_at(t + 1)) + along_lane;
#pragma unroll
            for (int i = 0; i < 16; i++) st[i] = dp[i] = 0;
#pragma unroll
            for (int kk = 0; kk < KK; kk++) {
                Fragment<true> f;
                T::along(ka, 0, kk, f);
                mma(st, f, q[kk]);
                T::along(va, 0, kk, f);
                mma(dp, f, g[kk]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        t++;
    }
    if (!live) return;
    const float by = s.bad ? __uint_as_float(0x7FC00000u) : a.scale;
    const int64_t o = token * a.lddq + (int64_t)head * D;
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) store1<true>(a.dq, o + 32 * d + 8 * j + 4 * h + e, out[d][4 * j + e] * by);
}

// dK and dV: a workgroup has 64 keys and passes over the rows 64 at a time; of the four
// 32 x 32 blocks of these one wave adds to dK, another to dV, and the two over the same
// keys are added at the end.  S is computed by both, five products in place of four, but
// a wave's registers then leave room for a second one to each unit.  (With both sums in a
// wave, and one wave to a unit, the unit stood still for most of the time: 432 us for 360.)
template <int D> struct DkvShape {
    static constexpr int kBytes = 64 * Tile<true, D>::kLineBytes, kLds = 8 * kBytes;  // queries and their gradients, four steps
};
template <int D, bool DIRECT>
__device__ inline void attention_dkv_beside(const PackedArgs& a, int group, char* lds, float2 (*stats)[64], int* odd_step) {
    typedef Tile<true, D> T;
    constexpr int kThreads = kBesideThreads, kKeys = 64, KK = D / 16, DB = D / 32, kBytes = DkvShape<D>::kBytes;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5, part = wave >> 1 & 1;
    const int kv_head = group % a.kv_heads;
    int seq, local;
    if (!find_tile<kKeys>(a.offsets_k, a.n, a.Tk, group / a.kv_heads, &seq, &local)) return;
    const Sequence s = sequence_of(a, seq);
    const int key0 = local * kKeys, wave_key = key0 + (wave & 1) * 32, key = wave_key + (lane & 31);
    if (key0 >= s.keys) return;
    const bool live = key < s.keys;
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);
    const int64_t token = s.k0 + key;

    // rows that see any of the workgroup's keys, 64 a step, the last ones first and the query
    // heads in turn: workgroups that run at the same time read the same rows
    const int last_key = min(key0 + kKeys, s.keys) - 1, wave_last_key = min(wave_key + 31, s.keys - 1);
    const int begin = a.causal ? max(0, key0 - s.shift) / 64 * 64 : 0;
    const int end = (int)min((int64_t)s.rows, a.window ? (int64_t)last_key - s.shift + a.window : s.rows);
    const int per = end > begin ? (end - begin + 63) / 64 : 0, total = per * a.per_head;
    const int first_head = kv_head * a.per_head, first_row = begin + (per - 1) * 64;
    int fetch_head = first_head, fetch_row = first_row;  // of the next step to be fetched
    // a step whose rows all see all of the workgroup's keys begins with one of these rows
    const int clear_from = a.causal ? last_key - s.shift : INT32_MIN;
    const int clear_to = min(s.rows - 64, a.window ? key0 - 64 - s.shift + a.window : INT32_MAX);
    auto masked_rows = [&](int r0) { return r0 < clear_from || r0 > clear_to; };
    Pipe<true, D, 64, kThreads, false> pq, pg;
    float2 of_row;
    auto queries_at = [&](int t) { return lds + (t & 3) * 2 * kBytes; };
    // what is fetched next: the first of 64 rows of queries, of their gradients and of
    // their L and delta, and this lane's places from there (rows past the last repeat it)
    const char* q_at = (const char*)a.q + (((int64_t)s.q0 + first_row) * a.ldq + (int64_t)first_head * D) * 2;
    const char* g_at = (const char*)a.dout + (((int64_t)s.q0 + first_row) * a.lddo + (int64_t)first_head * D) * 2;
    const float2* stats_at = a.rows + (int64_t)first_head * a.Tq + s.q0 + first_row;
    LinesToLds<D, 64, kThreads> to_q, to_g;
    uint32_t stats_place;
    auto places = [&](int rows) __attribute__((always_inline)) {
        to_q.places(a.ldq, rows);
        to_g.places(a.lddo, rows);
        stats_place = min(32 * wave + lane / 2, rows - 1) * 8 + (lane & 1) * 4;
    };
    if (DIRECT) places(s.rows - first_row);
    auto fetch = [&](int t) __attribute__((always_inline)) {
        if constexpr (DIRECT) {
            to_q.fetch(q_at, tile::lds_address(queries_at(t)), wave);
            to_g.fetch(g_at, tile::lds_address(queries_at(t)) + kBytes, wave);
            if (wave < 2) load_lds4(tile::lds_address(&stats[t & 3][32 * wave]), stats_place, stats_at);
        } else {
            pq.fetch(q_at, a.ldq, 0, s.rows - fetch_row, nullptr);
            pg.fetch(g_at, a.lddo, 0, s.rows - fetch_row, nullptr);
            if (threadIdx.x < 64) of_row = stats_at[min((int)threadIdx.x, s.rows - fetch_row - 1)];
        }
        q_at += D * 2;
        g_at += D * 2;
        stats_at += a.Tq;
        if (++fetch_head == first_head + a.per_head) {
            q_at -= (64 * a.ldq + a.per_head * D) * 2;
            g_at -= (64 * a.lddo + a.per_head * D) * 2;
            stats_at -= 64 + (int64_t)a.per_head * a.Tq;
            fetch_head = first_head;
            fetch_row -= 64;
            if (DIRECT) places(64);
        }
    };
    // Step t + 1 has arrived and t + 2 is fetched.
    auto advance = [&](int t, int r0, bool check) __attribute__((always_inline)) {
        if (t + 1 < total) {
            if (!DIRECT) {
                pq.arrive(queries_at(t + 1));
                pg.arrive(queries_at(t + 1) + kBytes);
            }
            if (!DIRECT && threadIdx.x < 64) stats[(t + 1) & 3][threadIdx.x] = of_row;
        }
        meet<DIRECT>();
        if (check && t >= 0 && masked_rows(r0)) {
            const bool bad_q = tile_not_finite<true, D, 64, kThreads>(queries_at(t)), bad_g = tile_not_finite<true, D, 64, kThreads>(queries_at(t) + kBytes);
            if (bad_q || bad_g) odd_step[t & 3] = t;
            __syncthreads();
        }
        if (t + 2 < total) fetch(t + 2);
    };
    if (threadIdx.x < 4) odd_step[threadIdx.x] = -1;
    const uint32_t along_lane = T::along_lane(lane) + part * 32 * T::kLineBytes, across_lane = T::across_lane(lane) + part * 32 * T::kLineBytes;
    if (total) fetch(0);

    auto pass = [&](auto which) __attribute__((always_inline)) {
        constexpr bool kDK = which.value;  // dK, or dV
        Fragment<true> k[KK], v[kDK ? KK : 1];
#pragma unroll
        for (int kk = 0; kk < KK; kk++) {
            along_memory<true>(a.k, token * a.ldk + (int64_t)kv_head * D, live, kk, lane, k[kk]);
            if constexpr (kDK) along_memory<true>(a.v, token * a.ldv + (int64_t)kv_head * D, live, kk, lane, v[kk]);
        }
        f32x16 sum[DB], st, dp, st_next, dp_next;
#pragma unroll
        for (int i = 0; i < 16; i++)
#pragma unroll
            for (int d = 0; d < DB; d++) sum[d][i] = 0;
        int t = -1, r0 = first_row, left = a.per_head + 1;  // step t's rows begin at r0, `left` steps of them are left
        auto step_on = [&]() __attribute__((always_inline)) {
            t++;
            if (--left == 0) {
                left = a.per_head;
                r0 -= 64;
            }
        };
        while (t < total) {
            constexpr int kScores = (kDK ? 2 : 1) * KK, kSums = 2 * DB, kPairs = 8;
            Fragment<true> f[kAhead + 1], pf[2];
            uint32_t qa, qx;
            auto read = [&](int i) __attribute__((always_inline)) {
                if (kDK) T::along(i & 1 ? qa + kBytes : qa, 0, i / 2, f[i % (kAhead + 1)]);
                else T::along(qa, 0, i, f[i % (kAhead + 1)]);
            };
            auto read_across = [&](int i, int at) __attribute__((always_inline)) { T::across(qx, 16 * (i / DB), 32 * (i % DB), f[(at + i) % (kAhead + 1)]); };
            auto scores = [&](int t) __attribute__((always_inline)) {  // of step t + 1, beside step t's exponentials
                const float2* rows = &stats[t & 3][32 * part + 4 * h];
                f32x4 two[3];  // L and delta of two rows
                auto read_stats = [&](int p) __attribute__((always_inline)) {
                    if (p < kPairs) two[p % 3] = *(const f32x4*)(rows + 8 * (p / 2) + 2 * (p & 1));
                };
                read_stats(0);
                read_stats(1);
#pragma unroll
                for (int i = 0; i < kAhead; i++) read(i);
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    st_next[i] = 0;
                    if (kDK) dp_next[i] = 0;
                }
#pragma unroll
                for (int i = 0; i < kScores; i++) {
                    if (i + kAhead < kScores) read(i + kAhead);
                    else if (kDK) read_across(i + kAhead - kScores, kScores);
                    if constexpr (kDK) {
                        if (i & 1) mma(dp_next, f[i % (kAhead + 1)], v[i / 2]);
                        else mma(st_next, f[i % (kAhead + 1)], k[i / 2]);
                    } else {
                        mma(st_next, f[i % (kAhead + 1)], k[i]);
                    }
#pragma unroll
                    for (int p = (i * kPairs + kScores - 1) / kScores; p < ((i + 1) * kPairs + kScores - 1) / kScores; p++) {
                        read_stats(p + 2);
                        const f32x4 of = two[p % 3];
#pragma unroll
                        for (int e = 2 * p; e < 2 * p + 2; e++) {
                            float x = __builtin_amdgcn_exp2f(fmaf(st[e], a.scale_log2, -of[2 * (e & 1)]));
                            if (kDK) x *= dp[e] - of[2 * (e & 1) + 1];
                            pf[e / 8].raw[e % 8] = (__bf16)x;
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                st = st_next;
                if (kDK) dp = dp_next;
            };
            auto sums = [&](int at) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < kSums; i++) {
                    if (i + kAhead < kSums) read_across(i + kAhead, at);
                    mma(sum[i % DB], f[(at + i) % (kAhead + 1)], pf[i / DB]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            // dK's waves sum at the end of a step; dV's at the beginning of the next one, so
            // that of a unit's two waves one sums while the other's vector work is done
            bool held = false;
            auto held_sums = [&](int t) __attribute__((always_inline)) {
                if (kDK || !held) return;
                qx = tile::lds_address(queries_at(t)) + kBytes + across_lane;
#pragma unroll
                for (int i = 0; i < kAhead; i++) read_across(i, 0);
                sums(0);
                held = false;
            };
#pragma unroll 1
            while (t >= 0 && t + 1 < total && !masked_rows(r0)) {
                advance(t, r0, false);
                held_sums(t - 1);
                qa = tile::lds_address(queries_at(t + 1)) + along_lane;
                if (kDK) qx = tile::lds_address(queries_at(t)) + across_lane;
                scores(t);
                if (kDK) sums(kScores);
                else held = true;
                step_on();
            }
            held_sums(t - 1);
            advance(t, r0, true);
            const int first = r0 + 32 * part;
            auto in_range = [&](int t, int first) {  // some row of the wave sees some key of it
                return t >= 0 && t < total && wave_key < s.keys && first < s.rows && !(a.causal && wave_key > first + 31 + s.shift) &&
                       !(a.window && wave_last_key <= first + s.shift - a.window);
            };
            if (in_range(t, first)) {
                const uint32_t qx = tile::lds_address(queries_at(t)) + (kDK ? 0 : kBytes) + across_lane;
                const float2* rows = &stats[t & 3][32 * part + 4 * h];
                const bool odd = odd_step[t & 3] == t;
                const Span span = rows_seeing(a, s, key, first, h);
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    Fragment<true> pf;
                    bf16x8 seen;
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int i = 8 * n + e;
                        const float2 r = rows[8 * (i >> 2) + (i & 3)];
                        const bool on = span.has(0, i);
                        float x = __builtin_amdgcn_exp2f(fmaf(st[i], a.scale_log2, -r.x));
                        if (kDK) x *= dp[i] - r.y;
                        pf.raw[e] = (__bf16)(on ? x : 0.f);
                        seen[e] = (__bf16)(on ? 1.f : 0.f);
                    }
#pragma unroll
                    for (int d = 0; d < DB; d++) {
                        Fragment<true> f;
                        T::across(qx, 16 * n, 32 * d, f);
                        if (odd) mma_seen(sum[d], f, pf, seen);
                        else mma(sum[d], f, pf);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            step_on();
            if (in_range(t, r0 + 32 * part)) {
                const uint32_t qa = tile::lds_address(queries_at(t)) + along_lane;
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    st[i] = 0;
                    if (kDK) dp[i] = 0;
                }
#pragma unroll
                for (int kk = 0; kk < KK; kk++) {
                    Fragment<true> f;
                    T::along(qa, 0, kk, f);
                    mma(st, f, k[kk]);
                    if constexpr (kDK) {
                        T::along(qa + kBytes, 0, kk, f);
                        mma(dp, f, v[kk]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        // the second rows' sums to the first rows' waves
        __syncthreads();
        f32x4* sums = (f32x4*)lds + ((wave & 1) * 2 + kDK) * DB * 4 * 64;
        if (part == 1) {
#pragma unroll
            for (int d = 0; d < DB; d++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    f32x4 x;
#pragma unroll
                    for (int e = 0; e < 4; e++) x[e] = sum[d][4 * j + e];
                    sums[(d * 4 + j) * 64 + lane] = x;
                }
        }
        __syncthreads();
        if (part == 1 || !live) return;
        const float by = s.bad ? __uint_as_float(0x7FC00000u) : kDK ? a.scale : 1.f;
        void* out = kDK ? a.dk : a.dv;
        const int64_t o = token * (kDK ? a.lddk : a.lddv) + (int64_t)kv_head * D;
#pragma unroll
        for (int d = 0; d < DB; d++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const f32x4 x = sums[(d * 4 + j) * 64 + lane];
#pragma unroll
                for (int e = 0; e < 4; e++) store1<true>(out, o + 32 * d + 8 * j + 4 * h + e, (sum[d][4 * j + e] + x[e]) * by);
            }
    };
    if (wave < 4) pass(std::true_type{});
    else pass(std::false_type{});
}

// In one launch, as above.
template <int D, bool DIRECT>
__global__ __launch_bounds__(kBesideThreads, 2) void attention_backward_kernel(PackedArgs a, int dkv_groups) {
    static_assert(DqShape<D>::kLds <= DkvShape<D>::kLds, "shared");
    __shared__ __attribute__((aligned(1024))) char lds[DkvShape<D>::kLds];
    __shared__ __attribute__((aligned(1024))) float2 stats[4][64];
    __shared__ int odd[4];
    const int group = blockIdx.y * gridDim.x + blockIdx.x;
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) {
        check_offsets(a.offsets_q, a.n, a.Tq, a.err);
        check_offsets(a.offsets_k, a.n, a.Tk, a.err);
    }
    if (group < dkv_groups) attention_dkv_beside<D, DIRECT>(a, group, lds, stats, odd);
    else attention_dq_beside<D, DIRECT>(a, group - dkv_groups, lds, odd);
}

inline dim3 grid_of(int64_t groups) {  // (threads of a grid's row: 32 bits)
    const int64_t across = 1 << 20;
    return dim3((unsigned)std::min(groups, across), (unsigned)((groups + across - 1) / across));
}
template <bool BF16, int D>
void launch_rows(const PackedArgs& a, hipStream_t s) {
    const int64_t groups = ((int64_t)a.Tq * a.q_heads + 7) / 8;
    hipLaunchKernelGGL((attention_rows_kernel<BF16, D>), dim3((unsigned)std::min<int64_t>(std::max<int64_t>(groups, 1), 8192)), dim3(kRowsThreads), 0, s, a);
}
template <int D, bool DIRECT>
void launch_beside(const PackedArgs& a, hipStream_t s) {
    const int64_t dkv = tile_slots(a.Tk, 64, a.n) * a.kv_heads, dq = tile_slots(a.Tq, kBesideThreads / 2, a.n) * a.q_heads;
    hipLaunchKernelGGL((attention_backward_kernel<D, DIRECT>), grid_of(dkv + dq), dim3(kBesideThreads), 0, s, a, (int)dkv);
}
template <bool BF16, int D, bool DIRECT>
void launch_parts(const PackedArgs& a, hipStream_t s) {
    typedef PartsShape<BF16, D> B;
    const int64_t dkv = tile_slots(a.Tk, B::kOwn, a.n) * a.kv_heads, dq = tile_slots(a.Tq, B::kOwn, a.n) * a.q_heads;
    if constexpr (D <= 96)
        if (dkv + dq >= 700) {
            hipLaunchKernelGGL((attention_parts_kernel<BF16, D, 1, DIRECT>), grid_of(dkv + dq), dim3(kPartsThreads), 0, s, a, (int)dkv);
            return;
        }
    hipLaunchKernelGGL((attention_parts_kernel<BF16, D, 2, DIRECT>), grid_of(2 * dkv + dq), dim3(kPartsThreads), 0, s, a, (int)dkv);
}
template <bool BF16, int D>
hipError_t launch_backward(const PackedArgs& a, hipStream_t s) {
    const bool direct = direct_lines(a.q, a.ldq, BF16) && direct_lines(a.k, a.ldk, BF16) && direct_lines(a.v, a.ldv, BF16) && direct_lines(a.dout, a.lddo, BF16);
    launch_rows<BF16, D>(a, s);
    if constexpr (BF16 && D <= 128) {
        if (direct) launch_beside<D, true>(a, s);
        else launch_beside<D, false>(a, s);
    } else {
        if (direct) launch_parts<BF16, D, true>(a, s);
        else launch_parts<BF16, D, false>(a, s);
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
