// Attention over packed sequences, forward:
//   S = scale Q K^T,  P = softmax of each row over the keys that it sees,  O = P V.
// One pass over the keys with a running maximum and sum.  In bf16 P is rounded to bf16 for
// the second product (S, the maximum, the sum and O are not): the result is 0.0021 off, its
// own rounding being 0.0016.  Two bf16 terms of P in the steady loop take 752 us for 564
// (8192 tokens of 32 and 8 heads of 128); who needs P whole calls in fp32.
#pragma once

#include <algorithm>

#include "attention_parts.h"

namespace moe {
namespace packed {

constexpr int kForwardWaves = 4;
template <bool BF16, int D> struct ForwardShape {
    static constexpr int kThreads = 64 * kForwardWaves;
    static constexpr int kRows = 32 * kForwardWaves;          // a wave has 32 rows
    static constexpr int kKeys = BF16 && D <= 128 ? 64 : 32;  // of a tile
    static constexpr int kTileBytes = kKeys * Tile<BF16, D>::kLineBytes;
};

// DIRECT: tiles go straight from memory into LDS (lines whole 16-byte chunks in memory);
// else through registers.  Two waves a SIMD, bf16 heads of up to 128 channels, spill 22
// registers at 128 (41 through registers), none of them in the steady loop; fp32 heads of
// 256 channels 114, inside it.
template <bool BF16, int D, bool DIRECT>
__global__ __launch_bounds__(kForwardWaves * 64, BF16 && D <= 128 ? 2 : 1) void attention_kernel(PackedArgs a) {
    typedef ForwardShape<BF16, D> F;
    typedef Tile<BF16, D> T;
    constexpr int BK = F::kKeys, KK = D / 16, DB = D / 32, KB = BK / 32;
    __shared__ __attribute__((aligned(1024))) char lds[4 * F::kTileBytes];
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
    const int row0 = (tiles - 1 - local) * F::kRows, wave_first = row0 + wave * 32, row = wave_first + (lane & 31);
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

    const bool live = row < s.rows;
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
    float m = -kInf, l = 0;  // of the row: m the largest q.k, about; l this lane's part of the sum

    // keys that any of the workgroup's rows, and of the wave's, sees
    const int last_row = min(row0 + F::kRows, s.rows) - 1;
    const int end = a.causal ? min(s.keys, last_row + s.shift + 1) : s.keys;
    const int begin = a.window ? max(0, row0 + s.shift - a.window + 1) / BK * BK : 0;
    const int wave_last = min(wave_first + 31, s.rows - 1);

    const char* kbase = (const char*)a.k + ((int64_t)s.k0 * a.ldk + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    const char* vbase = (const char*)a.v + ((int64_t)s.k0 * a.ldv + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    // a tile whose keys all the workgroup's rows see begins with one of these keys
    const int clear_from = a.window ? last_row + s.shift - a.window + 1 : INT32_MIN;
    const int clear_to = min(s.keys - BK, a.causal ? row0 + s.shift - BK + 1 : INT32_MAX);
    auto masked_tile = [&](int k0) { return k0 < clear_from || k0 > clear_to; };
    // tiles of bf16 heads of up to 128 channels that go straight into LDS are stepped through
    constexpr bool kLines = BF16 && D <= 128 && DIRECT;
    Pipe<BF16, D, BK, F::kThreads, DIRECT> pk, pv;
    LinesToLds<kLines ? D : 64, 64, F::kThreads> to_k, to_v;
    const char *k_at = kbase + (int64_t)begin * a.ldk * 2, *v_at = vbase + (int64_t)begin * a.ldv * 2;
    if (kLines && begin < end) {
        to_k.places(a.ldk, s.keys - begin);
        to_v.places(a.ldv, s.keys - begin);
    }
    auto fetch_keys = [&](int k0, char* to) __attribute__((always_inline)) {
        if constexpr (kLines) {
            if (k0 > begin && k0 + BK > s.keys) to_k.places(a.ldk, s.keys - k0);
            to_k.fetch(k_at, tile::lds_address(to), wave);
            k_at += BK * 2 * a.ldk;
        } else {
            pk.fetch(kbase, a.ldk, k0, s.keys - k0, to);
        }
    };
    auto fetch_values = [&](int k0, char* to) __attribute__((always_inline)) {
        if constexpr (kLines) {
            if (k0 > begin && k0 + BK > s.keys) to_v.places(a.ldv, s.keys - k0);
            to_v.fetch(v_at, tile::lds_address(to), wave);
            v_at += BK * 2 * a.ldv;
        } else {
            pv.fetch(vbase, a.ldv, k0, s.keys - k0, to);
        }
    };
    if (threadIdx.x < 2) odd_tile[threadIdx.x] = -1;
    // The products of a tile's scores run one tile ahead, beside the exponentials of the
    // tile before: keys of tile t + 1 and values of tile t are in LDS at a time.
    f32x16 st[KB], nx[KB];
    auto scores = [&](uint32_t ka, f32x16 (&to)[KB]) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < KB; b++) {
#pragma unroll
            for (int i = 0; i < 16; i++) to[b][i] = 0;
#pragma unroll
            for (int kk = 0; kk < KK; kk++) {
                Fragment<BF16> f;
                T::along(ka, 32 * b, kk, f);
                f.split();
                mma(to[b], f, q[kk]);
                __builtin_amdgcn_sched_barrier(0);  // (operands of one product at a time: registers are short)
            }
        }
    };
    auto exponentials = [&](float base, int b, int g, Fragment<BF16>& pf) __attribute__((always_inline)) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; e++) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(st[b][8 * g + e], a.scale_log2, -base));
            l += p[e];
        }
        operand_of(p, pf);
    };
    auto values = [&](uint32_t va, int b, int g, const Fragment<BF16>& pf) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < DB; d++) {
            Fragment<BF16> f;
            T::across(va, 32 * b + 16 * g, 32 * d, f);
            f.split();
            mma(out[d], f, pf);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto in_range = [&](int k0) {  // some row of the wave sees a key of the tile
        return k0 >= begin && k0 < end && wave_first < s.rows && !(a.causal && k0 > wave_last + s.shift) &&
               !(a.window && k0 + BK - 1 <= wave_first + s.shift - a.window);
    };
    const uint32_t along_lane = T::along_lane(lane), across_lane = T::across_lane(lane);
    int buffer = 0;
    if (begin < end) fetch_keys(begin, lds);
    // Tile k0's values and the next one's keys have arrived, and those after them are fetched.
    auto advance = [&](int k0, bool check) __attribute__((always_inline)) {
        char* kt = lds + 2 * buffer * F::kTileBytes;
        const int next = k0 + BK;
        if (next < end) pk.arrive(kt);
        if (k0 >= begin) pv.arrive(kt + F::kTileBytes);
        meet<DIRECT>();
        if (check && k0 >= begin && masked_tile(k0)) {
            if (tile_not_finite<BF16, D, BK, F::kThreads>(kt + F::kTileBytes)) odd_tile[buffer] = k0;
            __syncthreads();
        }
        if (next + BK < end) fetch_keys(next + BK, lds + 2 * (buffer ^ 1) * F::kTileBytes);
        if (next < end) fetch_values(next, lds + (2 * (buffer ^ 1) + 1) * F::kTileBytes);
    };
    // The next tile's scores, their maximum known, become this tile's.  The maximum that
    // exponentials are taken against follows only where a row's would pass 2^8: sums in
    // fp32 and factors in bf16 are as exact at any common scale.
    auto follow = [&](float top) __attribute__((always_inline)) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
        top = max_of(__uint_as_float(r[0]), __uint_as_float(r[1]));
        const float before = m;
        const bool grown = (top - before) * a.scale_log2 > 8.f;
        if (__any(grown)) {
            m = grown ? top : before;
            const float f = grown ? __builtin_amdgcn_exp2f((before - top) * a.scale_log2) : 1.f;
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; d++) out[d] *= f;
        }
#pragma unroll
        for (int b = 0; b < KB; b++) st[b] = nx[b];
    };
    int k0 = begin - BK;
    while (k0 < end) {
        if constexpr (BF16) {
            // Tiles that every row of the workgroup sees whole, as does the one after each:
            // a product of the next scores, then some exponentials of this tile; a product
            // with this tile's values, then some of the next scores' maximum.  The matrix
            // cores run while the wave goes on; operands are read a product ahead.
#pragma unroll 1
            while (k0 >= begin && k0 + BK < end && k0 >= clear_from && k0 + BK <= clear_to) {
                advance(k0, false);
                const uint32_t ka = tile::lds_address(lds + 2 * buffer * F::kTileBytes) + along_lane;
                const uint32_t va = tile::lds_address(lds + (2 * buffer + 1) * F::kTileBytes) + across_lane;
                const float base = m == -kInf ? 0.f : m * a.scale_log2;
                constexpr int kScores = KB * KK, kValues = 2 * KB * DB, kPairs = 8 * KB;
                constexpr int kAhead = 2;  // products between an operand's read and its use
                Fragment<BF16> pf[2 * KB], f[kAhead + 1];
                float sum = 0, top = -kInf;
                auto read = [&](int i) __attribute__((always_inline)) {
                    if (i < kScores) T::along(ka, 32 * (i / KK), i % KK, f[i % (kAhead + 1)]);
                    else if (i < kScores + kValues) T::across(va, 16 * ((i - kScores) / DB), 32 * ((i - kScores) % DB), f[i % (kAhead + 1)]);
                };
#pragma unroll
                for (int i = 0; i < kAhead; i++) read(i);
#pragma unroll
                for (int b = 0; b < KB; b++)
#pragma unroll
                    for (int i = 0; i < 16; i++) nx[b][i] = 0;
#pragma unroll
                for (int i = 0; i < kScores; i++) {
                    read(i + kAhead);
                    mma(nx[i / KK], f[i % (kAhead + 1)], q[i % KK]);
#pragma unroll
                    for (int p = (i * kPairs + kScores - 1) / kScores; p < ((i + 1) * kPairs + kScores - 1) / kScores; p++) {
                        const int e = 2 * p % 16;
                        const float x = __builtin_amdgcn_exp2f(fmaf(st[p / 8][e], a.scale_log2, -base)), y = __builtin_amdgcn_exp2f(fmaf(st[p / 8][e + 1], a.scale_log2, -base));
                        sum += x + y;
                        pf[p / 4].raw[e % 8] = (__bf16)x;
                        pf[p / 4].raw[e % 8 + 1] = (__bf16)y;
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                l += sum;
#pragma unroll
                for (int i = 0; i < kValues; i++) {
                    read(kScores + i + kAhead);
                    mma(out[i % DB], f[(kScores + i) % (kAhead + 1)], pf[i / DB]);
#pragma unroll
                    for (int p = (i * kPairs + kValues - 1) / kValues; p < ((i + 1) * kPairs + kValues - 1) / kValues; p++) {
                        const int e = 2 * p % 16;
                        top = max_of(top, max_of(nx[p / 8][e], nx[p / 8][e + 1]));
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                follow(top);
                k0 += BK;
                buffer ^= 1;
            }
        }
        advance(k0, true);
        const int next = k0 + BK;
        const uint32_t ka = tile::lds_address(lds + 2 * buffer * F::kTileBytes) + along_lane;
        const uint32_t va = tile::lds_address(lds + (2 * buffer + 1) * F::kTileBytes) + across_lane;
        const bool ahead = in_range(next);
        if (in_range(k0)) {
            const bool odd = odd_tile[buffer] == k0;
            const float base = m == -kInf ? 0.f : m * a.scale_log2;
            const Span span = keys_seen(a, s, row, k0, h);
#pragma unroll
            for (int b = 0; b < KB; b++)
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    Fragment<BF16> pf;
                    exponentials(base, b, g, pf);
                    if (odd) {
                        bf16x8 seen;
#pragma unroll
                        for (int e = 0; e < 8; e++) seen[e] = (__bf16)(span.has(b, 8 * g + e) ? 1.f : 0.f);
#pragma unroll
                        for (int d = 0; d < DB; d++) {
                            Fragment<BF16> f;
                            T::across(va, 32 * b + 16 * g, 32 * d, f);
                            mma_seen(out[d], f, pf, seen);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    } else {
                        values(va, b, g, pf);
                    }
                }
        }
        if (ahead) {
            scores(ka, nx);
            if (next + BK > s.keys || (a.causal && next + BK - 1 > wave_first + s.shift) || (a.window && next <= wave_last + s.shift - a.window)) {
                const Span span = keys_seen(a, s, row, next, h);
#pragma unroll
                for (int b = 0; b < KB; b++)
#pragma unroll
                    for (int i = 0; i < 16; i++) nx[b][i] = span.has(b, i) ? nx[b][i] : -kInf;
            }
            float top = -kInf;
#pragma unroll
            for (int b = 0; b < KB; b++)
#pragma unroll
                for (int i = 0; i < 16; i++) top = max_of(top, nx[b][i]);
            follow(top);
        }
        k0 += BK;
        buffer ^= 1;
    }
    const float nan = __uint_as_float(0x7FC00000u);
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    const float sum = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    if (!live) return;
    // a row that sees nothing: 0, and minus infinity (one whose scores are NaN leaves m so too, but not its sum)
    const bool none = m == -kInf && sum == 0.f;
    const float by = s.bad ? nan : none ? 0.f : 1.0f / sum;
    const int64_t token = s.q0 + row, o = token * a.ldo + (int64_t)head * D;
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) store1<BF16>(a.out, o + 32 * d + 8 * j + 4 * h + e, nan_if_infinite(out[d][4 * j + e] * by));
    if (a.lse && h == 0) a.lse[token * a.q_heads + head] = s.bad ? nan : none ? -kInf : fmaf(m, a.scale, __builtin_amdgcn_logf(sum) * kLn2);
}

// The same for few rows, by PartsShape: 32 (or 64) rows a workgroup, its waves over parts of
// the keys, each with a maximum and sums of its own that are joined at the end.  The next
// tile is on its way where LDS holds two.  Figures at its launch.
template <bool BF16, int D, bool DIRECT>
__global__ __launch_bounds__(kPartsThreads) void attention_few_kernel(PackedArgs a) {
    typedef PartsShape<BF16, D> B;
    typedef Tile<BF16, D> T;
    constexpr int BK = B::kOther, KK = D / 16, DB = D / 32, kBuffers = B::kTileBytes <= 32768 ? 2 : 1;
    __shared__ __attribute__((aligned(1024))) char lds[2 * kBuffers * B::kTileBytes];
    __shared__ float2 stats[kPartsWaves][32];
    __shared__ int odd_tile;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    const int block = wave % B::kBlocks, part = wave / B::kBlocks;
    const int kv_head = blockIdx.x % a.kv_heads, rest = blockIdx.x / a.kv_heads;
    const int head = kv_head * a.per_head + rest % a.per_head;
    if (blockIdx.x == gridDim.x - 1) {
        check_offsets(a.offsets_q, a.n, a.Tq, a.err);
        check_offsets(a.offsets_k, a.n, a.Tk, a.err);
    }
    int seq, local;
    if (!find_tile<B::kOwn>(a.offsets_q, a.n, a.Tq, rest / a.per_head, &seq, &local)) return;
    const Sequence s = sequence_of(a, seq);
    const int tiles = (s.rows + B::kOwn - 1) / B::kOwn;
    if (local >= tiles) return;
    const int row0 = (tiles - 1 - local) * B::kOwn, wave_first = row0 + block * 32, row = wave_first + (lane & 31);
    const bool live = row < s.rows;
    if (s.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

    const int last_row = min(row0 + B::kOwn, s.rows) - 1, wave_last = min(wave_first + 31, s.rows - 1);
    const int end = a.causal ? min(s.keys, last_row + s.shift + 1) : s.keys;
    const int begin = a.window ? max(0, row0 + s.shift - a.window + 1) / 32 * 32 : 0;
    const char* kbase = (const char*)a.k + ((int64_t)s.k0 * a.ldk + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    const char* vbase = (const char*)a.v + ((int64_t)s.k0 * a.ldv + (int64_t)kv_head * D) * (BF16 ? 2 : 4);
    Pipe<BF16, D, BK, kPartsThreads, DIRECT> pk, pv;
    int buffer = 0;
    auto fetch = [&](int t0, int b) __attribute__((always_inline)) {
        pk.fetch(kbase, a.ldk, t0, s.keys - t0, lds + 2 * b * B::kTileBytes);
        pv.fetch(vbase, a.ldv, t0, s.keys - t0, lds + (2 * b + 1) * B::kTileBytes);
    };
    if (kBuffers == 2 && begin < end) fetch(begin, 0);

    Fragment<BF16> q[KK];
    const int64_t token = s.q0 + row;
#pragma unroll
    for (int kk = 0; kk < KK; kk++) {
        along_memory<BF16>(a.q, token * a.ldq + (int64_t)head * D, live, kk, lane, q[kk]);
        q[kk].split();
    }
    f32x16 out[DB];
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int i = 0; i < 16; i++) out[d][i] = 0;
    float m = -kInf, l = 0;  // the largest q.k, about; this lane's part of the sum
    if (threadIdx.x == 0) odd_tile = -1;
    const uint32_t along_lane = T::along_lane(lane) + part * 32 * T::kLineBytes, across_lane = T::across_lane(lane) + part * 32 * T::kLineBytes;
#pragma unroll 1
    for (int t0 = begin; t0 < end; t0 += BK) {
        char *kt = lds + 2 * buffer * B::kTileBytes, *vt = kt + B::kTileBytes;
        if (kBuffers == 1) {
            __syncthreads();
            fetch(t0, 0);
        }
        pk.arrive(kt);
        pv.arrive(vt);
        meet<DIRECT>();
        if (kBuffers == 2 && t0 + BK < end) fetch(t0 + BK, buffer ^ 1);
        if (t0 + BK > s.keys || (a.causal && t0 + BK - 1 > row0 + s.shift) || (a.window && t0 <= last_row + s.shift - a.window)) {
            if (tile_not_finite<BF16, D, BK, kPartsThreads>(vt)) odd_tile = t0;
            __syncthreads();
        }
        const uint32_t ka = tile::lds_address(kt) + along_lane, vx = tile::lds_address(vt) + across_lane;
        buffer ^= kBuffers - 1;
        const int k0 = t0 + 32 * part;  // this wave's 32 keys
        if (k0 >= s.keys || wave_first >= s.rows || (a.causal && k0 > wave_last + s.shift) || (a.window && k0 + 31 <= wave_first + s.shift - a.window)) continue;
        const bool masked = k0 + 32 > s.keys || (a.causal && k0 + 31 > wave_first + s.shift) || (a.window && k0 <= wave_last + s.shift - a.window);
        const bool odd = masked && odd_tile == t0;
        const Span span = keys_seen(a, s, row, k0, h);
        f32x16 st;
#pragma unroll
        for (int i = 0; i < 16; i++) st[i] = 0;
        in_turn<KK, BF16>([&](int i, Fragment<BF16>& f) { T::along(ka, 0, i, f); }, [&](int i, const Fragment<BF16>& f) { mma(st, f, q[i]); });
        float top = -kInf;
#pragma unroll
        for (int i = 0; i < 16; i++) {
            st[i] = masked && !span.has(0, i) ? -kInf : st[i];
            top = max_of(top, st[i]);
        }
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
        top = max_of(__uint_as_float(r[0]), __uint_as_float(r[1]));
        const float before = m;
        const bool grown = (top - before) * a.scale_log2 > 8.f;  // (as above)
        if (__any(grown)) {
            m = grown ? top : before;
            const float f = grown ? __builtin_amdgcn_exp2f((before - top) * a.scale_log2) : 1.f;
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; d++) out[d] *= f;
        }
        const float base = m == -kInf ? 0.f : m * a.scale_log2;
        Fragment<BF16> pf[2];
#pragma unroll
        for (int n = 0; n < 2; n++) {
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                p[e] = __builtin_amdgcn_exp2f(fmaf(st[8 * n + e], a.scale_log2, -base));
                l += p[e];
            }
            operand_of(p, pf[n]);
        }
        auto read = [&](int i, Fragment<BF16>& f) { T::across(vx, 16 * (i / DB), 32 * (i % DB), f); };
        if (!odd) {
            in_turn<2 * DB, BF16>(read, [&](int i, const Fragment<BF16>& f) { mma(out[i % DB], f, pf[i / DB]); });
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
                read(DB * n + d, f);
                mma_seen(out[d], f, pf[n], seen);
                if (!BF16) __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // all parts to one maximum
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    if (h == 0) stats[wave][lane] = make_float2(m, l);
    __syncthreads();
    float all = -kInf, sum = 0;
#pragma unroll
    for (int p = 0; p < B::kParts; p++) all = fmaxf(all, stats[p * B::kBlocks + block][lane & 31].x);
    const float base = all == -kInf ? 0.f : all;
#pragma unroll
    for (int p = 0; p < B::kParts; p++) {
        const float2 of_part = stats[p * B::kBlocks + block][lane & 31];
        sum += of_part.y * __builtin_amdgcn_exp2f((of_part.x - base) * a.scale_log2);
    }
    const float f = __builtin_amdgcn_exp2f((m - base) * a.scale_log2);
#pragma unroll
    for (int d = 0; d < DB; d++) out[d] *= f;
    if (!add_parts<DB, B::kParts, B::kBlocks>(out, lds, part, block, lane) || !live) return;
    const float nan = __uint_as_float(0x7FC00000u);
    const bool none = all == -kInf && sum == 0.f;  // (as above)
    const float by = s.bad ? nan : none ? 0.f : 1.0f / sum;
    const int64_t o = token * a.ldo + (int64_t)head * D;
#pragma unroll
    for (int d = 0; d < DB; d++)
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int e = 0; e < 4; e++) store1<BF16>(a.out, o + 32 * d + 8 * j + 4 * h + e, nan_if_infinite(out[d][4 * j + e] * by));
    if (a.lse && h == 0) a.lse[token * a.q_heads + head] = s.bad ? nan : none ? -kInf : fmaf(all, a.scale, __builtin_amdgcn_logf(sum) * kLn2);
}

template <bool BF16, int D, bool DIRECT>
hipError_t launch_shape(const PackedArgs& a, hipStream_t s) {
    typedef ForwardShape<BF16, D> F;
    const int64_t groups = tile_slots(a.Tq, F::kRows, a.n) * a.q_heads;
    // Few, by calls of one prompt of 16 and 4 heads, us so and by parts.  200 tokens (32
    // groups), bf16, heads of 64 .. 256: 10 and 9, 12 and 10, 16 and 11, 18 and 15, 21 and 20;
    // 500 (64): 14 and 11, 16 and 14, 22 and 15, 29 and 21, 34 and 28; 1000 (128): 20 and 18, 24
    // and 28, 30 and 31, 44 and 43, 51 and 59; 1500 (192): 26 and 26 .. 65 and 116.  fp32, 1500:
    // 109 and 77, 146 and 107, 179 and 125, 250 and 172, 453 and 357; 3000 (384): 220 and 243,
    // 286 and 340, 350 and 395, 495 and 564, 998 and 1218.  (bf16 could go by parts up to about
    // 100 groups.)  Rows alone decide: few of them over many keys are passed over by few
    // workgroups (4 of 32 heads over 32768 keys 527 us).
    if (groups < (BF16 ? 64 : 200)) hipLaunchKernelGGL((attention_few_kernel<BF16, D, DIRECT>), dim3((unsigned)(tile_slots(a.Tq, PartsShape<BF16, D>::kOwn, a.n) * a.q_heads)), dim3(kPartsThreads), 0, s, a);
    else hipLaunchKernelGGL((attention_kernel<BF16, D, DIRECT>), dim3((unsigned)groups), dim3(F::kThreads), 0, s, a);
    return hipGetLastError();
}
template <bool BF16, int D>
hipError_t launch_forward(const PackedArgs& a, hipStream_t s) {
    const bool direct = direct_lines(a.k, a.ldk, BF16) && direct_lines(a.v, a.ldv, BF16);
    return direct ? launch_shape<BF16, D, true>(a, s) : launch_shape<BF16, D, false>(a, s);
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
