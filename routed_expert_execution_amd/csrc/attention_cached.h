// Attention over a paged cache held in 4 bits: the kernels.
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(scale_log2 q.k_j - m),
// with the running maximum m and both sums kept while the cache is read once.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attention_device.h"
#include "bf16_terms.h"

namespace moe {
namespace cached {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kWaves = 4, kThreads = 64 * kWaves, kStep = 32;  // tokens a wave takes at a time
constexpr float kInf = __builtin_huge_valf();

// The work of a call, for one key head: its row tiles (16 rows of a sequence's new
// tokens and the query heads of the key head), each through its sequence's rounds, one
// after another.  A round: a step of 32 tokens for each wave.  The line of all of them is
// cut into a.places runs of equal length, one for a workgroup; a tile that lies in
// several runs is joined from its parts afterwards.  (Chunks of one sequence each, a
// fourth of a run long where there was work for it, took 290 us where this takes 234: 40
// sequences of 1000 to 40000 tokens; 69 and 49: 64 of 2048; 631 and 210: one of 128 new
// tokens beside 63 single ones, of 8192.)
struct Work {
    int seq, begin, rows_new, length, first;  // first: the step that the sequence's rounds begin with
    int tile, rounds, start;                  // the tile's place on the line is [start, start + rounds)
    bool bad;                                 // not what it may be: its rows are NaN
};
// Sequence s: its tiles (none without new tokens) and each one's rounds.
struct Sequence { int begin, rows_new, length, first, tiles, rounds; bool bad; };
__device__ inline Sequence sequence_of(const CachedArgs& a, int s) {
    Sequence r;
    const int begin = a.batch.offsets[s], end = a.batch.offsets[s + 1], length = a.batch.lengths[s];
    r.bad = begin < 0 || end < begin || end > a.batch.T;
    r.begin = min(max(begin, 0), a.batch.T);
    r.rows_new = min(max(end, r.begin), a.batch.T) - r.begin;
    r.bad |= length < r.rows_new || length > (int64_t)a.batch.max_pages << a.cache.page_shift || r.rows_new > a.batch.most_new;
    r.length = r.bad ? 0 : length;
    const int first = a.window ? max(0, length - r.rows_new - a.window + 1) : 0;
    r.first = r.bad ? 0 : first / kStep;
    r.rounds = r.bad ? 1 : ((length + kStep - 1) / kStep - r.first + kWaves - 1) / kWaves;
    r.tiles = (int)(((int64_t)r.rows_new * a.per_head + 15) / 16);
    return r;
}

__device__ inline uint32_t wave_scan(uint32_t v) {  // inclusive, within the registers; stays at 2^32 - 1 once it is there
    auto add = [&](uint32_t x) { v = __builtin_elementwise_add_sat(v, x); };
    add(__builtin_amdgcn_update_dpp(0u, v, 0x111, 0xF, 0xF, false));  // from 1, 2, 4 and 8 lanes before, within 16
    add(__builtin_amdgcn_update_dpp(0u, v, 0x112, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0u, v, 0x114, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0u, v, 0x118, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0u, v, 0x142, 0xA, 0xF, false));  // the row before's last, then the half's
    add(__builtin_amdgcn_update_dpp(0u, v, 0x143, 0xC, 0xF, false));
    return v;
}
// Length of the line (and the sequences of the last 64 on the lanes), 0 where it passes 2^31: with good offsets and lengths it does not
// (the host sees to that), with others the call only reports them.
__device__ inline uint32_t line_of(const CachedArgs& a, Sequence* last) {
    const int lane = threadIdx.x & 63, n = a.batch.n;
    uint64_t total = 0;
    for (int base = 0; base < n; base += 64) {
        Sequence q{};
        if (base + lane < n) q = sequence_of(a, base + lane);
        *last = q;
        const uint32_t cost = (uint32_t)min((uint64_t)(uint32_t)q.tiles * (uint32_t)q.rounds, (uint64_t)1 << 31);
        total += (uint32_t)__builtin_amdgcn_readlane(wave_scan(cost), 63);
    }
    return total < (1u << 31) ? (uint32_t)total : 0;
}
// The tile at place `at` of the line, or the call's tile `at` (TILES).  Every wave finds
// it for itself, 64 sequences a pass, from where it found the one before (which does not
// lie after it).  all: the sequences, where there are no more than 64 and they are at hand.
struct Found { int base; uint32_t line, tiles; };  // a multiple of 64 sequences, and what lies before them
template <bool TILES>
__device__ inline bool find_work(const CachedArgs& a, uint32_t at, Work* out, Found* found, const Sequence* all) {
    const int lane = threadIdx.x & 63, n = a.batch.n;
    uint32_t before = found->line, tiles_before = found->tiles;
    for (int base = found->base; base < n; base += 64) {
        Sequence q{};
        if (all && n <= 64) q = *all;
        else if (base + lane < n) q = sequence_of(a, base + lane);
        const uint32_t line = wave_scan((uint32_t)q.tiles * (uint32_t)q.rounds), tiles = TILES ? wave_scan(q.tiles) : 0;
        const uint64_t past = __ballot((TILES ? tiles_before + tiles : before + line) > at);
        if (past) {
            const int k = __ffsll((unsigned long long)past) - 1;
            auto of_k = [&](int v) { return __builtin_amdgcn_readlane(v, k); };  // (wave-uniform, in scalar registers)
            out->seq = base + k;
            out->begin = of_k(q.begin);
            out->rows_new = of_k(q.rows_new);
            out->length = of_k(q.length);
            out->first = of_k(q.first);
            out->rounds = of_k(q.rounds);
            out->bad = of_k((int)q.bad);
            const uint32_t count = of_k(q.tiles), from = before + of_k(line) - count * out->rounds;
            out->tile = __builtin_amdgcn_readfirstlane(TILES ? at - (tiles_before + of_k(tiles) - count) : (at - from) / out->rounds);
            out->start = from + out->tile * out->rounds;
            *found = Found{base, before, tiles_before};
            return true;
        }
        before += __builtin_amdgcn_readlane(line, 63);
        if (TILES) tiles_before += __builtin_amdgcn_readlane(tiles, 63);
    }
    return false;
}
__device__ inline uint32_t run_of(const CachedArgs& a, uint32_t line) { return max((line + a.places - 1) / a.places, 1u); }
// Where the part of a tile that lies in run w is kept: a run has at most two that are
// not whole tiles, one that it begins with and one that it ends with.
__device__ inline int part_of(uint32_t run, int w, uint32_t start) { return 2 * w + (start > w * run); }

// Codes as bf16 16 + code, two to a word: part 0..3 takes bits 4 part..4 part + 3
// of each half word.
struct CodeMasks { uint32_t mask, bias; };
__device__ inline CodeMasks code_masks() {  // in registers, so that one instruction takes both
    CodeMasks c{0x00780078u, 0x41804180u};
    asm("" : "+s"(c.mask));
    asm("" : "+v"(c.bias));
    return c;
}
__device__ inline uint32_t codes16(uint32_t w, int part, const CodeMasks& c) {
    const uint32_t v = part == 0 ? w << 3 : part == 1 ? w >> 1 : part == 2 ? w >> 5 : w >> 9;
    return (v & c.mask) | c.bias;
}
// The same less 24: code - 8, which lies about zero as the values do.
__device__ inline uint32_t codes8(uint32_t w, int part, const CodeMasks& c) {
    const uint32_t v = codes16(w, part, c);
    const float lo = __uint_as_float(v << 16) - 24.f, hi = __uint_as_float(v & 0xFFFF0000u) - 24.f;  // (exact, in bf16 too)
    return __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xFFFF0000u);
}
// Maximum over the four 16-lane rows.
__device__ inline float cross_row_max(float v) {
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

template <int N> __device__ inline f32x4 product(bf16x8_t a, const bf16x8_t (&b)[N], f32x4 c) {
#pragma unroll
    for (int t = N - 1; t >= 0; t--) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[t], c, 0, 0, 0);
    return c;
}
template <int N> __device__ inline void terms_of(const float (&v)[8], bf16x8_t (&t)[N]) {
    if constexpr (N == 1) {
#pragma unroll
        for (int e = 0; e < 8; e++) t[0][e] = (__bf16)v[e];
    } else {
        bf16_terms(v, t);
    }
}

// W = D / 32, JP = group / 32.  A workgroup takes a run for one key head; the waves take
// the steps of 32 tokens of each tile's part in turn, each with sums of its own, joined
// at its end.
// Keys are the left operand of the first product, K Q^T, so that a lane holds four
// tokens of one row; these are, as they lie, the right operand of the second one,
// V^T P^T.  Neither goes through LDS.  Codes enter as they are held: the (step,
// lowest) pairs scale the first product's result and the second one's P.  P times
// the step is rounded to bf16 and multiplies code - 8, which lies about zero as the
// values do; the rest, lowest + 8 steps, is added in fp32.  (With code itself the
// result was 0.0031 off, its own rounding being 0.0016.)  P is rounded because two bf16
// terms of it, which leave the result's own rounding alone (0.0022 -> 0.0017 for one of 777
// tokens), take 140 us for 131 for the 64 sequences below and 57 for 52 for 130001 tokens;
// who needs it whole calls in fp32.
// Bound by the cache's bytes where sequences are long: 64 of up to 16000 tokens, 64 query
// and 8 key heads of 128, 126 us (3.9 TB/s); one of 130001 tokens, 32 and 8, 47 us (3.5
// TB/s); by latency where they are short: one of 777 tokens 7.5 us, the first read and one
// round.
template <int W, int JP, bool BF16>
__global__ __launch_bounds__(kThreads, cached_per_cu(W, BF16)) void cached_kernel(CachedArgs a) {
    constexpr int N = BF16 ? 1 : 3;  // bf16 terms of a factor
    // fp32: both products take code - 8, whose sums lose nothing to an offset; bf16, where
    // that is far below the rounding of P: 16 + code, and -24 by a product of its own in the second
    constexpr bool kCentred = !BF16;
    constexpr int D = 32 * W, G = W / JP;
    constexpr int kParams = (16 * G + 63) / 64;  // words of one tile's steps a lane loads
    // a step's (step, lowest) pairs: the step, and lowest + 8 steps (bf16: of keys lowest - 16 steps)
    __shared__ __attribute__((aligned(16))) float pairs[kWaves][4][2][16 * G];
    __shared__ float joined[2][16][D + 4];
    __shared__ float2 stats[kWaves][16];
    if (blockIdx.x == gridDim.x - 1) check_offsets(a.batch.offsets, a.batch.n, a.batch.T, a.err);
    const KvView& kv = a.cache;
    const int head = blockIdx.x % kv.heads, run_index = blockIdx.x / kv.heads;
    Sequence sequences;
    const uint32_t line = line_of(a, &sequences), run = __builtin_amdgcn_readfirstlane(run_of(a, line));
    const CodeMasks masks = code_masks();
    auto code = [&](uint32_t w, int part) { return kCentred ? codes8(w, part, masks) : codes16(w, part, masks); };
    const uint32_t head_bytes = (uint32_t)kv.tile_bytes << (kv.page_shift - 4), page_bytes = head_bytes * kv.heads;
    const uint8_t* heads_at = kv.data + (uint64_t)head * head_bytes;

    const uint32_t run_end = min((run_index + 1) * (uint64_t)run, (uint64_t)line);
    uint32_t place = run_index * (uint64_t)run < run_end ? run_index * run : run_end;
    Work c;
    Found found{};
    if (place >= run_end || !find_work<false>(a, place, &c, &found, &sequences)) return;
#pragma unroll 1
    for (;;) {
        // (what follows from the lane is worked out for each part: it is not kept beside the sums)
        int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        asm volatile("" : "+v"(lane), "+s"(wave));
        const int r16 = lane & 15, q4 = lane >> 4;
        const uint32_t part_end = min(run_end, (uint32_t)(c.start + c.rounds));
        const bool whole = place == (uint32_t)c.start && part_end == (uint32_t)(c.start + c.rounds);
        const int32_t* table = a.batch.pages + (int64_t)c.seq * a.batch.max_pages;
        const int rows = c.rows_new * a.per_head;
        const bool live = c.tile * 16 + r16 < rows;
        const int token = (c.tile * 16 + r16) / a.per_head;
        auto row_at = [&](int64_t ld) {  // (worked out where it is used: it is not kept through the loop)
            int row = c.tile * 16 + r16;
            asm("" : "+v"(row));
            const int of_token = row / a.per_head;
            return (int64_t)(c.begin + of_token) * ld + (int64_t)(head * a.per_head + row - of_token * a.per_head) * D;
        };
        // the row sees places from .. to - 1 (one past the last row all of them: it masks no step, and nothing of it is stored)
        const int old = c.length - c.rows_new, to = live ? old + token + 1 : INT32_MAX, from = live && a.window ? max(0, to - a.window) : 0;
        // the part's steps, less those at its ends that no row of the tile sees
        const int first_token = __builtin_amdgcn_readfirstlane(c.tile * 16 / a.per_head), last_token = __builtin_amdgcn_readfirstlane(min(c.tile * 16 + 15, rows - 1) / a.per_head);
        const int last_step = min(c.first + (int)(part_end - c.start) * kWaves, (old + last_token + kStep) / kStep);
        int step = c.first + (int)(place - c.start) * kWaves;
        const int tile_from = a.window ? old + first_token - a.window + 1 : 0;  // what lies before is seen by none: its pages may be gone
        step += max(0, tile_from / kStep - step) / kWaves * kWaves;
        step += wave;
        if (c.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);

        // (the first step's tokens on their way before the queries are waited for)
        bool bad = c.bad;

        struct Loaded { uint32_t k[2][W], v[2][W], steps[4][kParams]; };
        auto page_of = [&](int step, int i) -> int {  // wave-uniform
            const int at = step * kStep + 16 * i;
            return step < last_step && at < c.length && at + 16 > tile_from ? table[at >> kv.page_shift] : 0;
        };
        auto load = [&](int step, const int (&pages)[2], Loaded& d) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int at = step * kStep + 16 * i;
                int page = pages[i];
                if (page < 0 || page >= kv.pages) {
                    bad = true;
                    page = 0;
                }
                const uint32_t in = at & ((1 << kv.page_shift) - 1);
                const uint8_t* p = heads_at + (uint64_t)(uint32_t)page * page_bytes + (in >> 4) * (uint32_t)kv.tile_bytes;
                const uint8_t* pv = p + kv.tile_bytes / 2;
                __builtin_memcpy(d.k[i], p + lane * 4 * W, 4 * W);
                __builtin_memcpy(d.v[i], pv + lane * 4 * W, 4 * W);
                const uint32_t *ks = (const uint32_t*)(p + 256 * W), *vs = (const uint32_t*)(pv + 256 * W);
#pragma unroll
                for (int n = 0; n < kParams; n++) {
                    const int w = min(q4 + 4 * n, G - 1) * 16 + r16;
                    d.steps[i][n] = ks[w];
                    d.steps[2 + i][n] = vs[w];
                }
            }
        };
        Loaded now, next;
        int pages[2] = {page_of(step, 0), page_of(step, 1)};
        if (step < last_step) load(step, pages, now);
        pages[0] = page_of(step + kWaves, 0);
        pages[1] = page_of(step + kWaves, 1);

        bf16x8_t q[W][N];
        const int64_t q_at = row_at(a.ldq);
        float q_sum[G];
#pragma unroll
        for (int g = 0; g < G; g++) q_sum[g] = 0;
#pragma unroll
        for (int j = 0; j < W; j++) {
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (live) load8<BF16>(a.q, q_at + 32 * j + 8 * q4, v);
            terms_of<N>(v, q[j]);
            float s = 0;
#pragma unroll
            for (int e = 0; e < 8; e++) s += v[e];
            q_sum[j / JP] += cross_row_sum(s);
        }
        f32x4 out[2 * W];
        float low[G], m = -kInf, l = 0;
#pragma unroll
        for (int j = 0; j < 2 * W; j++) out[j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < G; g++) low[g] = 0;
#pragma unroll 1
        for (; step < last_step; step += kWaves) {
            // no value of the step is NaN or infinite.  What a sequence holds is not infinite,
            // but in place of a page before the tile's window page 0 is read, which nobody may
            // have written
            bool fine = true;
#pragma unroll
            for (int x = 0; x < 4; x++)
#pragma unroll
                for (int n = 0; n < kParams; n++)
                    if (lane + 64 * n < 16 * G) {
                        // past the sequence's end nothing has been written: step and lowest 0
                        const uint32_t w = step * kStep + 16 * (x & 1) + r16 < c.length ? now.steps[x][n] : 0u;
                        const float by = f16_bits_to_f32(w & 0xFFFF);
                        pairs[wave][x][0][lane + 64 * n] = by;
                        const float rest = fmaf(x < 2 && !kCentred ? -16.f : 8.f, by, f16_bits_to_f32(w >> 16));
                        pairs[wave][x][1][lane + 64 * n] = rest;
                        if (x >= 2) fine &= fabsf(rest) < kInf;  // (not so if either is infinite)
                    }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            if (step + kWaves < last_step) {
                load(step + kWaves, pages, next);
                pages[0] = page_of(step + 2 * kWaves, 0);
                pages[1] = page_of(step + 2 * kWaves, 1);
            }
            // scores of 8 tokens of the lane's row: 16 i + 4 q4 + e
            float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int g = 0; g < G; g++) {
                    f32x4 r = {0, 0, 0, 0};
#pragma unroll
                    for (int j = g * JP; j < (g + 1) * JP; j++) {
                        const u32x4 w = {code(now.k[i][j], 0), code(now.k[i][j], 1), code(now.k[i][j], 2), code(now.k[i][j], 3)};
                        r = product<N>(__builtin_bit_cast(bf16x8_t, w), q[j], r);
                    }
                    const int group = 16 * g + 4 * q4;
                    const f32x4 by = *(const f32x4*)&pairs[wave][i][0][group], less = *(const f32x4*)&pairs[wave][i][1][group];
#pragma unroll
                    for (int e = 0; e < 4; e++) s[4 * i + e] = fmaf(by[e], r[e], fmaf(less[e], q_sum[g], s[4 * i + e]));
                    __builtin_amdgcn_sched_barrier(0);
                }
            const int at = step * kStep;
            const bool all_seen = !__any(at + kStep > to || at < from);
            uint32_t seen = 0xFF;
            if (!all_seen) {
                seen = 0;
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int place = at + 16 * (e >> 2) + 4 * q4 + (e & 3);
                    const bool on = place < to && place >= from;
                    seen |= (uint32_t)on << e;
                    s[e] = on ? s[e] : -kInf;
                }
            }
            float top = s[0];
#pragma unroll
            for (int e = 1; e < 8; e++) top = fmaxf(top, s[e]);
            top = cross_row_max(top) * a.scale_log2;
            // (followed only where exponentials would pass 2^8: sums in fp32 and factors in
            // bf16 are as exact at any common scale)
            const float before = m;
            const bool grown = top - before > 8.f;
            if (__any(grown)) {
                m = grown ? top : before;
                const float f = grown ? __builtin_amdgcn_exp2f(before - top) : 1.f;
                l *= f;
#pragma unroll
                for (int j = 0; j < 2 * W; j++) out[j] *= f;
#pragma unroll
                for (int g = 0; g < G; g++) low[g] *= f;
            }
            const float base = m == -kInf ? 0.f : m;
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], a.scale_log2, -base));
                l += p[e];
            }
            auto values = [&](auto masked) {
#pragma unroll
                for (int g = 0; g < G; g++) {
                    float scaled[8];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const int group = 16 * g + 4 * q4;
                        const f32x4 by = *(const f32x4*)&pairs[wave][2 + i][0][group], middle = *(const f32x4*)&pairs[wave][2 + i][1][group];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            scaled[4 * i + e] = p[4 * i + e] * by[e];
                            if constexpr (masked.value) {  // a token that the row does not see adds nothing
                                const bool on = seen >> (4 * i + e) & 1;
                                scaled[4 * i + e] = on ? scaled[4 * i + e] : 0.f;
                                low[g] = on ? fmaf(p[4 * i + e], middle[e], low[g]) : low[g];
                            } else {
                                low[g] = fmaf(p[4 * i + e], middle[e], low[g]);
                            }
                        }
                    }
                    bf16x8_t b[N];
                    terms_of<N>(scaled, b);
#pragma unroll
                    for (int j = g * JP; j < (g + 1) * JP; j++) {
                        uint32_t w0 = now.v[0][j], w1 = now.v[1][j];
                        if constexpr (masked.value) asm("" : "+v"(w0), "+v"(w1));  // (so that the two branches' codes are not made before them)
                        const u32x4 lo = {code(w0, 0), code(w0, 2), code(w1, 0), code(w1, 2)};
                        const u32x4 hi = {code(w0, 1), code(w0, 3), code(w1, 1), code(w1, 3)};
                        if constexpr (!kCentred) {
                            const u32x4 bias = {0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};  // -24: code - 8 of 16 + code
                            out[2 * j] = product<N>(__builtin_bit_cast(bf16x8_t, bias), b, out[2 * j]);
                            out[2 * j + 1] = product<N>(__builtin_bit_cast(bf16x8_t, bias), b, out[2 * j + 1]);
                        }
                        out[2 * j] = product<N>(__builtin_bit_cast(bf16x8_t, lo), b, out[2 * j]);
                        out[2 * j + 1] = product<N>(__builtin_bit_cast(bf16x8_t, hi), b, out[2 * j + 1]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            };
            if (all_seen || !__any(!fine)) values(std::false_type{});
            else values(std::true_type{});
            now = next;
        }

        // the wave's sums to one scale for all waves, then waves 2 and 3 to 0 and 1, 1 to 0
        l = cross_row_sum(l);
        if (bad) l = __uint_as_float(0x7FC00000u);
        if (bad && !c.bad && lane == 0) atomicOr(a.err, kErrCache);
        if (q4 == 0) stats[wave][r16] = make_float2(m, l);
        __syncthreads();
        float all = -kInf, sum = 0;
#pragma unroll
        for (int w = 0; w < kWaves; w++) all = fmaxf(all, stats[w][r16].x);
        const float base = all == -kInf ? 0.f : all;
#pragma unroll
        for (int w = 0; w < kWaves; w++) sum += stats[w][r16].y * __builtin_amdgcn_exp2f(stats[w][r16].x - base);
        const float f = __builtin_amdgcn_exp2f(m - base);
#pragma unroll
        for (int g = 0; g < G; g++) low[g] = cross_row_sum(low[g]);
#pragma unroll
        for (int j = 0; j < 2 * W; j++) out[j] = (out[j] + low[j / 2 / JP]) * f;
#pragma unroll
        for (int half = 2; half >= 1; half /= 2) {
            if (wave >= half && wave < 2 * half)
#pragma unroll
                for (int j = 0; j < 2 * W; j++) *(f32x4*)&joined[wave - half][r16][16 * j + 4 * q4] = out[j];
            __syncthreads();
            if (wave < half)
#pragma unroll
                for (int j = 0; j < 2 * W; j++) out[j] += *(const f32x4*)&joined[wave][r16][16 * j + 4 * q4];
            __syncthreads();
        }
        if (wave == 0 && live) {
            if (whole) {
                const float by = 1.0f / sum;
                const int64_t at = row_at(a.ldo);
#pragma unroll
                for (int j = 0; j < 2 * W; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        store1<BF16>(a.out, at + 16 * j + 4 * q4 + e, out[j][e] * by);
            } else {
                const int64_t at = ((int64_t)part_of(run, run_index, place) * kv.heads + head) * a.part_rows + r16;
#pragma unroll
                for (int j = 0; j < 2 * W; j++) *(f32x4*)&a.part[at * D + 16 * j + 4 * q4] = out[j];
                if (q4 == 0) a.part_ml[at] = make_float2(all, sum);
            }
        }
        place = part_end;
        if (place >= run_end || !find_work<false>(a, place, &c, &found, nullptr)) return;
    }
}

// Rows of the tiles that were cut: their parts' sums, in the parts' order.  Rows of up to
// 16 parts are taken by a wave each, with more by a workgroup, each of its waves every
// 16th part: a row has up to a.places of them, of D fp32 values, and they are read at once.
// 6 to 9 us for the same calls, most of it one read after another.
// BY_TILE: a workgroup's tile is the call's tile blockIdx.x; otherwise the one that the
// end of run blockIdx.x cuts, if that is its first cut.
constexpr int kJoinWaves = 16, kJoinThreads = 64 * kJoinWaves;
template <bool BF16, bool BY_TILE>
__global__ __launch_bounds__(kJoinThreads) void cached_join_kernel(CachedArgs a) {
    __shared__ float sums[kJoinWaves][256];
    const int D = a.cache.D, heads = a.cache.heads, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Sequence sequences;
    const uint32_t line = line_of(a, &sequences), run = __builtin_amdgcn_readfirstlane(run_of(a, line));
    Work c;
    Found found{};
    const uint64_t cut = (blockIdx.x + 1) * (uint64_t)run;
    if (line == 0 || (!BY_TILE && cut >= line) || !find_work<BY_TILE>(a, BY_TILE ? blockIdx.x : (uint32_t)cut, &c, &found, &sequences)) return;
    const uint32_t start = c.start, end = start + c.rounds;
    if (!BY_TILE && (start >= cut || start + run < cut)) return;
    const int run_0 = start / run, of = (end - 1) / run - run_0 + 1;
    if (of == 1) return;
    const int live = min(16, c.rows_new * a.per_head - c.tile * 16), rows = live * heads;
    const int d0 = min(4 * lane, D - 4);  // (four channels a lane, past the last the last again)
    const int64_t per_part = (int64_t)heads * a.part_rows;
    // the place of a row's part i: the first's, then every second one from the next run on
    auto join = [&](int row, int first, int every, float* sum) -> f32x4 {  // this wave's parts, to the row's scale
        const int head = row / live, r = row - head * live;
        const int64_t at = (int64_t)head * a.part_rows + r;
        auto place = [&](int i) { return at + (i ? 2 * (run_0 + i) : part_of(run, run_0, start)) * per_part; };
        constexpr int kBatch = 4;
        f32x4 part[kBatch];  // the next ones, on their way before the stats are waited for
        auto load = [&](int i) {
#pragma unroll
            for (int x = 0; x < kBatch; x++)
                if (i + x * every < of) part[x] = *(const f32x4*)&a.part[place(i + x * every) * D + d0];
        };
        load(first);
        auto stats_of = [&](int i) { return i < of ? a.part_ml[place(i)] : make_float2(-kInf, 0.f); };
        float2 ml = stats_of(lane);  // 64 parts at a time, one a lane
        float m = ml.x, l = 0;
        for (int i = lane + 64; i < of; i += 64) m = fmaxf(m, a.part_ml[place(i)].x);
#pragma unroll
        for (int x = 1; x < 64; x *= 2) m = fmaxf(m, __shfl_xor(m, x));
        const float base = m == -kInf ? 0.f : m;
        f32x4 v = {0, 0, 0, 0};
        int i = first;
        for (int i0 = 0;;) {
            const float f = __builtin_amdgcn_exp2f(ml.x - base);
            l += ml.y * f;
            const int end = min(i0 + 64, of);
            while (i < end) {
#pragma unroll
                for (int x = 0; x < kBatch; x++)
                    if (i + x * every < end) v += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i + x * every - i0)) * part[x];
                i += kBatch * every;  // (divides 64)
                load(i);
            }
            i0 += 64;
            if (i0 >= of) break;
            ml = stats_of(i0 + lane);
        }
        *sum = seg_sum<64>(l);
        return v;
    };
    auto out_at = [&](int row) {
        const int head = row / live, r = c.tile * 16 + row - head * live, token = r / a.per_head;
        return (int64_t)(c.begin + token) * a.ldo + (int64_t)(head * a.per_head + r - token * a.per_head) * D;
    };
    if (of <= kJoinWaves) {
        for (int row = blockIdx.y * kJoinWaves + wave; row < rows; row += gridDim.y * kJoinWaves) {
            float sum;
            const f32x4 v = join(row, 0, 1, &sum);
            if (4 * lane < D)
#pragma unroll
                for (int e = 0; e < 4; e++) store1<BF16>(a.out, out_at(row) + d0 + e, v[e] / sum);
        }
        return;
    }
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
        float sum;
        const f32x4 v = join(row, wave, kJoinWaves, &sum);
        if (4 * lane < D) *(f32x4*)&sums[wave][d0] = v;
        __syncthreads();
        if (threadIdx.x < D) {
            float o = 0;
#pragma unroll
            for (int w = 0; w < kJoinWaves; w++) o += sums[w][threadIdx.x];
            store1<BF16>(a.out, out_at(row) + threadIdx.x, o / sum);
        }
        __syncthreads();
    }
}

template <int W, int JP, bool BF16>
hipError_t launch(const CachedArgs& a, const CachedPlan& p, hipStream_t s) {
    hipLaunchKernelGGL((cached_kernel<W, JP, BF16>), dim3(p.places * a.cache.heads), dim3(kThreads), 0, s, a);
    if (p.split) {
        const int cuts = p.places - 1, rows = a.part_rows * a.cache.heads;
        const bool by_tile = p.tiles <= cuts;
        const dim3 grid(by_tile ? (int)p.tiles : cuts, std::max(1, std::min(rows, 512 / (by_tile ? (int)p.tiles : cuts))));
        if (by_tile) hipLaunchKernelGGL((cached_join_kernel<BF16, true>), grid, dim3(kJoinThreads), 0, s, a);
        else hipLaunchKernelGGL((cached_join_kernel<BF16, false>), grid, dim3(kJoinThreads), 0, s, a);
    }
    return hipGetLastError();
}
template <int W, bool BF16>
hipError_t launch_by_group(const CachedArgs& a, const CachedPlan& p, hipStream_t s) {
    if constexpr (W % 2 == 0)
        if (a.cache.group_shift == 1) return launch<W, 2, BF16>(a, p, s);
    if constexpr (W % 4 == 0)
        if (a.cache.group_shift == 2) return launch<W, 4, BF16>(a, p, s);
    return launch<W, 1, BF16>(a, p, s);
}
template <bool BF16>
hipError_t launch_by_width(const CachedArgs& a, const CachedPlan& p, hipStream_t s) {
    switch (a.cache.words) {
        case 2: return launch_by_group<2, BF16>(a, p, s);
        case 3: return launch_by_group<3, BF16>(a, p, s);
        case 4: return launch_by_group<4, BF16>(a, p, s);
        case 6: return launch_by_group<6, BF16>(a, p, s);
        default: return launch_by_group<8, BF16>(a, p, s);
    }
}

}  // namespace cached
}  // namespace moe
