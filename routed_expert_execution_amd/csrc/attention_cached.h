// Attention over a paged cache held in 4 bits: the kernels.
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(scale_log2 q.k_j - m),
// with the running maximum m and both sums kept while the cache is read once.
#pragma once

#include <type_traits>

#include "attention_device.h"
#include "bf16_terms.h"

namespace moe {
namespace cached {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kWaves = 4, kThreads = 64 * kWaves, kStep = 32;  // tokens a wave takes at a time
constexpr float kInf = __builtin_huge_valf();

// Where a chunk lies.
struct Chunk {
    int seq, begin, rows_new, length, first, steps;  // first: step of 32 tokens it begins with
    int index, of;                                    // chunk of the sequence, how many it has
    int slot;                                         // its place among the partial results
    bool bad;
};

// A sequence as every chunk sees it: steps that its new tokens read, 1 where it is
// not what it may be (one chunk then says so), 0 without new tokens.
struct Sequence { int begin, rows_new, length, first, steps; bool bad; };
__device__ inline Sequence sequence_of(const CachedArgs& a, int s) {
    Sequence r;
    const int begin = a.batch.offsets[s], end = a.batch.offsets[s + 1], length = a.batch.lengths[s];
    r.bad = begin < 0 || end < begin || end > a.batch.T;
    r.begin = min(max(begin, 0), a.batch.T);
    r.rows_new = min(max(end, r.begin), a.batch.T) - r.begin;
    r.bad |= length < r.rows_new || length > (int64_t)a.batch.max_pages << a.cache.page_shift || r.rows_new > a.batch.most_new;
    r.length = r.bad ? 0 : length;
    const int first = a.window ? max(0, length - r.rows_new - a.window + 1) : 0;
    r.first = first / kStep;
    r.steps = r.bad ? 1 : r.rows_new ? (length + kStep - 1) / kStep - r.first : 0;
    if (r.bad && !r.rows_new) r.steps = 0;
    return r;
}

// Chunk `w` of the call: all steps of all sequences cut into about `target` chunks
// of equal size, none over two sequences.  Every wave finds it for itself, 64
// sequences a pass.  A sequence that is cut has more than 1 / target of all steps,
// so there are fewer than `target` of them, with fewer than 2 target chunks.
__device__ inline uint32_t wave_scan(uint32_t v) {  // inclusive, within the registers
    v += __builtin_amdgcn_update_dpp(0u, v, 0x111, 0xF, 0xF, false);  // from 1, 2, 4 and 8 lanes before, within 16
    v += __builtin_amdgcn_update_dpp(0u, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0u, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0u, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0u, v, 0x142, 0xA, 0xF, false);  // the row before's last, then the half's
    v += __builtin_amdgcn_update_dpp(0u, v, 0x143, 0xC, 0xF, false);
    return v;
}
__device__ inline int chunk_steps(int64_t total, const CachedArgs& a) {
    // a chunk for each place of the card, or a few where there is work for several
    // rounds: the last of them leaves less of the card idle
    const int64_t rounds = min(max(total * a.row_tiles / ((int64_t)a.places * 24), (int64_t)1), (int64_t)a.rounds), target = a.places * rounds;
    const int64_t c = (total + target - 1) / target;
    return (int)((max(c, (int64_t)1) + kWaves - 1) / kWaves * kWaves);
}
// which(chunks so far, chunks of it, cut sequences so far): the wanted sequence.
// CUT: `w` counts the sequences that are cut, in place of chunks.
template <bool CUT>
__device__ inline bool find_chunk(const CachedArgs& a, int w, Chunk* out) {
    const int lane = threadIdx.x & 63, n = a.batch.n;
    Sequence q{};
    int64_t total = 0;
    for (int base = 0; base < n; base += 64) {
        q = Sequence{};
        if (base + lane < n) q = sequence_of(a, base + lane);
        total += (uint32_t)__builtin_amdgcn_readlane(wave_scan(q.steps), 63);  // (64 times 2^25 at most)
    }
    const int steps = __builtin_amdgcn_readfirstlane(chunk_steps(total, a));
    int chunks_before = 0, cut_before = 0, slots_before = 0;
    for (int base = 0; base < n; base += 64) {
        if (n > 64) {
            q = Sequence{};
            if (base + lane < n) q = sequence_of(a, base + lane);
        }
        const int of = (q.steps + steps - 1) / steps, cut = of > 1;
        const int chunks = wave_scan(of), cuts = CUT ? wave_scan(cut) : 0, slots = wave_scan(cut ? of : 0);
        const int mine = CUT ? cut_before + cuts : chunks_before + chunks;
        const uint64_t past = __ballot(mine > w);
        if (past) {
            const int k = __ffsll((unsigned long long)past) - 1;
            out->seq = base + k;
            auto of_k = [&](int v) { return __builtin_amdgcn_readlane(v, k); };  // (wave-uniform, in scalar registers)
            out->begin = of_k(q.begin);
            out->rows_new = of_k(q.rows_new);
            out->length = of_k(q.length);
            out->bad = of_k((int)q.bad);
            out->of = of_k(of);
            out->index = CUT ? 0 : w - (chunks_before + of_k(chunks) - out->of);
            out->slot = slots_before + of_k(slots) - (out->of > 1 ? out->of : 0) + out->index;
            const int all = of_k(q.steps);
            out->first = of_k(q.first) + out->index * steps;
            out->steps = min(steps, all - out->index * steps);
            return true;
        }
        chunks_before += __builtin_amdgcn_readlane(chunks, 63);
        if (CUT) cut_before += __builtin_amdgcn_readlane(cuts, 63);
        slots_before += __builtin_amdgcn_readlane(slots, 63);
    }
    return false;
}

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

// W = D / 32, JP = group / 32.  A workgroup takes one chunk of a sequence's tokens, one key head and
// 16 rows (new tokens times the query heads of that key head); its waves take the
// chunk's steps of 32 tokens in turn, each with sums of its own, joined at the end.
// Keys are the left operand of the first product, K Q^T, so that a lane holds four
// tokens of one row; these are, as they lie, the right operand of the second one,
// V^T P^T.  Neither goes through LDS.  Codes enter as they are held: the (step,
// lowest) pairs scale the first product's result and the second one's P.  P times
// the step is rounded to bf16 and multiplies code - 8, which lies about zero as the
// values do; the rest, lowest + 8 steps, is added in fp32.  (With code itself the
// result was 0.0031 off, its own rounding being 0.0016.)
template <int W, int JP, bool BF16>
__global__ __launch_bounds__(kThreads, W <= 4 ? (BF16 ? 3 : 2) : W <= 6 ? 2 : 1) void cached_kernel(CachedArgs a) {
    constexpr int N = BF16 ? 1 : 3;  // bf16 terms of a factor
    constexpr int D = 32 * W, G = W / JP;
    constexpr int kParams = (16 * G + 63) / 64;  // words of one tile's steps a lane loads
    // a step's (step, lowest) pairs: of keys the step and lowest - 16 steps, of values the step and lowest + 8 steps
    __shared__ __attribute__((aligned(16))) float pairs[kWaves][4][2][16 * G];
    __shared__ float joined[2][16][D + 4];
    __shared__ float2 stats[kWaves][16];
    if (blockIdx.x == gridDim.x - 1) check_offsets(a.batch.offsets, a.batch.n, a.batch.T, a.err);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q4 = lane >> 4;
    // (all of a chunk's workgroups side by side: those of chunks that there are not come last)
    const KvView& kv = a.cache;
    const int units = kv.heads * a.row_tiles, unit = blockIdx.x % units, head = unit % kv.heads;
    Chunk c;
    if (!find_chunk<false>(a, blockIdx.x / units, &c)) return;
    const int rows = c.rows_new * a.per_head;
    if (c.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);
    const CodeMasks masks = code_masks();
    const int32_t* table = a.batch.pages + (int64_t)c.seq * a.batch.max_pages;
    const int last_step = c.first + c.steps;
    const uint32_t head_bytes = (uint32_t)kv.tile_bytes << (kv.page_shift - 4), page_bytes = head_bytes * kv.heads;
    const uint8_t* heads_at = kv.data + (uint64_t)head * head_bytes;

#pragma unroll 1
    for (int tile = unit / kv.heads; tile * 16 < rows; tile += a.row_tiles) {
        const int row = tile * 16 + r16, token = row / a.per_head, q_head = head * a.per_head + row - token * a.per_head;
        const bool live = row < rows;
        // the row sees places from .. to - 1 (one past the last row all of them: it masks no step, and nothing of it is stored)
        const int to = live ? c.length - c.rows_new + token + 1 : INT32_MAX, from = live && a.window ? max(0, to - a.window) : 0;

        // (the first step's tokens on their way before the queries are waited for)
        bool bad = c.bad;

        struct Loaded { uint32_t k[2][W], v[2][W], steps[4][kParams]; };
        auto page_of = [&](int step, int i) -> int {  // wave-uniform
            const int at = step * kStep + 16 * i;
            return step < last_step && at < c.length ? table[at >> kv.page_shift] : 0;
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
        int step = c.first + wave;
        int pages[2] = {page_of(step, 0), page_of(step, 1)};
        if (step < last_step) load(step, pages, now);
        pages[0] = page_of(step + kWaves, 0);
        pages[1] = page_of(step + kWaves, 1);

        bf16x8_t q[W][N];
        float q_sum[G];
#pragma unroll
        for (int g = 0; g < G; g++) q_sum[g] = 0;
#pragma unroll
        for (int j = 0; j < W; j++) {
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (live) load8<BF16>(a.q, (int64_t)(c.begin + token) * a.ldq + (int64_t)q_head * D + 32 * j + 8 * q4, v);
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
            bool fine = true;  // no value of the step is NaN
#pragma unroll
            for (int x = 0; x < 4; x++)
#pragma unroll
                for (int n = 0; n < kParams; n++)
                    if (lane + 64 * n < 16 * G) {
                        // past the sequence's end nothing has been written: step and lowest 0
                        const uint32_t w = step * kStep + 16 * (x & 1) + r16 < c.length ? now.steps[x][n] : 0u;
                        const float by = f16_bits_to_f32(w & 0xFFFF);
                        pairs[wave][x][0][lane + 64 * n] = by;
                        const float rest = fmaf(x < 2 ? -16.f : 8.f, by, f16_bits_to_f32(w >> 16));
                        pairs[wave][x][1][lane + 64 * n] = rest;
                        if (x >= 2) fine &= rest == rest;
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
                        const u32x4 w = {codes16(now.k[i][j], 0, masks), codes16(now.k[i][j], 1, masks), codes16(now.k[i][j], 2, masks), codes16(now.k[i][j], 3, masks)};
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
                        const u32x4 lo = {codes16(w0, 0, masks), codes16(w0, 2, masks), codes16(w1, 0, masks), codes16(w1, 2, masks)};
                        const u32x4 hi = {codes16(w0, 1, masks), codes16(w0, 3, masks), codes16(w1, 1, masks), codes16(w1, 3, masks)};
                        const u32x4 bias = {0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};  // -24: code - 8 of 16 + code
                        out[2 * j] = product<N>(__builtin_bit_cast(bf16x8_t, bias), b, out[2 * j]);
                        out[2 * j + 1] = product<N>(__builtin_bit_cast(bf16x8_t, bias), b, out[2 * j + 1]);
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
            if (c.of == 1) {
                const float by = 1.0f / sum;
#pragma unroll
                for (int j = 0; j < 2 * W; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        store1<BF16>(a.out, (int64_t)(c.begin + token) * a.ldo + (int64_t)q_head * D + 16 * j + 4 * q4 + e, out[j][e] * by);
            } else {
                const int64_t at = (int64_t)c.slot * a.batch.most_new * a.q_heads + (int64_t)token * a.q_heads + q_head;
#pragma unroll
                for (int j = 0; j < 2 * W; j++) *(f32x4*)&a.part[at * D + 16 * j + 4 * q4] = out[j];
                if (q4 == 0) a.part_ml[at] = make_float2(all, sum);
            }
        }
    }
}

// Rows of the sequences that were cut: their chunks' sums, in the chunks' order.  Rows
// of up to 16 chunks are taken by a wave each, with more by a workgroup, each of its
// waves every 16th chunk: a row has up to `target` of them, of D fp32 values, and they
// are read at once.
constexpr int kJoinWaves = 16, kJoinThreads = 64 * kJoinWaves;
template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void cached_join_kernel(CachedArgs a) {
    __shared__ float sums[kJoinWaves][256];
    const int D = a.cache.D, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Chunk c;
    if (!find_chunk<true>(a, blockIdx.x, &c)) return;
    const int64_t per_chunk = (int64_t)a.batch.most_new * a.q_heads;
    const int rows = c.rows_new * a.q_heads, d0 = min(4 * lane, D - 4);  // (four channels a lane, past the last the last again)
    auto join = [&](int row, int first, int every, float* sum) -> f32x4 {  // this wave's chunks, to the row's scale
        const int64_t at = (int64_t)c.slot * per_chunk + row;
        float m = -kInf, l = 0;
        for (int i = lane; i < c.of; i += 64) m = fmaxf(m, a.part_ml[at + i * per_chunk].x);
#pragma unroll
        for (int x = 1; x < 64; x *= 2) m = fmaxf(m, __shfl_xor(m, x));
        const float base = m == -kInf ? 0.f : m;
        for (int i = lane; i < c.of; i += 64) {
            const float2 ml = a.part_ml[at + i * per_chunk];
            l += ml.y * __builtin_amdgcn_exp2f(ml.x - base);
        }
        *sum = seg_sum<64>(l);
        f32x4 v = {0, 0, 0, 0};
#pragma unroll 4
        for (int i = first; i < c.of; i += every) {
            const float f = __builtin_amdgcn_exp2f(a.part_ml[at + i * per_chunk].x - base);
            v += f * *(const f32x4*)&a.part[(at + i * per_chunk) * D + d0];
        }
        return v;
    };
    auto out_at = [&](int row) {
        const int token = row / a.q_heads, q_head = row - token * a.q_heads;
        return (int64_t)(c.begin + token) * a.ldo + (int64_t)q_head * D;
    };
    if (c.of <= kJoinWaves) {
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
hipError_t launch(const CachedArgs& a, int split, hipStream_t s) {
    const dim3 grid((a.batch.n + (split ? a.target : 0)) * a.cache.heads * a.row_tiles);
    hipLaunchKernelGGL((cached_kernel<W, JP, BF16>), grid, dim3(kThreads), 0, s, a);
    if (split) {
        // (fewer than `target` sequences are cut)
        const int cut = a.batch.n < a.target ? a.batch.n : a.target, rows = a.batch.most_new * a.q_heads, share = 512 / cut;
        hipLaunchKernelGGL((cached_join_kernel<BF16>), dim3(cut, rows < share ? rows : share < 1 ? 1 : share), dim3(kJoinThreads), 0, s, a);
    }
    return hipGetLastError();
}
template <int W, bool BF16>
hipError_t launch_by_group(const CachedArgs& a, int split, hipStream_t s) {
    if constexpr (W % 2 == 0)
        if (a.cache.group_shift == 1) return launch<W, 2, BF16>(a, split, s);
    if constexpr (W % 4 == 0)
        if (a.cache.group_shift == 2) return launch<W, 4, BF16>(a, split, s);
    return launch<W, 1, BF16>(a, split, s);
}
template <bool BF16>
hipError_t launch_by_width(const CachedArgs& a, int split, hipStream_t s) {
    switch (a.cache.words) {
        case 2: return launch_by_group<2, BF16>(a, split, s);
        case 3: return launch_by_group<3, BF16>(a, split, s);
        case 4: return launch_by_group<4, BF16>(a, split, s);
        case 6: return launch_by_group<6, BF16>(a, split, s);
        default: return launch_by_group<8, BF16>(a, split, s);
    }
}

}  // namespace cached
}  // namespace moe
