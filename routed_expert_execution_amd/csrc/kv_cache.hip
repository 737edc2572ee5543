// Keys and values into a paged cache held in 4 bits, and back.  By token, head and
// group of channels, for x the value (a key after its rotation):
//   lowest = fp16(min x),  step = fp16((max x - lowest) / 15),
//   code = round((x - lowest) / step) in 0..15 (step 0: 0),  value = lowest + step * code.
#include <algorithm>

#include "rotary_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kTokens = 4;  // of a workgroup, where there are many tokens

// Reductions over a group's neighbouring threads (N = group / 8 of them, aligned), by
// the partner exchanges of seg_sum.
template <int CTRL> __device__ inline double dpp_f64(double v) { return __builtin_bit_cast(double, dpp_u64<CTRL>(__builtin_bit_cast(uint64_t, v))); }
template <typename F> __device__ inline float over_group(float v, int n, F f) {
    v = f(v, dpp_f<0xB1>(v));
    v = f(v, dpp_f<0x4E>(v));
    if (n > 4) v = f(v, dpp_f<0x141>(v));
    if (n > 8) v = f(v, dpp_f<0x140>(v));
    return v;
}

// Eight channels of a thread to codes.  Which of two values next to their border a step
// or a code takes is decided in 64 bits, by the value and not by roundings on the way;
// but only there, and 32 bits say where that is: x less the lowest value is taken in 64
// bits (its own rounding to fp32 would be up to |x| 2^-24, many steps' parts where a group
// lies far from zero for how far its values lie apart), so that the quotients are within
// 2^-21 of theirs, relative, of 15 at most.
// Returns eight codes, four bits each; *steps the word that stands for the group.
__device__ inline uint32_t to_codes(const double (&x)[8], int group, uint32_t* steps) {
    const int n = group / 8;
    float xf[8], lo, hi;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        xf[i] = (float)x[i];
        lo = i ? fminf(lo, xf[i]) : xf[i];
        hi = i ? fmaxf(hi, xf[i]) : xf[i];
        fine &= fabs(x[i]) <= 65504.0;  // (false for a NaN)
    }
    lo = over_group(lo, n, [](float a, float b) { return fminf(a, b); });
    hi = over_group(hi, n, [](float a, float b) { return fmaxf(a, b); });
    const bool all_fine = over_group(fine ? 1.f : 0.f, n, [](float a, float b) { return fminf(a, b); }) != 0.f;
    const _Float16 low16 = (_Float16)lo;  // (rounding keeps order: the fp32 of the lowest value)
    const float low = (float)low16;
    // the step, and whether its rounding to fp16 is certain: not within 2^-20 of it of a
    // border, which lies half way between two fp16 values
    float exact_step = (hi - low) / 15.0f;
    const float slack = fabsf(exact_step) * 0x1p-20f + fabsf(low) * 0x1p-26f;
    if (__any((_Float16)(exact_step - slack) != (_Float16)(exact_step + slack))) {
        double top = x[0];
#pragma unroll
        for (int i = 1; i < 8; i++) top = fmax(top, x[i]);
        top = fmax(top, dpp_f64<0xB1>(top));
        top = fmax(top, dpp_f64<0x4E>(top));
        if (n > 4) top = fmax(top, dpp_f64<0x141>(top));
        if (n > 8) top = fmax(top, dpp_f64<0x140>(top));
        exact_step = (float)((top - (double)low) / 15.0);
    }
    const _Float16 step16 = (_Float16)exact_step;
    const float step = (float)step16;
    // a group with a value that is none reads back as NaN
    *steps = all_fine ? (uint32_t)__builtin_bit_cast(uint16_t, step16) | (uint32_t)__builtin_bit_cast(uint16_t, low16) << 16 : 0x7E007E00u;
    const bool some = all_fine && step > 0.f;
    const float inverse = some ? 1.0f / step : 0.f;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float t = fminf(fmaxf((float)(x[i] - (double)low) * inverse, 0.f), 15.f);
        float q = rintf(t);
        const bool near = some && fabsf(fabsf(t - q) - 0.5f) < 1e-4f;
        if (__any(near)) {  // halves go to the even code
            const double left = 2.0 * fma(-(double)q, (double)step, x[i] - (double)low);
            const bool odd = (int)q & 1;
            if (near && (left > (double)step || (left == (double)step && odd))) q += 1.f;
            else if (near && (left < -(double)step || (left == -(double)step && odd))) q -= 1.f;
            q = fminf(fmaxf(q, 0.f), 15.f);
        }
        codes |= (uint32_t)(int)(some ? q : 0.f) << (4 * i);
    }
    return codes;
}

__device__ inline uint8_t* tile_at(const KvView& c, int page, int head, int in_page) {
    return c.data + (((int64_t)page * c.heads + head) * (1 << (c.page_shift - 4)) + (in_page >> 4)) * c.tile_bytes;
}
__device__ inline int value_byte(int t) { return (t & 1) * 2 + (t >> 1 & 1); }  // place of token t % 4 in its word

// What a workgroup knows of each of its tokens.
struct TokenInfo { int place, page, in_page, has; };  // has: 0 no sequence, 1 one, 2 and a page
__device__ inline TokenInfo info_of(const KvView& c, const KvBatchView& b, int token, int* err) {
    TokenInfo t{};
    TokenPlace p;
    if (!find_token(b, token, &p)) {
        if (p.bad && (threadIdx.x & 63) == 0) atomicOr(err, kErrCache);
        return t;
    }
    t.has = 1;
    t.place = (int)p.place;
    if (!p.bad && p.place >= 0 && p.place < (int64_t)b.max_pages << c.page_shift) {
        t.page = b.pages[(int64_t)p.seq * b.max_pages + (p.place >> c.page_shift)];
        t.in_page = (int)(p.place & ((1 << c.page_shift) - 1));
        if (t.page >= 0 && t.page < c.pages) t.has = 2;
    }
    if (t.has != 2 && (threadIdx.x & 63) == 0) atomicOr(err, kErrCache);
    return t;
}

// The first token of a workgroup.  Tokens side by side share lines of the cache, which
// is written a few bytes a token: where there are many tokens, workgroups that go to one
// XCD (every eighth) take a run of them, so that its L2 has whole lines to write back.
__device__ inline int first_token(int tokens) {
    if (tokens == 1) return blockIdx.x;
    const int per = gridDim.x / 8;  // (a multiple of 8 workgroups)
    return (blockIdx.x % 8 * per + blockIdx.x / 8) * tokens;
}

// `tokens` tokens a workgroup (or gridDim.y workgroups for one, where tokens are few):
// a wave finds each one's place; their angles once into LDS; then eight channels a
// thread of keys, of values, and eight pairs of queries.  Bound by bytes in flight
// (leaving out the codes' arithmetic, their stores or the cosines changes nothing):
// five prompts, 32 query and 8 key heads of 128 in bf16, 86 us, 2.8 TB/s of the 242 MB
// read and written (waves wait for 0.56 of their time and issue vector instructions for
// 0.19); 64 single tokens 6.5 us, the launch and one read after another.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendArgs a, int tokens) {
    __shared__ double2 turns[kTokens][128];
    __shared__ float2 turns_q[kTokens][128];
    __shared__ TokenInfo infos[kTokens];
    const int first = first_token(tokens), count = min(tokens, a.batch.T - first), wave = threadIdx.x >> 6;
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == 0) check_offsets(a.batch.offsets, a.batch.n, a.batch.T, a.err);
    if (wave < count) {
        const TokenInfo t = info_of(a.cache, a.batch, first + wave, a.err);
        if ((threadIdx.x & 63) == 0) infos[wave] = t;
    }
    __syncthreads();
    const RotaryView r = a.rotary;
    if (r.freqs) {
        for (int i = threadIdx.x; i < count * r.half; i += kThreads) {
            const int t = i / r.half, p = i - t * r.half;
            double c, s;
            turn_of(a.positions ? a.positions[first + t] : infos[t].place, r.freqs[p], &c, &s);
            c *= r.scale;
            s *= r.scale;
            turns[t][p] = make_double2(c, s);
            turns_q[t][p] = make_float2((float)c, (float)s);
        }
        __syncthreads();
    }
    const KvView& c = a.cache;
    const int per_row = c.D / 8, keys = c.heads * per_row, group = 32 << c.group_shift;
    const int units = a.q ? rotate_units(r.half, c.D, a.q == a.q_out) : 0;
    const int total = 2 * keys + a.q_heads * units;
    // A thread does the same unit of all tokens, and all of them are read before the
    // first is worked on: a workgroup is bound by the time that a read takes.
    // (whole groups of channels lie on neighbouring threads: keys is a multiple of group / 8)
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < total; i += gridDim.y * kThreads) {
        if (i >= 2 * keys) {
            const int h = (i - 2 * keys) / units, u = (i - 2 * keys) - h * units;
            RotateUnit<BF16> unit(r, c.D, u);
#pragma unroll
            for (int t = 0; t < kTokens; t++)
                if (t < count && infos[t].has) unit.load(t, a.q, (first + t) * a.ldq + (int64_t)h * c.D);
#pragma unroll
            for (int t = 0; t < kTokens; t++)
                if (t < count && infos[t].has) unit.finish(t, a.q, (first + t) * a.ldq + (int64_t)h * c.D, a.q_out, (first + t) * a.ldqo + (int64_t)h * c.D, turns_q[t]);
            continue;
        }
        const bool value = i >= keys;
        const int row = value ? i - keys : i, head = row / per_row, chunk = row - head * per_row, c0 = 8 * chunk;
        const void* p = value ? a.v : a.k;
        const int64_t ld = value ? a.ldv : a.ldk, in_row = (int64_t)head * c.D;
        const bool turned = !value && r.freqs && c0 < 2 * r.half, halves = turned && !r.interleaved;
        Raw8<BF16> own[kTokens], other[kTokens];  // the chunk, and its channels' partners
#pragma unroll
        for (int t = 0; t < kTokens; t++)
            if (t < count && infos[t].has == 2) {
                own[t].load(p, (first + t) * ld + in_row + c0);
                if (halves && r.half % 8 == 0) other[t].load(p, (first + t) * ld + in_row + (c0 < r.half ? c0 + r.half : c0 - r.half));
            }
#pragma unroll
        for (int t = 0; t < kTokens; t++) {
            if (t >= count || infos[t].has != 2) continue;
            const TokenInfo info = infos[t];
            float mine[8], partner[8];
            own[t].get(mine);
            double x[8];
#pragma unroll
            for (int e = 0; e < 8; e++) x[e] = (double)mine[e];
            if (turned && r.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    if (c0 + e < 2 * r.half) {
                        const double2 w = turns[t][(c0 + e) / 2];
                        const double v0 = x[e], v1 = x[e + 1];
                        x[e] = v0 * w.x - v1 * w.y;
                        x[e + 1] = v0 * w.y + v1 * w.x;
                    }
            } else if (halves) {
                if (r.half % 8 == 0) {
                    other[t].get(partner);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int ch = c0 + e;
                        partner[e] = ch < 2 * r.half ? load1<BF16>(p, (first + t) * ld + in_row + (ch < r.half ? ch + r.half : ch - r.half)) : 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int ch = c0 + e;
                    if (ch < r.half) {
                        const double2 w = turns[t][ch];
                        x[e] = x[e] * w.x - (double)partner[e] * w.y;
                    } else if (ch < 2 * r.half) {
                        const double2 w = turns[t][ch - r.half];
                        x[e] = (double)partner[e] * w.y + x[e] * w.x;
                    }
                }
            }
            uint32_t steps;
            const uint32_t codes = to_codes(x, group, &steps);
            uint8_t* tile = tile_at(c, info.page, head, info.in_page) + (value ? c.tile_bytes / 2 : 0);
            const int in = info.in_page & 15, j = chunk >> 2;
            if (chunk % (group / 8) == 0) ((uint32_t*)(tile + 256 * c.words))[c0 / group * 16 + in] = steps;
            // channels 16 apart share a byte of the values: the threads of each pair write half of theirs
            const uint32_t theirs = __builtin_amdgcn_update_dpp(0u, codes, 0x4E, 0xF, 0xF, false);
            if (!value) {
                uint32_t w = 0;
#pragma unroll
                for (int e = 0; e < 8; e++) w |= (codes >> (4 * e) & 15) << (4 * (e >> 1) + 16 * (e & 1));
                ((uint32_t*)tile)[((chunk & 3) * 16 + in) * c.words + j] = w;
            } else {
                const bool high = chunk & 2;
                const uint32_t lo = high ? theirs : codes, hi = high ? codes : theirs;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int k = e + (high ? 4 : 0), n = 8 * (chunk & 1) + k;
                    tile[(((in >> 2) * 16 + n) * c.words + j) * 4 + value_byte(in & 3)] =
                        (uint8_t)((lo >> (4 * k) & 15) | (hi >> (4 * k) & 15) << 4);
                }
            }
        }
    }
}

// The values kept for each packed token, eight channels a thread: the five prompts'
// 20 us (59 MB: 2.9 TB/s, a thread's eight bytes of values one by one), the single tokens' 4 us.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadArgs a, int tokens) {
    __shared__ TokenInfo infos[kTokens];
    const int first = first_token(tokens), count = min(tokens, a.batch.T - first), wave = threadIdx.x >> 6;
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == 0) check_offsets(a.batch.offsets, a.batch.n, a.batch.T, a.err);
    if (wave < count) {
        const TokenInfo t = info_of(a.cache, a.batch, first + wave, a.err);
        if ((threadIdx.x & 63) == 0) infos[wave] = t;
    }
    __syncthreads();
    const KvView& c = a.cache;
    const int per_row = c.D / 8, keys = c.heads * per_row;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < count * 2 * keys; i += gridDim.y * kThreads) {
        const int t = i / (2 * keys), u = i - t * 2 * keys;
        const TokenInfo info = infos[t];
        const int64_t token = first + t;
        if (info.has == 0) continue;
        const bool value = u >= keys;
        const int row = value ? u - keys : u, head = row / per_row, chunk = row - head * per_row;
        const int in = info.in_page & 15, j = chunk >> 2;
        float x[8];
        if (info.has == 2) {
            const uint8_t* tile = tile_at(c, info.page, head, info.in_page) + (value ? c.tile_bytes / 2 : 0);
            const uint32_t steps = ((const uint32_t*)(tile + 256 * c.words))[(chunk >> (2 + c.group_shift)) * 16 + in];
            const float step = f16_bits_to_f32(steps & 0xFFFF), low = f16_bits_to_f32(steps >> 16);
            if (!value) {
                const uint32_t w = ((const uint32_t*)tile)[((chunk & 3) * 16 + in) * c.words + j];
#pragma unroll
                for (int e = 0; e < 8; e++) x[e] = fmaf(step, (float)(w >> (4 * (e >> 1) + 16 * (e & 1)) & 15), low);
            } else {
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int n = 8 * (chunk & 1) + e;
                    const uint32_t b = tile[(((in >> 2) * 16 + n) * c.words + j) * 4 + value_byte(in & 3)];
                    x[e] = fmaf(step, (float)(chunk & 2 ? b >> 4 : b & 15), low);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) x[e] = __uint_as_float(0x7FC00000u);
        }
        store8<BF16>(value ? a.v : a.k, token * (value ? a.ldv : a.ldk) + (int64_t)head * c.D + 8 * chunk, x);
    }
}

// Tokens a workgroup takes, and workgroups that share them: enough to fill the card
// where there are few.  8192 tokens of 32 query and 8 key heads of 128: four tokens each
// 56 us, one 70; 2048 of 8 and 2 of 64: four 17 us, one 13.
dim3 grid_of(int total, int T, int* tokens) {
    *tokens = T >= 4096 ? kTokens : 1;
    const int share = std::max(1, std::min((total + kThreads - 1) / kThreads, 1024 / T));
    const int groups = (T + *tokens - 1) / *tokens;
    return dim3(*tokens == 1 ? groups : (groups + 7) / 8 * 8, share);
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s) {
    const int total = 2 * a.cache.heads * a.cache.D / 8 + (a.q ? a.q_heads * rotate_units(a.rotary.half, a.cache.D, a.q == a.q_out) : 0);
    int tokens;
    const dim3 grid = grid_of(total, a.batch.T, &tokens);
    if (a.bf16) hipLaunchKernelGGL((kv_append_kernel<true>), grid, dim3(kThreads), 0, s, a, tokens);
    else hipLaunchKernelGGL((kv_append_kernel<false>), grid, dim3(kThreads), 0, s, a, tokens);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
    int tokens;
    const dim3 grid = grid_of(2 * a.cache.heads * a.cache.D / 8, a.batch.T, &tokens);
    if (a.bf16) hipLaunchKernelGGL((kv_read_kernel<true>), grid, dim3(kThreads), 0, s, a, tokens);
    else hipLaunchKernelGGL((kv_read_kernel<false>), grid, dim3(kThreads), 0, s, a, tokens);
    return hipGetLastError();
}

}  // namespace moe
