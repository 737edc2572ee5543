// Keys and values into a paged cache held in 4 bits, and back.  By token, head and
// group of channels, for x the value (a key after its rotation):
//   lowest = fp16(min x),  step = fp16((max x - lowest) / 15),
//   code = round((x - lowest) / step) in 0..15 (step 0: 0),  value = lowest + step * code.
#include <algorithm>

#include "rotary_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ inline double shuffle_xor(double v, int mask) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_xor((int)(uint32_t)b, mask), hi = __shfl_xor((int)(uint32_t)(b >> 32), mask);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Eight channels of a thread to codes, with the others of its group on the
// neighbouring threads (group / 8 of them, aligned).  In 64 bits throughout: which
// of two codes a value next to their border gets is then decided by the value and
// not by roundings on the way, and 64 bits cost little beside the bytes.
// Returns eight codes, four bits each; *steps the word that stands for the group.
__device__ inline uint32_t to_codes(const double (&x)[8], int group, uint32_t* steps) {
    double lo = x[0], hi = x[0];
    int fine = 1;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        lo = fmin(lo, x[i]);
        hi = fmax(hi, x[i]);
        fine &= (int)(fabs(x[i]) <= 65504.0);  // (false for a NaN)
    }
    for (int m = 1; m < group / 8; m *= 2) {
        lo = fmin(lo, shuffle_xor(lo, m));
        hi = fmax(hi, shuffle_xor(hi, m));
        fine &= __shfl_xor(fine, m);
    }
    if (!fine) {  // the whole group reads back as NaN
        *steps = 0x7E007E00u;
        return 0;
    }
    const _Float16 low16 = (_Float16)(float)lo;
    const double low = (double)low16;
    const _Float16 step16 = (_Float16)(float)((hi - low) / 15.0);
    const double step = (double)step16;
    *steps = (uint32_t)__builtin_bit_cast(uint16_t, step16) | (uint32_t)__builtin_bit_cast(uint16_t, low16) << 16;
    if (!(step > 0.0)) return 0;
    const float inverse = 1.0f / (float)step;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        // a guess that is off by one at most, then by what it leaves: halves go to the even code
        const double d = x[i] - low;
        int q = (int)rintf(fminf(fmaxf((float)d * inverse, 0.f), 15.f));
        const double left = 2.0 * fma(-(double)q, step, d);
        if (left > step || (left == step && (q & 1))) q++;
        else if (left < -step || (left == -step && (q & 1))) q--;
        codes |= (uint32_t)min(max(q, 0), 15) << (4 * i);
    }
    return codes;
}

__device__ inline uint8_t* tile_at(const KvView& c, int page, int head, int in_page) {
    return c.data + (((int64_t)page * c.heads + head) * (1 << (c.page_shift - 4)) + (in_page >> 4)) * c.tile_bytes;
}
__device__ inline int value_byte(int t) { return (t & 1) * 2 + (t >> 1 & 1); }  // place of token t % 4 in its word

// The page and the place in it; false where there is none.
__device__ inline bool find_page(const KvView& c, const KvBatchView& b, const TokenPlace& p, int* page, int* in_page) {
    if (p.bad || p.place < 0 || p.place >= (int64_t)b.max_pages << c.page_shift) return false;
    *page = b.pages[(int64_t)p.seq * b.max_pages + (p.place >> c.page_shift)];
    *in_page = (int)(p.place & ((1 << c.page_shift) - 1));
    return *page >= 0 && *page < c.pages;
}

// One token a workgroup (gridDim.y of them share few tokens' heads): its angles
// once into LDS, then eight channels a thread of keys, of values, and eight pairs
// of queries.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(KvAppendArgs a) {
    __shared__ double2 turns[128];
    __shared__ float2 turns_q[128];
    const int token = blockIdx.x;
    if (token == (int)gridDim.x - 1 && blockIdx.y == 0) check_offsets(a.batch.offsets, a.batch.n, a.batch.T, a.err);
    TokenPlace at;
    if (!find_token(a.batch, token, &at)) {
        if (at.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);
        return;
    }
    int page = 0, in_page = 0;
    const bool kept = find_page(a.cache, a.batch, at, &page, &in_page);
    if (!kept && threadIdx.x == 0) atomicOr(a.err, kErrCache);
    const RotaryView r = a.rotary;
    if (r.freqs) {
        const int position = a.positions ? a.positions[token] : (int)at.place;
        for (int i = threadIdx.x; i < r.half; i += kThreads) {
            double c, s;
            turn_of(position, r.freqs[i], &c, &s);
            c *= r.scale;
            s *= r.scale;
            turns[i] = make_double2(c, s);
            turns_q[i] = make_float2((float)c, (float)s);
        }
    }
    __syncthreads();
    const KvView& c = a.cache;
    const int per_row = c.D / 8, keys = c.heads * per_row, group = 32 << c.group_shift;
    const int units = a.q ? rotate_units(r.half, c.D, a.q == a.q_out) : 0;
    const int total = 2 * keys + a.q_heads * units;
    // (whole groups of channels lie on neighbouring threads: keys is a multiple of group / 8)
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < total; i += gridDim.y * kThreads) {
        if (i >= 2 * keys) {
            const int h = (i - 2 * keys) / units, u = (i - 2 * keys) - h * units;
            rotate_unit<BF16>(a.q, token * a.ldq + (int64_t)h * c.D, a.q_out, token * a.ldqo + (int64_t)h * c.D, c.D, r, u, turns_q);
            continue;
        }
        if (!kept) continue;
        const bool value = i >= keys;
        const int row = value ? i - keys : i, head = row / per_row, chunk = row - head * per_row, c0 = 8 * chunk;
        const void* p = value ? a.v : a.k;
        const int64_t base = token * (value ? a.ldv : a.ldk) + (int64_t)head * c.D;
        float own[8];
        load8<BF16>(p, base + c0, own);
        double x[8];
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = (double)own[e];
        if (!value && r.freqs && c0 < 2 * r.half) {
            if (r.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    if (c0 + e < 2 * r.half) {
                        const double2 t = turns[(c0 + e) / 2];
                        const double v0 = x[e], v1 = x[e + 1];
                        x[e] = v0 * t.x - v1 * t.y;
                        x[e + 1] = v0 * t.y + v1 * t.x;
                    }
            } else {
                float other[8];  // the channels' partners
                if (r.half % 8 == 0) {
                    load8<BF16>(p, base + (c0 < r.half ? c0 + r.half : c0 - r.half), other);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int ch = c0 + e;
                        other[e] = ch < 2 * r.half ? load1<BF16>(p, base + (ch < r.half ? ch + r.half : ch - r.half)) : 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int ch = c0 + e;
                    if (ch < r.half) {
                        const double2 t = turns[ch];
                        x[e] = x[e] * t.x - (double)other[e] * t.y;
                    } else if (ch < 2 * r.half) {
                        const double2 t = turns[ch - r.half];
                        x[e] = (double)other[e] * t.y + x[e] * t.x;
                    }
                }
            }
        }
        uint32_t steps;
        const uint32_t codes = to_codes(x, group, &steps);
        uint8_t* tile = tile_at(c, page, head, in_page) + (value ? c.tile_bytes / 2 : 0);
        const int in = in_page & 15, j = chunk >> 2;
        if (chunk % (group / 8) == 0) ((uint32_t*)(tile + 256 * c.words))[c0 / group * 16 + in] = steps;
        if (!value) {
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 8; e++) w |= (codes >> (4 * e) & 15) << (4 * (e >> 1) + 16 * (e & 1));
            ((uint32_t*)tile)[((chunk & 3) * 16 + in) * c.words + j] = w;
        } else {
            // channels 16 apart share a byte: the threads of each pair write half of theirs
            const uint32_t theirs = __shfl_xor((int)codes, 2);
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

// The values kept for each packed token, eight channels a thread.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadArgs a) {
    const int token = blockIdx.x;
    if (token == (int)gridDim.x - 1 && blockIdx.y == 0) check_offsets(a.batch.offsets, a.batch.n, a.batch.T, a.err);
    TokenPlace at;
    if (!find_token(a.batch, token, &at)) {
        if (at.bad && threadIdx.x == 0) atomicOr(a.err, kErrCache);
        return;
    }
    int page = 0, in_page = 0;
    const bool kept = find_page(a.cache, a.batch, at, &page, &in_page);
    if (!kept && threadIdx.x == 0) atomicOr(a.err, kErrCache);
    const KvView& c = a.cache;
    const int per_row = c.D / 8, keys = c.heads * per_row;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < 2 * keys; i += gridDim.y * kThreads) {
        const bool value = i >= keys;
        const int row = value ? i - keys : i, head = row / per_row, chunk = row - head * per_row;
        const int in = in_page & 15, j = chunk >> 2;
        float x[8];
        if (kept) {
            const uint8_t* tile = tile_at(c, page, head, in_page) + (value ? c.tile_bytes / 2 : 0);
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

// Workgroups for one token's work: enough to fill the card where there are few tokens.
int share_of(int total, int T) {
    return std::max(1, std::min((total + kThreads - 1) / kThreads, 1024 / std::max(1, T)));
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s) {
    const int total = 2 * a.cache.heads * a.cache.D / 8 + (a.q ? a.q_heads * rotate_units(a.rotary.half, a.cache.D, a.q == a.q_out) : 0);
    const dim3 grid(a.batch.T, share_of(total, a.batch.T));
    if (a.bf16) hipLaunchKernelGGL((kv_append_kernel<true>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((kv_append_kernel<false>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
    const dim3 grid(a.batch.T, share_of(2 * a.cache.heads * a.cache.D / 8, a.batch.T));
    if (a.bf16) hipLaunchKernelGGL((kv_read_kernel<true>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((kv_read_kernel<false>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
