// Device helpers shared by the attention layer's kernels.
#pragma once

#include "attention.h"
#include "device_util.h"
#include "internal.h"

namespace moe {

struct __attribute__((packed, aligned(2))) Words4 { uint32_t v[4]; };

template <bool BF16> __device__ inline float load1(const void* p, int64_t i) {
    if (BF16) return bf16_bits_to_f32(((const uint16_t*)p)[i]);
    return ((const float*)p)[i];
}
template <bool BF16> __device__ inline void store1(void* p, int64_t i, float v) {
    if (BF16) ((__bf16*)p)[i] = (__bf16)v;
    else ((float*)p)[i] = v;
}
// Eight elements from index i on (16 or 32 bytes, aligned as elements are), as they lie
// in memory and as values.
template <bool BF16> struct Raw8 {
    Words4 w[BF16 ? 1 : 2];
    __device__ void load(const void* p, int64_t i) {
        w[0] = *(const Words4*)((const char*)p + i * (BF16 ? 2 : 4));
        if constexpr (!BF16) w[1] = *(const Words4*)((const float*)p + i + 4);
    }
    __device__ void get(float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; e++) {
            if constexpr (BF16) {
                v[2 * e] = __uint_as_float(w[0].v[e] << 16);
                v[2 * e + 1] = __uint_as_float(w[0].v[e] & 0xFFFF0000u);
            } else {
                v[e] = __uint_as_float(w[0].v[e]);
                v[4 + e] = __uint_as_float(w[1].v[e]);
            }
        }
    }
};
template <bool BF16> __device__ inline void load8(const void* p, int64_t i, float (&v)[8]) {
    Raw8<BF16> r;
    r.load(p, i);
    r.get(v);
}
template <bool BF16> __device__ inline void store8(void* p, int64_t i, const float (&v)[8]) {
    if (BF16) {
        Words4 w;
        __bf16 b[8];
#pragma unroll
        for (int e = 0; e < 8; e++) b[e] = (__bf16)v[e];
        __builtin_memcpy(&w, b, 16);
        *(Words4*)((uint16_t*)p + i) = w;
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            Words4 w;
#pragma unroll
            for (int e = 0; e < 4; e++) w.v[e] = __float_as_uint(v[4 * h + e]);
            *(Words4*)((float*)p + i + 4 * h) = w;
        }
    }
}

// Largest i in [0, n) with key(i) <= at, for keys that do not descend and
// key(0) <= at; whole wave, every lane gets it.  64 keys a step, so one load up to
// 64 of them.  Whatever the keys are, the result is in [0, n).
template <typename Key>
__device__ inline int wave_find(int n, int64_t at, Key key) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const int i = lo + lane * step;
        const uint64_t below = __ballot(i < hi && key(i) <= at);
        const int k = 63 - __clzll(below | 1);
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Sets the error word if any of the n sequences' offsets cannot be: by one workgroup
// of a launch, for the sequences that no other workgroup meets.
__device__ inline void check_offsets(const int32_t* offsets, int n, int T, int* err) {
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= offsets[i] < 0 || offsets[i + 1] < offsets[i] || offsets[i + 1] > T;
    if (bad) atomicOr(err, kErrCache);
}

// The sequence and the place of packed token `token`; false where no sequence has
// it, with `bad` where offsets or the length cannot be.
struct TokenPlace { int seq; int64_t place; bool bad; };
__device__ inline bool find_token(const KvBatchView& b, int token, TokenPlace* p) {
    const int s = wave_find(b.n, token, [&](int i) { return (int64_t)b.offsets[i]; });
    const int64_t begin = b.offsets[s], end = b.offsets[s + 1], length = b.lengths[s];
    p->seq = s;
    p->place = length - (end - token);
    p->bad = begin < 0 || end < begin || end > b.T;
    if (token < begin || token >= end) return false;
    p->bad |= length < end - begin;
    return true;
}

// Cosine and sine of position * frequency: the product in 64 bits, since 24 bits
// of a far position's angle leave little of it, then its part of a turn (position
// 2^31 at one radian a position: 2e-7 off).
__device__ inline void turn_of(int position, float freq, double* c, double* s) {
    const double turns = (double)position * (double)freq * 0.15915494309189535;
    sincospi(2.0 * (turns - rint(turns)), s, c);
}

}  // namespace moe
