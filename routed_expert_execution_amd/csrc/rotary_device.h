// Rotation of a row's channels by position, as moe_rotate and moe_kv_append do it.
#pragma once

#include "attention_device.h"

namespace moe {

// A head's work in units: eight pairs of channels, or eight channels that are only
// copied (none of them in place).  Pairs are read and written by one thread, so a
// row may be rotated in place.
__device__ __host__ inline int rotate_pair_units(int half) { return (half + 7) / 8; }
__device__ __host__ inline int rotate_units(int half, int D, bool in_place) {
    return rotate_pair_units(half) + (in_place ? 0 : (D - 2 * half + 7) / 8);
}

// Unit u of the heads of up to N tokens: load() of each, then finish(), so that all
// are read before the first is waited for.  turns[pair] = (cos, sin), times the scale.
template <bool BF16, int N = 4>
struct RotateUnit {
    const RotaryView& r;
    int a0, b0, n;  // the places of the unit's first and second eight channels; pairs, or -1 where it copies
    bool whole;     // all eight of them, or eight channels
    int D;
    Raw8<BF16> a[N], b[N];

    __device__ RotateUnit(const RotaryView& rotary, int head_dim, int u) : r(rotary), D(head_dim) {
        const int pairs = rotate_pair_units(r.half), p0 = 8 * u;
        if (u >= pairs) {
            n = -1;
            a0 = 2 * r.half + 8 * (u - pairs);
            b0 = 0;
            whole = a0 + 8 <= D;
        } else {
            n = min(8, r.half - p0);
            a0 = r.interleaved ? 2 * p0 : p0;
            b0 = r.interleaved ? 2 * p0 + 8 : p0 + r.half;
            whole = n == 8;
        }
    }
    __device__ void load(int t, const void* x, int64_t xi) {
        if (!whole) return;
        a[t].load(x, xi + a0);
        if (n > 0) b[t].load(x, xi + b0);
    }
    __device__ void finish(int t, const void* x, int64_t xi, void* y, int64_t yi, const float2* turns) const {
        const int p0 = r.interleaved ? a0 / 2 : a0;
        if (!whole) {
            if (n < 0)
                for (int i = a0; i < D; i++) store1<BF16>(y, yi + i, load1<BF16>(x, xi + i));
            for (int i = 0; i < n; i++) {
                const int e = r.interleaved ? 2 * (p0 + i) : p0 + i, f = r.interleaved ? e + 1 : e + r.half;
                const float2 w = turns[p0 + i];
                const float va = load1<BF16>(x, xi + e), vb = load1<BF16>(x, xi + f);
                store1<BF16>(y, yi + e, fmaf(va, w.x, -(vb * w.y)));
                store1<BF16>(y, yi + f, fmaf(va, w.y, vb * w.x));
            }
            return;
        }
        float va[8], vb[8], c[8], d[8];
        a[t].get(va);
        if (n < 0) {
            store8<BF16>(y, yi + a0, va);
            return;
        }
        b[t].get(vb);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 w = turns[p0 + i];
            if (r.interleaved) {
                float* in = i < 4 ? va : vb;
                float* out = i < 4 ? c : d;
                const int e = 2 * (i & 3);
                out[e] = fmaf(in[e], w.x, -(in[e + 1] * w.y));
                out[e + 1] = fmaf(in[e], w.y, in[e + 1] * w.x);
            } else {
                c[i] = fmaf(va[i], w.x, -(vb[i] * w.y));
                d[i] = fmaf(va[i], w.y, vb[i] * w.x);
            }
        }
        store8<BF16>(y, yi + a0, c);
        store8<BF16>(y, yi + b0, d);
    }
};

}  // namespace moe
