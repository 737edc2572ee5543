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

// Unit u of the head at x: turns[pair] = (cos, sin), times the scale.
template <bool BF16>
__device__ inline void rotate_unit(const void* x, int64_t xi, void* y, int64_t yi, int D, const RotaryView& r, int u,
                                   const float2* turns) {
    const int pairs = rotate_pair_units(r.half);
    if (u >= pairs) {
        const int c = 2 * r.half + 8 * (u - pairs);
        float v[8];
        if (c + 8 <= D) {
            load8<BF16>(x, xi + c, v);
            store8<BF16>(y, yi + c, v);
        } else {
            for (int i = c; i < D; i++) store1<BF16>(y, yi + i, load1<BF16>(x, xi + i));
        }
        return;
    }
    const int p0 = 8 * u, n = min(8, r.half - p0);
    // the places of the unit's first and second eight channels, and which of the 16 a pair takes
    const int a0 = r.interleaved ? 2 * p0 : p0, b0 = r.interleaved ? 2 * p0 + 8 : p0 + r.half;
    if (n == 8) {
        float a[8], b[8], c[8], d[8];
        load8<BF16>(x, xi + a0, a);
        load8<BF16>(x, xi + b0, b);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 t = turns[p0 + i];
            if (r.interleaved) {
                float* in = i < 4 ? a : b;
                float* out = i < 4 ? c : d;
                const int e = 2 * (i & 3);
                out[e] = fmaf(in[e], t.x, -(in[e + 1] * t.y));
                out[e + 1] = fmaf(in[e], t.y, in[e + 1] * t.x);
            } else {
                c[i] = fmaf(a[i], t.x, -(b[i] * t.y));
                d[i] = fmaf(a[i], t.y, b[i] * t.x);
            }
        }
        store8<BF16>(y, yi + a0, c);
        store8<BF16>(y, yi + b0, d);
        return;
    }
    for (int i = 0; i < n; i++) {
        const int e = r.interleaved ? 2 * (p0 + i) : p0 + i, f = r.interleaved ? e + 1 : e + r.half;
        const float2 t = turns[p0 + i];
        const float va = load1<BF16>(x, xi + e), vb = load1<BF16>(x, xi + f);
        store1<BF16>(y, yi + e, fmaf(va, t.x, -(vb * t.y)));
        store1<BF16>(y, yi + f, fmaf(va, t.y, vb * t.x));
    }
}

}  // namespace moe
