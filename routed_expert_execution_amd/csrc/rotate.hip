// Rotary positions: each pair (x1, x2) of a token's channels turned by the angle
// position * frequency of the pair,
//   y1 = x1 c - x2 s,  y2 = x1 s + x2 c,  c = scale cos, s = scale sin
// (the inverse, and the gradient, with -s).
#include <algorithm>

#include "rotary_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kMaxTokens = 16;

// Bound by bytes.  A workgroup takes a few tokens and turns each one's angles into
// cosines and sines once, in LDS, for all heads; then eight pairs a thread, 16 bytes
// a load.  Few tokens of many heads are shared out over gridDim.y workgroups.  8192
// tokens of 32 heads of 128 in bf16, 32 pairs of each turned: 38 us, 3.5 TB/s (31 where the
// last-level cache still holds half of it); one token 3 us.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void rotate_kernel(RotateArgs a, int per_group) {
    extern __shared__ float2 turns[];  // [per_group][half]
    const RotaryView r = a.rotary;
    const int64_t t0 = (int64_t)blockIdx.x * per_group;
    const int tokens = (int)min((int64_t)per_group, a.T - t0);
    for (int i = threadIdx.x; i < tokens * r.half; i += kThreads) {
        double c, s;
        turn_of(a.positions[t0 + i / r.half], r.freqs[i % r.half], &c, &s);
        turns[i] = make_float2((float)(c * r.scale), (float)((a.inverse ? -s : s) * r.scale));
    }
    __syncthreads();
    const int units = rotate_units(r.half, a.D, a.x == a.y), total = tokens * a.heads * units;
    for (int i = blockIdx.y * kThreads + threadIdx.x; i < total; i += gridDim.y * kThreads) {
        const int head = i / units, t = head / a.heads, h = head - t * a.heads;
        const int64_t xi = (t0 + t) * a.ldx + (int64_t)h * a.D, yi = (t0 + t) * a.ldy + (int64_t)h * a.D;
        RotateUnit<BF16, 1> unit(r, a.D, i - head * units);
        unit.load(0, a.x, xi);
        unit.finish(0, a.x, xi, a.y, yi, turns + t * r.half);
    }
}

}  // namespace

hipError_t launch_rotate(const RotateArgs& a, hipStream_t s) {
    const int units = a.heads * rotate_units(a.rotary.half, a.D, a.x == a.y);
    const int per_group = std::max(1, std::min(kMaxTokens, kThreads / units));
    const int64_t groups = (a.T + per_group - 1) / per_group;
    const int share = (int)std::max<int64_t>(1, std::min<int64_t>((units + kThreads - 1) / kThreads, 512 / groups));
    const dim3 grid((unsigned)groups, share);
    const size_t lds = (size_t)per_group * a.rotary.half * sizeof(float2);
    if (a.bf16) hipLaunchKernelGGL((rotate_kernel<true>), grid, dim3(kThreads), lds, s, a, per_group);
    else hipLaunchKernelGGL((rotate_kernel<false>), grid, dim3(kThreads), lds, s, a, per_group);
    return hipGetLastError();
}

}  // namespace moe
