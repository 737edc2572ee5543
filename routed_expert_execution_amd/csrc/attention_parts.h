// Attention over packed sequences in small tiles: what the kernels share whose waves
// divide the others' axis.
#pragma once

#include "attention_tiles.h"

namespace moe {
namespace packed {

constexpr int kPartsWaves = 4, kPartsThreads = 64 * kPartsWaves;

// A workgroup has 32 BLOCKS rows (or, of the backward pass, keys) of its own and passes over
// the others 32 PARTS at a time, BLOCKS PARTS = 4 waves, each with sums of its own that are
// joined in order at the end: small tiles, for few and short sequences and for the products
// of fp32, six of bf16 terms each, which leave the time to load more.
template <bool BF16, int D> struct PartsShape {
    static constexpr int kParts = BF16 || D <= 128 ? 4 : 2, kBlocks = kPartsWaves / kParts;
    static constexpr int kOwn = 32 * kBlocks, kOther = 32 * kParts;
    static constexpr int kTileBytes = kOther * Tile<BF16, D>::kLineBytes;  // 64 KiB at most
};

// Sums of several waves: those of parts 1.. through LDS to part 0's, which adds them in
// order.  N blocks of 16 registers; true for the waves that hold the result.
template <int N, int PARTS, int BLOCKS>
__device__ inline bool add_parts(f32x16 (&acc)[N], char* lds, int part, int block, int lane) {
    f32x4* at = (f32x4*)lds;
#pragma unroll 1
    for (int p = 1; p < PARTS; p++) {
        __syncthreads();
        if (part == p)
#pragma unroll
            for (int n = 0; n < N; n++)
#pragma unroll
                for (int j = 0; j < 4; j++) at[((block * N + n) * 4 + j) * 64 + lane] = f32x4{acc[n][4 * j], acc[n][4 * j + 1], acc[n][4 * j + 2], acc[n][4 * j + 3]};
        __syncthreads();
        if (part == 0)
#pragma unroll
            for (int n = 0; n < N; n++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const f32x4 v = at[((block * N + n) * 4 + j) * 64 + lane];
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[n][4 * j + e] += v[e];
                }
    }
    return part == 0;
}

// A tile into LDS, through registers a few chunks at a time or straight.
template <bool BF16, int D, int R, bool DIRECT>
__device__ inline void bring(const char* base, int64_t ld, int64_t first, int lines, char* lds) {
    typedef Tile<BF16, D> T;
    if constexpr (DIRECT) {
        Pipe<BF16, D, R, kPartsThreads, true> p;
        p.fetch(base, ld, first, lines, lds);
    } else {
#pragma unroll 4
        for (int n = threadIdx.x; n < R * T::kChunks; n += kPartsThreads) {
            const int r = n / T::kChunks, c = n - r * T::kChunks;
            u32x4 v = {0, 0, 0, 0};
            if (r < lines) {
                const Words4 w = *(const Words4*)(base + ((first + r) * ld + c * T::kPer) * (BF16 ? 2 : 4));
                v = u32x4{w.v[0], w.v[1], w.v[2], w.v[3]};
            }
            *(u32x4*)(lds + T::at(r, c)) = v;
        }
    }
}

// N products with an operand each from LDS, the second next one's read and the next one's
// terms made beside a product.
template <int N, bool BF16, typename Read, typename Use>
__device__ inline void in_turn(Read read, Use use) {
    Fragment<BF16> f[3];
    read(0, f[0]);
    if (N > 1) read(1, f[1]);
    f[0].split();
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (i + 2 < N) read(i + 2, f[(i + 2) % 3]);
        if (i + 1 < N) f[(i + 1) % 3].split();
        use(i, f[i % 3]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

}  // namespace packed
}  // namespace moe
