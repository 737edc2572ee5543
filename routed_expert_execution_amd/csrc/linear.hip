// 4-bit matrices with group scales: packing into the tiles of dense.h, the
// values back in fp32, and the choice of the product kernel.
#include "dense.h"
#include "device_util.h"
#include "linear_rows.h"

namespace moe {
namespace {

// A thread makes one word of a tile (8 codes of a row), the first threads of a
// tile its scales and zero points too.  Once per matrix, bound by its bytes.
__global__ __launch_bounds__(256) void pack_kernel(QuantGeom g, const uint8_t* __restrict__ codes,
                                                   const uint16_t* __restrict__ scales, const uint8_t* __restrict__ zeros,
                                                   uint8_t* __restrict__ data) {
    const int lane = threadIdx.x >> 2, j = threadIdx.x & 3, S = g.per_tile;
    for (int64_t tile = blockIdx.x; tile < g.row_groups * g.col_tiles; tile += gridDim.x) {
        const int64_t rg = tile / g.col_tiles, kt = tile % g.col_tiles;
        const int64_t row = rg * 16 + (lane & 15), col = kt * 128 + 32 * j + 8 * (lane >> 4);
        uint32_t word = 0;
        if (row < g.rows && col < g.cols) {  // (columns come in whole 32s)
            const uint8_t* src = codes + row * (g.cols / 2) + col / 2;
            for (int p = 0; p < 4; p++) word |= (uint32_t)(src[p] & 15) << (4 * p) | (uint32_t)(src[p] >> 4) << (16 + 4 * p);
        }
        ((uint32_t*)data)[tile * 256 + lane * 4 + j] = word;
        if ((int)threadIdx.x < 16 * S) {
            const int64_t r = rg * 16 + threadIdx.x / S, c = kt * S + threadIdx.x % S, per_row = g.cols / g.group;
            const bool in = r < g.rows && c < per_row;
            ((uint16_t*)(data + g.scales_at))[tile * 16 * S + threadIdx.x] = in ? scales[r * per_row + c] : 0;
            if (g.affine) (data + g.zeros_at)[tile * 16 * S + threadIdx.x] = in ? zeros[r * per_row + c] : 0;
        }
    }
}

// fp32 value s (q - z) of every element, row-major: exact, as 11 bits of scale
// times at most 8 of code fit in 24.
__global__ __launch_bounds__(256) void dequant_kernel(QuantGeom g, const uint8_t* __restrict__ data, float* __restrict__ out) {
    const int64_t words = g.cols / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < g.rows * words; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / words, col = i % words * 8;
        const int64_t tile = row / 16 * g.col_tiles + col / 128;
        const int lane = (int)(row % 16) + 16 * (int)(col % 32 / 8), j = (int)(col % 128 / 32);
        const uint32_t word = ((const uint32_t*)data)[tile * 256 + lane * 4 + j];
        const int64_t at = (tile * 16 + row % 16) * g.per_tile + col % 128 / g.group;
        const float s = f16_bits_to_f32(((const uint16_t*)(data + g.scales_at))[at]);
        const float z = g.affine ? (float)(data + g.zeros_at)[at] : 8.f;
        for (int e = 0; e < 8; e++) {
            const uint32_t q = word >> (e % 2 * 16 + e / 2 * 4) & 15;
            out[row * g.cols + col + e] = s * ((float)q - z);
        }
    }
}

// workgroups of a pass that goes round (2^32 threads are the most of a launch)
dim3 workgroups(int64_t n) { return dim3((unsigned)(n < (1 << 20) ? n : 1 << 20)); }

}  // namespace

hipError_t launch_linear_pack(const QuantGeom& g, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                              void* data, hipStream_t s) {
    hipLaunchKernelGGL(pack_kernel, workgroups(g.row_groups * g.col_tiles), dim3(256), 0, s, g, codes, scales, zeros, (uint8_t*)data);
    return hipGetLastError();
}

hipError_t launch_linear_dequant(const QuantGeom& g, const void* data, float* out, hipStream_t s) {
    const int64_t words = g.rows * (g.cols / 8);
    hipLaunchKernelGGL(dequant_kernel, workgroups((words + 255) / 256), dim3(256), 0, s, g, (const uint8_t*)data, out);
    return hipGetLastError();
}

// Tiles or shared rows for many bf16 tokens, by estimated time.  A workgroup of
// the shared rows (64 tokens, 4 row groups) takes 0.9 us for two column tiles
// where few are at work and 1.5 where one is on every CU, gated 1.5 and 3.1, and
// more workgroups as much longer; the tiles need 1.5 us more around their steps.
// Measured, us, rows against tiles (4-bit matrices of groups of 64 unless said):
// 384 tokens, 4096 x 512, groups of 128 8.2 / 11.9; 128 tokens, 8192 x 1024 9.5 /
// 9.9; 106 tokens, gated 3360 x 2208, groups of 32 19.2 / 18.4; 128 tokens, gated
// 8192 x 2048 22 / 27, 256 tokens 44 / 37; 512 tokens, 4096 x 4096, groups of 32 50
// / 58; 2048 tokens, 4096 x 4096 190 / 84.
DensePlan linear_plan(const LinearArgs& a, bool gated) {
    if (a.T > 64 && a.x_bf16 && a.y_bf16) {
        const float on_cu = (float)((a.row_groups + 3) / 4) * (float)((a.T + 63) / 64) / 256.f;
        const float few = gated ? 1.5f : 0.9f, full = gated ? 3.1f : 1.5f;
        const float rows_us = (float)((a.col_tiles + 1) / 2) * (on_cu < 1.f ? few + (full - few) * on_cu : full * on_cu);
        float tiles_us;
        const DensePlan tiles = linear_tiles_plan(a, gated, &tiles_us);
        if (tiles_us + 1.5f < rows_us) return tiles;
    }
    return linear::rows_plan(a);
}

hipError_t launch_linear(const LinearArgs& a, bool gated, hipStream_t s) {
    const DensePlan p = linear_plan(a, gated);
    if (p.kind == MOE_PLAN_TILES) return launch_linear_tiles(a, gated, p.shape, s);
    return a.x_bf16 ? launch_linear_rows_bf16(a, gated, p, s) : launch_linear_rows_f32(a, gated, p, s);
}

}  // namespace moe
