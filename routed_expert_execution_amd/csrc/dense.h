// Declarations of the dense operators (moe_linear*, moe_gated*): the packed
// 4-bit matrix, argument blocks and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// Geometry of a packed 4-bit matrix [rows, cols] with one scale (and, affine,
// one zero point) per `group` columns of a row.  Tiles of 16 rows x 128 columns,
// by row group, then column group, so that 16 consecutive rows are one run:
//   codes   1024 B a tile: lane l of a wave owns the 16 bytes at 16 l, word j of
//           them its B operand of the j-th 16x16x32 product of the tile, the
//           codes of row l % 16, columns 32 j + 8 (l / 16) + 0..7: column 2p in
//           bits 4p..4p+3, column 2p + 1 in bits 16+4p..16+4p+3
//   scales  [16 rows][128 / group] fp16 a tile, after all codes
//   zeros   [16 rows][128 / group] bytes a tile, after all scales (affine only)
// Rows past the last and columns past the last are stored as code 0, scale 0.
struct QuantGeom {
    int64_t rows = 0, cols = 0;
    int group = 0, affine = 0;
    int64_t row_groups = 0, col_tiles = 0;  // ceil(rows / 16), ceil(cols / 128)
    int per_tile = 0;                       // scales a row has in one tile: 128 / group
    int64_t scales_at = 0, zeros_at = 0, bytes = 0;

    bool init(int64_t rows_, int64_t cols_, int group_, int affine_) {
        rows = rows_; cols = cols_; group = group_; affine = affine_;
        if (group != 32 && group != 64 && group != 128) return false;
        if (affine != 0 && affine != 1) return false;
        if (rows < 1 || cols < 1 || rows > (1 << 24) || cols > (1 << 24) || cols % group) return false;
        row_groups = (rows + 15) / 16;
        col_tiles = (cols + 127) / 128;
        per_tile = 128 / group;
        const int64_t tiles = row_groups * col_tiles;
        scales_at = tiles * 1024;
        zeros_at = scales_at + tiles * 32 * per_tile;
        bytes = zeros_at + (affine ? tiles * 16 * per_tile : 0);
        return true;
    }
};

struct QuantView {  // a packed matrix as the kernels address it
    const uint4* codes;
    const uint16_t* scales;
    const uint8_t* zeros;  // null: every zero point is 8
};
inline QuantView quant_view(const QuantGeom& g, const void* data) {
    const uint8_t* p = (const uint8_t*)data;
    return {(const uint4*)p, (const uint16_t*)(p + g.scales_at), g.affine ? p + g.zeros_at : nullptr};
}

hipError_t launch_linear_pack(const QuantGeom& g, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                              void* data, hipStream_t s);
hipError_t launch_linear_dequant(const QuantGeom& g, const void* data, float* out, hipStream_t s);

// The kernel of a call, chosen by sizes and types alone.
struct DensePlan {
    int kind;          // MOE_PLAN_*
    int tokens, rows;  // of a workgroup; rows of each matrix (backward: the tile of both products)
    int parts;         // of the columns (k), summed inside a workgroup
    int dx_parts, dw_parts;  // backward: of k over workgroups
    int shape;         // tiles: row of the table of shapes
};

struct LinearArgs {
    QuantView w[2];  // the matrix; or gate and up
    int rows, cols;  // of each
    int row_groups, col_tiles;
    int group;
    const void* x;   // [T, cols], rows ldx elements apart
    int64_t ldx;
    int x_bf16;
    int64_t T;
    void* y;         // [T, rows], rows ldy elements apart
    int64_t ldy;
    int y_bf16;
};
DensePlan linear_plan(const LinearArgs& a, bool gated);
hipError_t launch_linear(const LinearArgs& a, bool gated, hipStream_t s);
// Many tokens, x and y bf16: on tiles; and the time that is estimated to take.
hipError_t launch_linear_tiles(const LinearArgs& a, bool gated, int shape, hipStream_t s);
DensePlan linear_tiles_plan(const LinearArgs& a, bool gated, float* us);

struct GatedArgs {
    const void* x;  // [T, d], rows ldx elements apart
    int64_t ldx;
    int64_t T;
    int d, F;
    int bf16;       // element type of everything here: bf16 or fp32
    const void *w_gate, *w_up;  // [F, d]
    void* h;                    // [T, F]
    void *gate, *up;            // [T, F] or null
};
DensePlan gated_plan(int64_t T, int d, int F, int bf16);
hipError_t launch_gated(const GatedArgs& a, hipStream_t s);

struct GatedBackwardArgs {
    const void* dh;  // [T, F], rows lddh elements apart
    int64_t lddh;
    const void* x;   // [T, d], rows ldx elements apart
    int64_t ldx;
    int64_t T;
    int d, F;
    int bf16;
    const void *w_gate, *w_up;  // [F, d]
    const void *gate, *up;      // [T, F]
    void* dx;                   // [T, d] or null
    void *dw_gate, *dw_up;      // [F, d] or null
    void* workspace;
};
DensePlan gated_backward_plan(int64_t T, int d, int F, int bf16);
size_t gated_backward_bytes(int64_t T, int d, int F, int bf16);
hipError_t launch_gated_backward(const GatedBackwardArgs& a, hipStream_t s);

}  // namespace moe
