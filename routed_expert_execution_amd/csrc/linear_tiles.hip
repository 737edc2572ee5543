// Many tokens against 4-bit weights: bf16 in, bf16 out, tiles on the matrix cores.
#include "tile_kernel.h"

namespace moe {

namespace {
int plan(const LinearArgs& a, bool gated, float* us = nullptr) {
    return tile::plan_tiles(tile::kQuant4, a.T, (int64_t)a.rows * (gated ? 2 : 1), (a.cols + 63) / 64, us);
}
}  // namespace

float linear_tiles_us(const LinearArgs& a, bool gated) {
    float us;
    plan(a, gated, &us);
    return us;
}

// Each weight s (q - z) is rounded to bf16 here, once, because scaling the sums
// of exact codes group by group, as the row products do, costs the vector unit
// more than the matrix cores take for a large tile (two fp32 operations an
// element and group, in registers a 256 x 256 tile does not have).  The rounding
// is independent from weight to weight; it adds to the result's norm-wise error
// about what the rounding of the result itself does (0.17 % to 0.24 %; gated,
// where two sums meet, 0.29 %).
hipError_t launch_linear_tiles(const LinearArgs& a, bool gated, hipStream_t s) {
    using namespace tile;
    TileArgs t{};
    t.a = Operand{{a.x, nullptr}, a.ldx, 0};
    t.M = a.T;
    t.N = a.rows;
    t.K = a.cols;
    t.out[0] = a.y;
    t.ldo = a.ldy;
    t.q[0] = a.w[0];
    t.q[1] = a.w[1];
    t.per_tile = 128 / a.group;
    t.row_groups = a.row_groups;
    t.col_tiles = a.col_tiles;
    const int shape = plan(a, gated);
    return gated ? launch_tiles<true, kAlongK, kQuantised, kGatedForward>(t, shape, s)
                 : launch_tiles<true, kAlongK, kQuantised, kOneResult>(t, shape, s);
}

}  // namespace moe
