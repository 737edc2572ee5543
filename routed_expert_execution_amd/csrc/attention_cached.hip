// Attention over a paged cache held in 4 bits: how a call is cut and launched
// (the kernels: attention_cached.h).
#include <algorithm>

#include "attention_cached.h"

namespace moe {

hipError_t launch_cached_f32(const CachedArgs& a, int split, hipStream_t s);

// Few rows leave most of the card idle unless a sequence's tokens are cut: into so
// many chunks that there are about 768 workgroups, three for each CU, or a few times
// that.
CachedPlan cached_plan(const KvGeom& g, int n, int most_new, int max_pages, int q_heads, int bf16) {
    CachedPlan p{};
    p.tile_rows = 16;
    const int64_t tiles = std::max<int64_t>(1, ((int64_t)most_new * (q_heads / g.heads) + p.tile_rows - 1) / p.tile_rows);
    // steps of a round of a workgroup's waves that the sequences can have at most
    const int64_t longest = (int64_t)max_pages * g.page_tokens, round = cached::kStep * cached::kWaves, most = (int64_t)n * ((longest + round - 1) / round);
    p.places = (int)std::max<int64_t>(1, 768 / (g.heads * tiles));
    p.rounds = 4;
    p.target = (int)std::max<int64_t>(1, std::min<int64_t>(p.places * p.rounds, most));
    p.split = p.target > n || (p.target > 1 && longest > round);
    if (!p.split) p.places = p.rounds = p.target = 1;
    // (workgroups of a sequence past its own rows end at once; not too many of them)
    p.row_tiles = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, std::max<int64_t>(8192 / ((int64_t)g.heads * (n + p.target)), 256 / g.heads)));
    p.bytes = p.split ? (size_t)2 * p.target * most_new * q_heads * (g.D + 2) * sizeof(float) : 0;
    return p;
}

hipError_t launch_cached(const CachedArgs& a, int split, hipStream_t s) {
    return a.bf16 ? cached::launch_by_width<true>(a, split, s) : launch_cached_f32(a, split, s);
}

}  // namespace moe
