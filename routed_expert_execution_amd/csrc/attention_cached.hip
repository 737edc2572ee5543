// Attention over a paged cache held in 4 bits: how a call is cut and launched
// (the kernels: attention_cached.h).
#include <algorithm>

#include "attention_cached.h"

namespace moe {

hipError_t launch_cached_f32(const CachedArgs& a, const CachedPlan& p, hipStream_t s);

// Runs: as many as the card's 256 CUs take at a time.
CachedPlan cached_plan(const KvGeom& g, int n, int64_t tokens, int most_new, int max_pages, int q_heads, int bf16) {
    CachedPlan p{};
    const int per_head = q_heads / g.heads, round = cached::kStep * cached::kWaves;
    // what the call can have at most: row tiles, rounds of one, runs
    const int64_t rounds = ((int64_t)max_pages * g.page_tokens + round - 1) / round;
    p.tiles = tokens * per_head / 16 + n;
    p.line = p.tiles * rounds;
    p.places = (int)std::max<int64_t>(1, std::min<int64_t>(256 * cached_per_cu(g.D / 32, bf16) / g.heads, p.line));
    p.split = rounds > 1 && p.places > 1;
    p.part_rows = std::min<int64_t>(16, (int64_t)most_new * per_head);
    p.bytes = p.split ? (size_t)2 * p.places * g.heads * p.part_rows * (g.D + 2) * sizeof(float) : 0;
    return p;
}

hipError_t launch_cached(const CachedArgs& a, const CachedPlan& p, hipStream_t s) {
    return a.bf16 ? cached::launch_by_width<true>(a, p, s) : launch_cached_f32(a, p, s);
}

}  // namespace moe
