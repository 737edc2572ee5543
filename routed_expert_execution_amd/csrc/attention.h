// Declarations of the attention layer's operators (moe_rotate, moe_kv_*,
// moe_attention*): the paged 4-bit cache, argument blocks and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

inline bool head_dim_valid(int D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

// A cache of pages of `page_tokens` tokens, each with `heads` key and value heads
// of D channels in 4 bits.  A page holds, head after head, page_tokens / 16 tiles
// of 16 tokens; a tile is what the products of one wave load, in this order:
//   key codes    [64 lanes][D / 32] words: lane l's word j is its operand of the
//                product over channels 32 j..32 j + 31: the codes of token l % 16,
//                channels 32 j + 8 (l / 16) + 0..7, the channel 2 p of them in bits
//                4 p..4 p + 3, the channel 2 p + 1 in bits 16 + 4 p..19 + 4 p
//   key steps    [D / group][16 tokens] words: step (fp16) in the low half, lowest
//                value (fp16) in the high half
//   value codes  [64 lanes][D / 32] words: lane l's word j holds tokens
//                4 (l / 16) + 0..3 in bytes 0, 2, 1, 3, of each the channel
//                32 j + l % 16 in the low four bits, 16 channels on in the high ones
//   value steps  as the keys'
// A value is lowest + step * code.
struct KvGeom {
    int64_t pages = 0;
    int page_tokens = 0, heads = 0, D = 0, group = 0;
    int words = 0, groups = 0, tiles = 0;  // D / 32, D / group, page_tokens / 16
    int64_t tile_bytes = 0, bytes = 0;

    bool init(int64_t pages_, int page_tokens_, int heads_, int D_, int group_) {
        pages = pages_; page_tokens = page_tokens_; heads = heads_; D = D_; group = group_;
        if (pages < 1 || pages > INT32_MAX || heads < 1 || heads > 1024 || !head_dim_valid(D)) return false;
        if (page_tokens < 16 || page_tokens > 1024 || (page_tokens & (page_tokens - 1))) return false;
        if ((group != 32 && group != 64 && group != 128) || D % group) return false;
        words = D / 32;
        groups = D / group;
        tiles = page_tokens / 16;
        tile_bytes = 2 * (256 * words + 64 * groups);
        if (pages > ((int64_t)1 << 46) / (heads * tiles * tile_bytes)) return false;
        bytes = pages * heads * tiles * tile_bytes;
        return true;
    }
};

struct KvView {  // a cache as the kernels address it
    uint8_t* data;
    int64_t pages, tile_bytes;
    int page_shift, heads, D, words, groups, group_shift;  // log2 of page_tokens, of group / 32
};
inline KvView kv_view(const KvGeom& g, void* data) {
    auto log2 = [](int v) { int s = 0; while ((1 << s) < v) s++; return s; };
    return {(uint8_t*)data, g.pages, g.tile_bytes, log2(g.page_tokens), g.heads, g.D, g.words, g.groups, log2(g.group / 32)};
}

// Sequences of a call: the new tokens packed, the pages of each one's tokens.
struct KvBatchView {
    const int32_t* offsets;  // [n + 1]
    const int32_t* lengths;  // [n] tokens held once the new ones are
    const int32_t* pages;    // [n][max_pages]
    int n, max_pages;
    int T;                   // rows of the packed tensors
    int most_new;            // no sequence has more new tokens
};

struct RotaryView {
    const float* freqs;  // [half], null: nothing is rotated
    int half, interleaved;
    float scale;
};

struct RotateArgs {
    const void* x;
    int64_t ldx;
    void* y;
    int64_t ldy;
    int bf16;
    int64_t T;
    int heads, D;
    const int32_t* positions;
    RotaryView rotary;
    int inverse;
};
hipError_t launch_rotate(const RotateArgs& a, hipStream_t s);

struct KvAppendArgs {
    KvView cache;
    KvBatchView batch;
    const void *k, *v;
    int64_t ldk, ldv;
    int bf16;
    RotaryView rotary;
    const int32_t* positions;  // [T] or null: the tokens' places in their sequences
    const void* q;             // or null
    int64_t ldq;
    int q_heads;
    void* q_out;
    int64_t ldqo;
    int* err;
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s);

struct KvReadArgs {
    KvView cache;
    KvBatchView batch;
    void *k, *v;
    int64_t ldk, ldv;
    int bf16;
    int* err;
};
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s);

// Attention over a cache.
struct CachedArgs {
    KvView cache;
    KvBatchView batch;
    const void* q;
    int64_t ldq;
    int bf16, per_head;           // per_head: query heads of one key head
    float scale_log2;             // scale / ln 2: the exponentials are powers of two
    int window;                   // 0: none
    void* out;
    int64_t ldo;
    int places, part_rows;        // runs that the call's work is cut into; rows kept of a part of a row tile
    float* part;                  // [2 places][cache.heads][part_rows][D]
    float2* part_ml;              // [2 places][cache.heads][part_rows] running maximum and sum
    int* err;
};
// How a call is cut, by sizes alone.
struct CachedPlan { int places, part_rows, split; int64_t tiles, line; size_t bytes; };
CachedPlan cached_plan(const KvGeom& g, int n, int64_t tokens, int most_new, int max_pages, int q_heads, int bf16);
// Workgroups of a CU at a time, by the registers that a row of 32 `words` channels takes.
constexpr int cached_per_cu(int words, bool bf16) { return words <= 4 ? (bf16 ? 3 : 2) : words <= 6 && bf16 ? 2 : 1; }
hipError_t launch_cached(const CachedArgs& a, const CachedPlan& p, hipStream_t s);

// Attention over packed sequences.
struct PackedArgs {
    const void *q, *k, *v;  // [Tq][q_heads][D], [Tk][kv_heads][D]; tokens ld* elements apart
    int64_t ldq, ldk, ldv;
    int bf16, D, q_heads, kv_heads, per_head;
    int Tq, Tk, n;
    const int32_t *offsets_q, *offsets_k;  // [n + 1]
    int causal, window;                    // window: 0 none
    float scale, scale_log2;               // scale / ln 2
    void* out;                             // forward: written; backward: read
    int64_t ldo;
    float* lse;                            // [Tq][q_heads], forward: or null
    int* err;
    // backward
    const void* dout;
    int64_t lddo;
    void *dq, *dk, *dv;
    int64_t lddq, lddk, lddv;
    float2* rows;                          // workspace [q_heads][Tq]: lse / ln 2, delta
};
hipError_t launch_attention_bf16(const PackedArgs& a, hipStream_t s);
hipError_t launch_attention_f32(const PackedArgs& a, hipStream_t s);
hipError_t launch_attention_backward_bf16(const PackedArgs& a, hipStream_t s);
hipError_t launch_attention_backward_f32(const PackedArgs& a, hipStream_t s);

}  // namespace moe
