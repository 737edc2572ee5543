// The attention layer's C entry points: checks of arguments, dispatch.
// (As for the dense layers, arguments are judged before the context's device, so
// that a host-only context names a bad argument too.)
#include <cmath>

#include "attention.h"
#include "host.h"

using namespace moe::host;

namespace {

constexpr int64_t kMaxT = 1 << 22;
constexpr int32_t kMaxHeads = 1024;
constexpr int32_t kMaxSequences = 65536;

#define CHECK(cond, ...) \
    do { if (!(cond)) return fail(c, MOE_EINVAL, __VA_ARGS__); } while (0)
#define LAUNCH(call)                                                                             \
    do {                                                                                         \
        const hipError_t e_ = (call);                                                            \
        if (e_ != hipSuccess) return fail(c, MOE_EHIP, "%s: %s", fn, hipGetErrorString(e_));      \
        return MOE_OK;                                                                           \
    } while (0)

// Activations [T, heads, D] of one argument.
moe_status tokens_check(moe_ctx* c, const char* fn, const char* name, const void* p, int32_t dtype, int64_t T, int64_t width, int64_t ld) {
    CHECK(T == 0 || p, "%s: null %s", fn, name);
    CHECK(aligned_to(p, elem_bytes(dtype)), "%s: misaligned %s", fn, name);
    CHECK(T <= 1 || (ld >= width && ld <= ((int64_t)1 << 40)), "%s: tokens of %s must be at least %lld elements apart", fn, name, (long long)width);
    return MOE_OK;
}

moe_status rotary_check(moe_ctx* c, const char* fn, const moe_rotary* r, int32_t head_dim, moe::RotaryView* v) {
    CHECK(r->freqs && aligned_to(r->freqs, 4), "%s: null or misaligned frequencies", fn);
    CHECK(r->rot >= 2 && r->rot % 2 == 0 && r->rot <= head_dim, "%s: rot=%d not an even number in [2, head_dim]", fn, r->rot);
    CHECK(r->interleaved == 0 || r->interleaved == 1, "%s: interleaved must be 0 or 1", fn);
    CHECK(std::isfinite(r->scale), "%s: the rotary's scale is not finite", fn);
    *v = moe::RotaryView{r->freqs, r->rot / 2, r->interleaved, r->scale};
    return MOE_OK;
}

moe_status cache_check(moe_ctx* c, const char* fn, const moe_kv_cache* m, moe::KvGeom* g) {
    CHECK(m && m->data, "%s: null cache", fn);
    CHECK(g->init(m->pages, m->page_tokens, m->heads, m->head_dim, m->group),
          "%s: bad cache: pages >= 1, page_tokens a power of two in [16, 1024], heads in [1, 1024], head_dim 64, 96, 128, 192 or 256, "
          "group 32, 64 or 128 and a divisor of it", fn);
    CHECK(aligned_to(m->data, 16), "%s: cache data must be 16-byte aligned", fn);
    return MOE_OK;
}

// (sizes alone, so that workspaces can be asked for before there are arrays)
bool batch_sizes(const moe_kv_batch* b, int32_t page_tokens) {
    return b && b->n >= 0 && b->n <= kMaxSequences && b->max_pages >= 1 && (int64_t)b->max_pages * page_tokens <= (1 << 30) &&
           b->tokens >= 0 && b->tokens <= kMaxT && b->most_new >= 0 && b->most_new <= b->tokens;
}
moe_status batch_check(moe_ctx* c, const char* fn, const moe_kv_batch* b, int32_t page_tokens, moe::KvBatchView* v) {
    CHECK(batch_sizes(b, page_tokens),
          "%s: bad batch: n in [0, 65536], max_pages >= 1 and max_pages * page_tokens up to 2^30, tokens in [0, 2^22], most_new in [0, tokens]", fn);
    CHECK(b->n == 0 || (b->offsets && b->lengths && b->pages), "%s: null offsets, lengths or pages", fn);
    CHECK(aligned_to(b->offsets, 4) && aligned_to(b->lengths, 4) && aligned_to(b->pages, 4), "%s: misaligned offsets, lengths or pages", fn);
    *v = moe::KvBatchView{b->offsets, b->lengths, b->pages, b->n, b->max_pages, (int)b->tokens, (int)b->most_new};
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_rotary_freqs(int32_t rot, double base, int32_t kind, double factor, double context, double fast, double slow,
                            float* freqs, float* scale) {
    if (rot < 2 || rot % 2 || rot > 256 || !freqs || !scale || !(base > 1) || !std::isfinite(base)) return MOE_EINVAL;
    if (kind != MOE_ROTARY_PLAIN && (!(factor >= 1) || !std::isfinite(factor))) return MOE_EINVAL;
    const int half = rot / 2;
    double low = 0, high = 0;
    *scale = 1.0f;
    switch (kind) {
        case MOE_ROTARY_PLAIN:
        case MOE_ROTARY_LINEAR: break;
        case MOE_ROTARY_BASE:
            if (rot <= 2) return MOE_EINVAL;
            base *= std::pow(factor, (double)rot / (rot - 2));
            break;
        case MOE_ROTARY_RAMP: {
            if (!(context >= 1) || !(slow > 0) || !(fast > slow) || !std::isfinite(context) || !std::isfinite(fast)) return MOE_EINVAL;
            // the pair that turns n times: context * base^(-2 i / rot) = 2 pi n
            const double pi = 3.14159265358979323846;
            auto pair_of = [&](double n) { return rot * std::log(context / (2 * pi * n)) / (2 * std::log(base)); };
            low = std::fmax(std::floor(pair_of(fast)), 0);
            high = std::fmin(std::ceil(pair_of(slow)), rot - 1);  // (may lie past the last pair)
            if (high <= low) {  // all pairs on one side: none turns more than `slow` times, or all at least `fast`
                if (low == 0) low = high - 1;
                else high = low + 1;
            }
            *scale = (float)(0.1 * std::log(factor) + 1);
            break;
        }
        default: return MOE_EINVAL;
    }
    for (int i = 0; i < half; i++) {
        double f = std::pow(base, -2.0 * i / rot);
        if (kind == MOE_ROTARY_LINEAR) f /= factor;
        if (kind == MOE_ROTARY_RAMP) {
            const double t = std::fmin(std::fmax((i - low) / (high - low), 0), 1);
            f = f * (1 - t) + f / factor * t;
        }
        freqs[i] = (float)f;
    }
    return MOE_OK;
}

moe_status moe_rotate(moe_ctx* c, const void* x, int32_t dtype, int64_t ldx, int64_t T, int32_t heads, int32_t head_dim,
                      const int32_t* positions, const moe_rotary* rotary, int32_t inverse, void* y, int64_t ldy, moe_stream stream) {
    const char* fn = "moe_rotate";
    if (!c) return MOE_EINVAL;
    CHECK(T >= 0 && T <= kMaxT, "%s: T=%lld outside [0, 2^22]", fn, (long long)T);
    CHECK(heads >= 1 && heads <= kMaxHeads && moe::head_dim_valid(head_dim), "%s: heads in [1, 1024], head_dim 64, 96, 128, 192 or 256", fn);
    CHECK(dtype_valid(dtype), "%s: bad type", fn);
    const int64_t width = (int64_t)heads * head_dim;
    if (moe_status st = tokens_check(c, fn, "x", x, dtype, T, width, ldx)) return st;
    if (moe_status st = tokens_check(c, fn, "y", y, dtype, T, width, ldy)) return st;
    CHECK(T == 0 || (positions && aligned_to(positions, 4)), "%s: null or misaligned positions", fn);
    CHECK(rotary, "%s: null rotary", fn);
    CHECK(inverse == 0 || inverse == 1, "%s: inverse must be 0 or 1", fn);
    CHECK(x != y || T <= 1 || ldx == ldy, "%s: in place, but x and y differ in ld", fn);
    moe::RotateArgs a{x, T > 1 ? ldx : width, y, T > 1 ? ldy : width, dtype == MOE_BF16, T, heads, head_dim, positions, {}, inverse};
    if (moe_status st = rotary_check(c, fn, rotary, head_dim, &a.rotary)) return st;
    if (moe_status st = need_device(c)) return st;
    if (T == 0) return MOE_OK;
    DeviceGuard dg(device_of(c));
    LAUNCH(moe::launch_rotate(a, (hipStream_t)stream));
}

size_t moe_kv_bytes(int64_t pages, int32_t page_tokens, int32_t heads, int32_t head_dim, int32_t group) {
    moe::KvGeom g;
    return g.init(pages, page_tokens, heads, head_dim, group) ? (size_t)g.bytes : 0;
}

moe_status moe_kv_append(moe_ctx* c, const moe_kv_cache* cache, const moe_kv_batch* batch, const void* k, int64_t ldk,
                         const void* v, int64_t ldv, int32_t dtype, const moe_rotary* rotary, const int32_t* positions,
                         const void* q, int64_t ldq, int32_t q_heads, void* q_out, int64_t ldqo, moe_stream stream) {
    const char* fn = "moe_kv_append";
    if (!c) return MOE_EINVAL;
    moe::KvGeom g;
    moe::KvAppendArgs a{};
    if (moe_status st = cache_check(c, fn, cache, &g)) return st;
    if (moe_status st = batch_check(c, fn, batch, g.page_tokens, &a.batch)) return st;
    CHECK(dtype_valid(dtype), "%s: bad type", fn);
    const int64_t T = batch->tokens, width = (int64_t)g.heads * g.D;
    if (moe_status st = tokens_check(c, fn, "k", k, dtype, T, width, ldk)) return st;
    if (moe_status st = tokens_check(c, fn, "v", v, dtype, T, width, ldv)) return st;
    CHECK(aligned_to(positions, 4), "%s: misaligned positions", fn);
    if (rotary)
        if (moe_status st = rotary_check(c, fn, rotary, g.D, &a.rotary)) return st;
    CHECK(!q == !q_out, "%s: q without q_out, or q_out without q", fn);
    int64_t q_width = 0;
    if (q) {
        CHECK(q_heads >= 1 && q_heads <= kMaxHeads, "%s: q_heads=%d outside [1, 1024]", fn, q_heads);
        q_width = (int64_t)q_heads * g.D;
        if (moe_status st = tokens_check(c, fn, "q", q, dtype, T, q_width, ldq)) return st;
        if (moe_status st = tokens_check(c, fn, "q_out", q_out, dtype, T, q_width, ldqo)) return st;
        CHECK(q != q_out || T <= 1 || ldq == ldqo, "%s: in place, but q and q_out differ in ld", fn);
    }
    if (moe_status st = need_device(c)) return st;
    if (T == 0 || batch->n == 0) return MOE_OK;
    a.cache = moe::kv_view(g, cache->data);
    a.k = k; a.v = v;
    a.ldk = T > 1 ? ldk : width; a.ldv = T > 1 ? ldv : width;
    a.bf16 = dtype == MOE_BF16;
    a.positions = positions;
    a.q = q; a.q_out = q_out; a.q_heads = q ? q_heads : 0;
    a.ldq = T > 1 ? ldq : q_width; a.ldqo = T > 1 ? ldqo : q_width;
    a.err = error_word(c);
    DeviceGuard dg(device_of(c));
    LAUNCH(moe::launch_kv_append(a, (hipStream_t)stream));
}

moe_status moe_kv_read(moe_ctx* c, const moe_kv_cache* cache, const moe_kv_batch* batch, void* k, int64_t ldk, void* v,
                       int64_t ldv, int32_t dtype, moe_stream stream) {
    const char* fn = "moe_kv_read";
    if (!c) return MOE_EINVAL;
    moe::KvGeom g;
    moe::KvReadArgs a{};
    if (moe_status st = cache_check(c, fn, cache, &g)) return st;
    if (moe_status st = batch_check(c, fn, batch, g.page_tokens, &a.batch)) return st;
    CHECK(dtype_valid(dtype), "%s: bad type", fn);
    const int64_t T = batch->tokens, width = (int64_t)g.heads * g.D;
    if (moe_status st = tokens_check(c, fn, "k", k, dtype, T, width, ldk)) return st;
    if (moe_status st = tokens_check(c, fn, "v", v, dtype, T, width, ldv)) return st;
    if (moe_status st = need_device(c)) return st;
    if (T == 0 || batch->n == 0) return MOE_OK;
    a.cache = moe::kv_view(g, cache->data);
    a.k = k; a.v = v;
    a.ldk = T > 1 ? ldk : width; a.ldv = T > 1 ? ldv : width;
    a.bf16 = dtype == MOE_BF16;
    a.err = error_word(c);
    DeviceGuard dg(device_of(c));
    LAUNCH(moe::launch_kv_read(a, (hipStream_t)stream));
}

// The kernels' exponentials are powers of two: scale / ln 2 has to be finite as well.
static float scale_log2_of(float scale) { return (float)((double)scale * 1.4426950408889634); }
static bool scale_valid(float scale) { return scale > 0 && scale < 0x1p127f; }
static bool query_heads_valid(int32_t q_heads, int32_t heads) { return q_heads >= 1 && q_heads <= kMaxHeads && q_heads % heads == 0; }

size_t moe_attention_cached_workspace(const moe_kv_cache* m, const moe_kv_batch* b, int32_t q_heads) {
    moe::KvGeom g;
    if (!m || !g.init(m->pages, m->page_tokens, m->heads, m->head_dim, m->group) || !batch_sizes(b, g.page_tokens) ||
        !query_heads_valid(q_heads, g.heads))
        return 0;
    const size_t n = moe::cached_plan(g, b->n, b->tokens, (int)b->most_new, b->max_pages, q_heads, 1).bytes;
    return n < 256 ? 256 : n;
}

moe_status moe_attention_cached(moe_ctx* c, const moe_kv_cache* cache, const moe_kv_batch* batch, const void* q, int64_t ldq,
                                int32_t dtype, int32_t q_heads, float scale, int64_t window, void* out, int64_t ldo,
                                void* workspace, size_t workspace_bytes, moe_stream stream) {
    const char* fn = "moe_attention_cached";
    if (!c) return MOE_EINVAL;
    moe::KvGeom g;
    moe::CachedArgs a{};
    if (moe_status st = cache_check(c, fn, cache, &g)) return st;
    if (moe_status st = batch_check(c, fn, batch, g.page_tokens, &a.batch)) return st;
    CHECK(dtype_valid(dtype), "%s: bad type", fn);
    CHECK(query_heads_valid(q_heads, g.heads), "%s: q_heads=%d not a multiple of the cache's heads in [1, 1024]", fn, q_heads);
    const int64_t T = batch->tokens, width = (int64_t)q_heads * g.D;
    if (moe_status st = tokens_check(c, fn, "q", q, dtype, T, width, ldq)) return st;
    if (moe_status st = tokens_check(c, fn, "out", out, dtype, T, width, ldo)) return st;
    CHECK(scale_valid(scale), "%s: scale must be positive and below 2^127", fn);
    CHECK(window >= 0, "%s: negative window", fn);
    CHECK(workspace && aligned_to(workspace, 256), "%s: workspace must be 256-byte aligned", fn);
    const size_t need = moe_attention_cached_workspace(cache, batch, q_heads);
    CHECK(workspace_bytes >= need, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
    a.bf16 = dtype == MOE_BF16;
    const moe::CachedPlan p = moe::cached_plan(g, batch->n, T, (int)batch->most_new, batch->max_pages, q_heads, a.bf16);
    CHECK(p.line < ((int64_t)1 << 31) && p.tiles < (1 << 27), "%s: too many tokens over too long a page table for one call", fn);
    if (moe_status st = need_device(c)) return st;
    if (T == 0 || batch->n == 0) return MOE_OK;
    a.cache = moe::kv_view(g, cache->data);
    a.q = q; a.ldq = T > 1 ? ldq : width;
    a.per_head = q_heads / g.heads;
    a.scale_log2 = scale_log2_of(scale);
    a.window = (int)(window < (1 << 30) ? window : 0);  // (none reaches further back)
    a.out = out; a.ldo = T > 1 ? ldo : width;
    a.places = p.places; a.part_rows = p.part_rows;
    a.part = (float*)workspace;
    a.part_ml = (float2*)(a.part + (size_t)2 * p.places * g.heads * p.part_rows * g.D);
    a.err = error_word(c);
    DeviceGuard dg(device_of(c));
    LAUNCH(moe::launch_cached(a, p, (hipStream_t)stream));
}

// What both passes judge alike.
static moe_status attn_check(moe_ctx* c, const char* fn, const moe_attn* t, moe::PackedArgs* a) {
    CHECK(t, "%s: null description", fn);
    CHECK(t->n >= 0 && t->n <= kMaxSequences && t->tokens_q >= 0 && t->tokens_q <= kMaxT && t->tokens_k >= 0 && t->tokens_k <= kMaxT,
          "%s: n outside [0, 65536] or tokens outside [0, 2^22]", fn);
    CHECK(t->n == 0 || (t->offsets_q && t->offsets_k), "%s: null offsets", fn);
    CHECK(aligned_to(t->offsets_q, 4) && aligned_to(t->offsets_k, 4), "%s: misaligned offsets", fn);
    CHECK(dtype_valid(t->dtype), "%s: bad type", fn);
    CHECK(t->kv_heads >= 1 && t->kv_heads <= kMaxHeads && query_heads_valid(t->q_heads, t->kv_heads),
          "%s: q_heads=%d not a multiple of kv_heads=%d in [1, 1024]", fn, t->q_heads, t->kv_heads);
    CHECK(moe::head_dim_valid(t->head_dim), "%s: head_dim=%d not 64, 96, 128, 192 or 256", fn, t->head_dim);
    CHECK(t->causal == 0 || t->causal == 1, "%s: causal must be 0 or 1", fn);
    CHECK(t->window >= 0 && (t->window == 0 || t->causal), "%s: a window is not negative, and needs causal", fn);
    CHECK(scale_valid(t->scale), "%s: scale must be positive and below 2^127", fn);
    *a = moe::PackedArgs{};
    a->bf16 = t->dtype == MOE_BF16;
    a->D = t->head_dim; a->q_heads = t->q_heads; a->kv_heads = t->kv_heads; a->per_head = t->q_heads / t->kv_heads;
    a->Tq = (int)t->tokens_q; a->Tk = (int)t->tokens_k; a->n = t->n;
    a->offsets_q = t->offsets_q; a->offsets_k = t->offsets_k;
    a->causal = t->causal;
    a->window = (int)(t->window < (1 << 23) ? t->window : 0);  // (none reaches further back)
    a->scale = t->scale;
    a->scale_log2 = scale_log2_of(t->scale);
    // (a workgroup of 256 threads for each head of every 32 tokens at most, and one more a sequence: 2^32 threads)
    CHECK((t->tokens_q / 32 + t->n) * t->q_heads < ((int64_t)1 << 24) && (t->tokens_k / 32 + t->n) * t->kv_heads < ((int64_t)1 << 24),
          "%s: too many heads of too many tokens for one call", fn);
    return MOE_OK;
}

moe_status moe_attention(moe_ctx* c, const moe_attn* t, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                         int64_t ldv, void* out, int64_t ldo, float* lse, moe_stream stream) {
    const char* fn = "moe_attention";
    if (!c) return MOE_EINVAL;
    moe::PackedArgs a;
    if (moe_status st = attn_check(c, fn, t, &a)) return st;
    const int64_t Tq = t->tokens_q, Tk = t->tokens_k, qw = (int64_t)a.q_heads * a.D, kw = (int64_t)a.kv_heads * a.D;
    if (moe_status st = tokens_check(c, fn, "q", q, t->dtype, Tq, qw, ldq)) return st;
    if (moe_status st = tokens_check(c, fn, "k", k, t->dtype, Tk, kw, ldk)) return st;
    if (moe_status st = tokens_check(c, fn, "v", v, t->dtype, Tk, kw, ldv)) return st;
    if (moe_status st = tokens_check(c, fn, "out", out, t->dtype, Tq, qw, ldo)) return st;
    CHECK(aligned_to(lse, 4), "%s: misaligned lse", fn);
    if (moe_status st = need_device(c)) return st;
    if (Tq == 0 || t->n == 0) return MOE_OK;
    a.q = q; a.k = k; a.v = v; a.out = out; a.lse = lse;
    a.ldq = Tq > 1 ? ldq : qw; a.ldk = Tk > 1 ? ldk : kw; a.ldv = Tk > 1 ? ldv : kw; a.ldo = Tq > 1 ? ldo : qw;
    a.err = error_word(c);
    DeviceGuard dg(device_of(c));
    LAUNCH(a.bf16 ? moe::launch_attention_bf16(a, (hipStream_t)stream) : moe::launch_attention_f32(a, (hipStream_t)stream));
}

size_t moe_attention_workspace(int64_t tokens_q, int32_t q_heads) {
    if (tokens_q < 0 || tokens_q > kMaxT || q_heads < 1 || q_heads > kMaxHeads) return 0;
    const size_t n = (size_t)tokens_q * q_heads * sizeof(float2);
    return n < 256 ? 256 : n;
}

moe_status moe_attention_backward(moe_ctx* c, const moe_attn* t, const void* dout, int64_t lddo, const void* q, int64_t ldq,
                                  const void* k, int64_t ldk, const void* v, int64_t ldv, const void* out, int64_t ldo,
                                  const float* lse, void* dq, int64_t lddq, void* dk, int64_t lddk, void* dv, int64_t lddv,
                                  void* workspace, size_t workspace_bytes, moe_stream stream) {
    const char* fn = "moe_attention_backward";
    if (!c) return MOE_EINVAL;
    moe::PackedArgs a;
    if (moe_status st = attn_check(c, fn, t, &a)) return st;
    const int64_t Tq = t->tokens_q, Tk = t->tokens_k, qw = (int64_t)a.q_heads * a.D, kw = (int64_t)a.kv_heads * a.D;
    if (moe_status st = tokens_check(c, fn, "dout", dout, t->dtype, Tq, qw, lddo)) return st;
    if (moe_status st = tokens_check(c, fn, "q", q, t->dtype, Tq, qw, ldq)) return st;
    if (moe_status st = tokens_check(c, fn, "k", k, t->dtype, Tk, kw, ldk)) return st;
    if (moe_status st = tokens_check(c, fn, "v", v, t->dtype, Tk, kw, ldv)) return st;
    if (moe_status st = tokens_check(c, fn, "out", out, t->dtype, Tq, qw, ldo)) return st;
    if (moe_status st = tokens_check(c, fn, "dq", dq, t->dtype, Tq, qw, lddq)) return st;
    if (moe_status st = tokens_check(c, fn, "dk", dk, t->dtype, Tk, kw, lddk)) return st;
    if (moe_status st = tokens_check(c, fn, "dv", dv, t->dtype, Tk, kw, lddv)) return st;
    CHECK(Tq == 0 || (lse && aligned_to(lse, 4)), "%s: null or misaligned lse", fn);
    CHECK(workspace && aligned_to(workspace, 256), "%s: workspace must be 256-byte aligned", fn);
    const size_t need = moe_attention_workspace(Tq, a.q_heads);
    CHECK(workspace_bytes >= need, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
    if (moe_status st = need_device(c)) return st;
    if (t->n == 0) return MOE_OK;
    a.q = q; a.k = k; a.v = v; a.out = (void*)out; a.lse = (float*)lse; a.dout = dout; a.dq = dq; a.dk = dk; a.dv = dv;
    a.ldq = Tq > 1 ? ldq : qw; a.ldo = Tq > 1 ? ldo : qw; a.lddo = Tq > 1 ? lddo : qw; a.lddq = Tq > 1 ? lddq : qw;
    a.ldk = Tk > 1 ? ldk : kw; a.ldv = Tk > 1 ? ldv : kw; a.lddk = Tk > 1 ? lddk : kw; a.lddv = Tk > 1 ? lddv : kw;
    a.rows = (float2*)workspace;
    a.err = error_word(c);
    DeviceGuard dg(device_of(c));
    LAUNCH(a.bf16 ? moe::launch_attention_backward_bf16(a, (hipStream_t)stream) : moe::launch_attention_backward_f32(a, (hipStream_t)stream));
}

}  // extern "C"
