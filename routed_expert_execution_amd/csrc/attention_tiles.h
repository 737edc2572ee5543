// What the kernels of attention over packed sequences share: tiles of tokens in
// LDS, operands of the matrix cores from them, and which keys a row sees.
//
// Products are taken so that a lane holds one row of a result: S^T = K Q^T has the
// row (of queries) of lane % 32 and 16 keys in its registers.  The next product
// sums over these keys, O^T = V^T P^T, and takes its operands' keys in the order in
// which the registers hold them, so that P goes from one product into the next
// without leaving the lane.  The backward products are laid out likewise.
#pragma once

#include "attention_device.h"
#include "tile_gemm.h"

namespace moe {
namespace packed {

using tile::f32x16;
using tile::Fragment;
using tile::mma;
using tile::s16x4;
using tile::s16x8;
using tile::u32x4;
typedef bf16x8_t bf16x8;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kInf = __builtin_huge_valf(), kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;

// The larger, NaN where one is: one instruction for three values (fmaxf, which takes
// the other one, has the compiler quieten each first).
__device__ inline float max_of(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Key of result register i of a 32 x 32 block in lane half h: 8 (i / 4) + 4 h + i % 4.
__device__ inline int reg_line(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// A tile of R lines (tokens) of D channels in LDS: 16-byte chunks, lines padded to a
// power of two of them; chunk c of line r lies at c ^ x(r), such that 16 lines read
// at one chunk, and the 4 lines x 32 bytes that a transposing read takes, lie in
// different banks.  (Heads of 96 and 192 channels pay for the padding with a third more LDS
// and loads: what goes straight into LDS fills the pad too.)
template <bool BF16, int D>
struct Tile {
    static constexpr int kPer = BF16 ? 8 : 4;  // elements a chunk
    static constexpr int kChunks = D / kPer;
    static constexpr int kLine = kChunks <= 8 ? 8 : kChunks <= 16 ? 16 : kChunks <= 32 ? 32 : 64;
    static constexpr int kLineBytes = kLine * 16;

    __device__ static int at(int r, int c) {
        const int x = kLine == 8 ? (r >> 1 & 3) * 2 ^ (r >> 3 & 1) : (r & 7) * 2 ^ (r >> 3 & 1);
        return (r * kLine + (c ^ x)) << 4;
    }
    // Operands, read at the tile's LDS address plus the lane's part of it.  What differs
    // between the reads of one lane is a constant: bits of the chunk's number, which the
    // swizzle leaves where they are (xor), and whole lines (the instruction's offset).
    // Lane's part of along(): line lane % 32, and of across(): lines 4 (lane / 32) + .. on.
    __device__ static uint32_t along_lane(int lane) { return at(lane & 31, (BF16 ? 1 : 2) * (lane >> 5)); }
    __device__ static uint32_t across_lane(int lane) {
        const int h = lane >> 5;
        if (BF16) return at(4 * h + (lane >> 2 & 3), 2 * (lane >> 4 & 1) + (lane >> 1 & 1)) + (lane & 1) * 8;
        return at(4 * h, (lane & 31) >> 2) + (lane & 3) * 4;
    }
    // A line a lane: lines r0 + lane % 32 (r0 a multiple of 32), channels 16 kk + 8 (lane / 32) + 0..7.
    __device__ static void along(uint32_t from, int r0, int kk, Fragment<BF16>& f) {
        if constexpr (BF16) {
            f.raw = *(__attribute__((address_space(3))) const bf16x8*)(uintptr_t)((from ^ (32 * kk)) + r0 * kLineBytes);
        } else {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const f32x4 v = *(__attribute__((address_space(3))) const f32x4*)(uintptr_t)((from ^ (64 * kk + 16 * i)) + r0 * kLineBytes);
#pragma unroll
                for (int e = 0; e < 4; e++) f.raw[4 * i + e] = v[e];
            }
        }
    }
    // A channel a lane, c0 + lane % 32 (c0 a multiple of 32), over the 16 lines from r0 on
    // (a multiple of 16) in the order of result registers: r0 + reg_line(e, lane / 32).
    __device__ static void across(uint32_t from, int r0, int c0, Fragment<BF16>& f) {
        if constexpr (BF16) {
            s16x8 v;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                typedef __attribute__((address_space(3))) s16x4 lds4;
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(uintptr_t)((from ^ (2 * c0 ^ 16 * i)) + (r0 + 8 * i) * kLineBytes));
#pragma unroll
                for (int e = 0; e < 4; e++) v[4 * i + e] = t[e];
            }
            f.raw = __builtin_bit_cast(bf16x8, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const int i = e >> 2, j = e & 3;
                f.raw[e] = *(__attribute__((address_space(3))) const float*)(uintptr_t)((from ^ (4 * c0 ^ 32 * j ^ 16 * i)) + (r0 + 8 * i + j) * kLineBytes);
            }
        }
    }
};

// An operand straight from memory, a line a lane: as Tile::along, zero past the lines' end.
template <bool BF16>
__device__ inline void along_memory(const void* p, int64_t line, bool inside, int kk, int lane, Fragment<BF16>& f) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if constexpr (BF16) {
        u32x4 w = {0, 0, 0, 0};
        if (inside) {
            const Words4 m = *(const Words4*)((const uint16_t*)p + line + 16 * kk + 8 * (lane >> 5));
            w = u32x4{m.v[0], m.v[1], m.v[2], m.v[3]};
        }
        f.raw = __builtin_bit_cast(bf16x8, w);
    } else {
        if (inside) load8<false>(p, line + 16 * kk + 8 * (lane >> 5), v);
#pragma unroll
        for (int e = 0; e < 8; e++) f.raw[e] = v[e];
    }
}

// Eight fp32 values as an operand.
__device__ inline void operand_of(const float (&v)[8], Fragment<true>& f) {
#pragma unroll
    for (int e = 0; e < 8; e++) f.raw[e] = (__bf16)v[e];
}
__device__ inline void operand_of(const float (&v)[8], Fragment<false>& f) {
#pragma unroll
    for (int e = 0; e < 8; e++) f.raw[e] = v[e];
    f.split();
}

// R lines of a tensor on their way from memory into a tile by THREADS threads, a
// chunk a thread at a time, zeros past `lines`.
template <bool BF16, int D, int R, int THREADS>
struct Staged {
    typedef Tile<BF16, D> T;
    static constexpr int kEach = (R * T::kChunks + THREADS - 1) / THREADS;
    u32x4 v[kEach];
    __device__ void load(const void* base, int64_t ld, int64_t first, int lines) {
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const int n = threadIdx.x + i * THREADS, r = n / T::kChunks, c = n - r * T::kChunks;
            v[i] = u32x4{0, 0, 0, 0};
            if (r < min(R, lines)) {
                const Words4 w = *(const Words4*)((const char*)base + ((first + r) * ld + c * T::kPer) * (BF16 ? 2 : 4));
                v[i] = u32x4{w.v[0], w.v[1], w.v[2], w.v[3]};
            }
        }
    }
    __device__ void store(char* lds) const {
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const int n = threadIdx.x + i * THREADS, r = n / T::kChunks, c = n - r * T::kChunks;
            if (n < R * T::kChunks) *(u32x4*)(lds + T::at(r, c)) = v[i];
        }
    }
};

// The same tile fetched ahead: straight into LDS (DIRECT) or by registers on the way.
// fetch() begins it, arrive() ends it; meet() lies between that and the first use.
// DIRECT: lines past the last repeat it, where the others hold zeros; both are masked.
template <bool BF16, int D, int R, int THREADS, bool DIRECT> struct Pipe;
template <bool BF16, int D, int R, int THREADS> struct Pipe<BF16, D, R, THREADS, false> {
    Staged<BF16, D, R, THREADS> s;
    __device__ void fetch(const char* base, int64_t ld, int64_t first, int lines, char*) { s.load(base, ld, first, lines); }
    __device__ void arrive(char* lds) const { s.store(lds); }
};
template <bool BF16, int D, int R, int THREADS> struct Pipe<BF16, D, R, THREADS, true> {
    typedef Tile<BF16, D> T;
    static constexpr int kEach = R * T::kLine / THREADS;
    static_assert(R * T::kLine % THREADS == 0, "whole waves");
    __device__ void fetch(const char* base, int64_t ld, int64_t first, int lines, char* lds) {
        const uint32_t line_bytes = (uint32_t)ld * (BF16 ? 2 : 4);
        const char* p = base + first * ld * (BF16 ? 2 : 4);
        const uint32_t to = tile::lds_address(lds) + (threadIdx.x >> 6) * 1024;
        // this lane's 16 bytes of LDS, and the line and chunk that belong there: of the
        // next ones too, whole multiples of 16 lines on
        constexpr int kStep = THREADS / T::kLine;
        if (kStep % 16 == 0 && lines >= R) {
            const int r = threadIdx.x / T::kLine, c = (T::at(r, threadIdx.x % T::kLine) >> 4) % T::kLine;
            const uint32_t offset = r * line_bytes + (c < T::kChunks ? c : 0) * 16;
#pragma unroll
            for (int i = 0; i < kEach; i++) tile::load_lds16(to + i * THREADS * 16, offset, p + (int64_t)i * kStep * line_bytes);
            return;
        }
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const int n = threadIdx.x + i * THREADS, r = n / T::kLine, c = (T::at(r, n % T::kLine) >> 4) % T::kLine;
            tile::load_lds16(to + i * THREADS * 16, min(r, lines - 1) * line_bytes + (c < T::kChunks ? c : 0) * 16, p);
        }
    }
    __device__ void arrive(char*) const {}
};
// Lines of a bf16 tensor straight into a tile of LDS, for loops that step through it: the
// lane's places from the first line on are kept, and a wave's loads are one block, with
// one wait for the scalar registers of their address (see tile::load_lds16).
template <int D, int R, int THREADS> struct LinesToLds {
    typedef Tile<true, D> T;
    static constexpr int kLoading = R * T::kLine < THREADS ? R * T::kLine : THREADS;  // threads that do
    static constexpr int kEach = R * T::kLine / kLoading;
    static_assert(R * T::kLine % kLoading == 0 && (kEach == 1 || kEach == 2 || kEach == 4), "the blocks below");
    uint32_t at[kEach];
    __device__ void places(int64_t ld, int lines) {  // lines past the last repeat it
#pragma unroll
        for (int i = 0; i < kEach; i++) {
            const int n = threadIdx.x + i * THREADS, r = n / T::kLine, c = (T::at(r, n % T::kLine) >> 4) % T::kLine;
            at[i] = min(r, lines - 1) * (uint32_t)ld * 2 + (c < T::kChunks ? c : 0) * 16;
        }
    }
    __device__ void fetch(const char* first, uint32_t lds, int wave) const {
        if (kLoading < THREADS && wave >= kLoading / 64) return;
        uint32_t to = __builtin_amdgcn_readfirstlane(lds + wave * 1024);
        const void* p = tile::uniform(first);
        if constexpr (kEach == 1)
            asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" : "+{m0}"(to) : "v"(at[0]), "s"(p) : "memory");
        else if constexpr (kEach == 2)
            asm volatile(
                "s_nop 4\n\tglobal_load_lds_dwordx4 %1, %3\n\t"
                "s_add_u32 m0, m0, %4\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3"
                : "+{m0}"(to) : "v"(at[0]), "v"(at[1]), "s"(p), "i"(THREADS * 16) : "memory", "scc");
        else
            asm volatile(
                "s_nop 4\n\tglobal_load_lds_dwordx4 %1, %5\n\t"
                "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %5\n\t"
                "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %3, %5\n\t"
                "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %4, %5"
                : "+{m0}"(to) : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "s"(p), "i"(THREADS * 16) : "memory", "scc");
    }
};
template <bool DIRECT> __device__ inline void meet() {
    if (DIRECT) tile::wait_loads_and_meet();
    else __syncthreads();
}
// 4 bytes a lane from base + offset straight into LDS at `lds` + 4 * lane (see tile::load_lds16).
__device__ inline void load_lds4(uint32_t lds, uint32_t offset, const void* base) {
    asm volatile(
        "s_nop 4\n\t"
        "global_load_lds_dword %0, %1"
        :
        : "v"(offset), "s"(tile::uniform(base)), "{m0}"(__builtin_amdgcn_readfirstlane(lds))
        : "memory");
}
// Lines that may go straight into LDS: whole 16-byte chunks, a tile of 128 within 32 bits.
inline bool direct_lines(const void* p, int64_t ld, bool bf16) {
    const int64_t bytes = ld * (bf16 ? 2 : 4);
    return (uintptr_t)p % 16 == 0 && bytes % 16 == 0 && bytes * 128 < ((int64_t)1 << 31);
}
// Whether a tile in LDS holds a value that is not finite (this thread's part of it).
template <bool BF16, int D, int R, int THREADS>
__device__ inline bool tile_not_finite(const char* lds) {
    typedef Tile<BF16, D> T;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < (R * T::kChunks + THREADS - 1) / THREADS; i++) {
        const int n = threadIdx.x + i * THREADS, r = n / T::kChunks, c = n - r * T::kChunks;
        if (n < R * T::kChunks) {
            const u32x4 v = *(const u32x4*)(lds + T::at(r, c));
#pragma unroll
            for (int e = 0; e < 4; e++) bad |= (BF16 && (v[e] & 0x7F80u) == 0x7F80u) || (v[e] & 0x7F800000u) == 0x7F800000u;
        }
    }
    return bad;
}

// acc += a b where b's values are 0 for pairs that do not see each other, and a may
// hold values that are not finite: 0 times these must add nothing.  They are taken
// out, and results that see one become NaN.  seen: 1 or 0 for each of b's pairs.
__device__ inline void mma_seen(f32x16& acc, const Fragment<true>& a, const Fragment<true>& b, const bf16x8& seen) {
    // (in words and out of the compiler's sight: it takes a test of a bf16's bits for
    // not finite to be false)
    u32x4 w = __builtin_bit_cast(u32x4, a.raw), odd;
    bool any = false;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        uint32_t v = w[e];
        asm("" : "+v"(v));
        const bool lo = (v & 0x7F80u) == 0x7F80u, hi = (v & 0x7F800000u) == 0x7F800000u;
        any |= lo || hi;
        odd[e] = (lo ? 0x3F80u : 0u) | (hi ? 0x3F800000u : 0u);
        w[e] = (lo ? 0u : v & 0xFFFFu) | (hi ? 0u : v & 0xFFFF0000u);
    }
    Fragment<true> clean;
    clean.raw = __builtin_bit_cast(bf16x8, w);
    mma(acc, clean, b);
    if (__any(any)) {
        f32x16 n;
#pragma unroll
        for (int i = 0; i < 16; i++) n[i] = 0;
        n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, odd), seen, n, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 16; i++) acc[i] = n[i] > 0.f ? __uint_as_float(0x7FC00000u) : acc[i];
    }
}
__device__ inline void mma_seen(f32x16& acc, const Fragment<false>& a, const Fragment<false>& b, const bf16x8& seen) {
    Fragment<false> clean;
    bf16x8 odd;
    bool any = false;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        uint32_t v = __float_as_uint(a.raw[e]);
        asm("" : "+v"(v));
        const bool bad = (v & 0x7F800000u) == 0x7F800000u;
        any |= bad;
        odd[e] = (__bf16)(bad ? 1.f : 0.f);
        clean.raw[e] = bad ? 0.f : a.raw[e];
    }
    clean.split();
    mma(acc, clean, b);
    if (__any(any)) {
        f32x16 n;
#pragma unroll
        for (int i = 0; i < 16; i++) n[i] = 0;
        n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(odd, seen, n, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 16; i++) acc[i] = n[i] > 0.f ? __uint_as_float(0x7FC00000u) : acc[i];
    }
}

// A result that met an infinity: NaN, as a masked tile's values give it (mma_seen), and not
// an infinity or NaN by where in the sequence the value lies.
__device__ inline float nan_if_infinite(float v) { return fmaf(v, 0.f, v); }

// A sequence's rows of queries and keys; what lies outside the tensors is cut off
// and makes it bad.
struct Sequence {
    int q0, rows, k0, keys;
    bool bad;
    int shift;  // row i sees keys up to i + shift if causal
};
__device__ inline int clamp_to(int v, int T) { return min(max(v, 0), T); }
__device__ inline Sequence sequence_of(const PackedArgs& a, int s) {
    const int qa = a.offsets_q[s], qb = a.offsets_q[s + 1], ka = a.offsets_k[s], kb = a.offsets_k[s + 1];
    Sequence r;
    r.bad = qa < 0 || qb < qa || qb > a.Tq || ka < 0 || kb < ka || kb > a.Tk;
    r.q0 = clamp_to(qa, a.Tq);
    r.rows = max(0, clamp_to(qb, a.Tq) - r.q0);
    r.k0 = clamp_to(ka, a.Tk);
    r.keys = max(0, clamp_to(kb, a.Tk) - r.k0);
    r.shift = r.keys - r.rows;
    return r;
}
// Tile `slot` of all sequences' tiles of B tokens: sequence s has the slots from
// offsets[s] / B + s on, as many as it has tiles or one more, so that a slot's
// sequence is found without a sum over the others.
template <int B>
__device__ inline bool find_tile(const int32_t* offsets, int n, int T, int slot, int* seq, int* local) {
    auto first = [&](int i) { return (int64_t)(clamp_to(offsets[i], T) / B + i); };
    *seq = __builtin_amdgcn_readfirstlane(wave_find(n, slot, first));
    *local = __builtin_amdgcn_readfirstlane((int)(slot - first(*seq)));
    return *local >= 0;
}
inline int64_t tile_slots(int T, int B, int n) { return (int64_t)T / B + n; }

// Which lines of a tile from `first` on a lane's row (or key) sees: those of the
// result registers i of block b with lo <= 32 b + 8 (i / 4) + i % 4 < hi.
struct Span {
    int lo, hi;
    __device__ bool has(int b, int i) const {
        const int c = 32 * b + 8 * (i >> 2) + (i & 3);
        return c >= lo && c < hi;
    }
};
__device__ inline Span keys_seen(const PackedArgs& a, const Sequence& s, int row, int first, int h) {
    const int off = first + 4 * h, last = row + s.shift;
    return {a.window ? last - a.window + 1 - off : INT32_MIN, (a.causal ? min(s.keys, last + 1) : s.keys) - off};
}
__device__ inline Span rows_seeing(const PackedArgs& a, const Sequence& s, int key, int first, int h) {
    const int off = first + 4 * h, own = key - s.shift;
    return {a.causal ? own - off : INT32_MIN, (a.window ? min(s.rows, own + a.window) : s.rows) - off};
}

}  // namespace packed
}  // namespace moe
