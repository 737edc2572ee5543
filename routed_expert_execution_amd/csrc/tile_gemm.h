// Matrix products on the matrix cores, tiles of both operands in LDS:
//   C[m, n] = sum_k A(m, k) B(n, k)
// for operands stored along k (kAlongK: element (r, k) at p[r * ld + k]) or
// across it (kAcrossK: at p[k * ld + r], so that a gradient's transposed
// operand is read as it lies), bf16 or fp32, any sizes.
#pragma once

#include "bf16_terms.h"
#include "device_util.h"

namespace moe {
namespace tile {

typedef bf16x8_t bf16x8;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

enum { kAlongK = 0, kAcrossK = 1 };

template <bool BF16> struct Elem;
template <> struct Elem<true> { typedef __bf16 type; typedef uint16_t raw; static constexpr int kChunk = 8; };
template <> struct Elem<false> { typedef float type; typedef uint32_t raw; static constexpr int kChunk = 4; };

struct __attribute__((packed, aligned(2))) Loose { u32x4 v; };

// An operand of one or two products.
struct Operand {
    const void* p[2];
    int64_t ld;
    int padded;  // its lines are whole 16-byte chunks in memory, whatever their length
};

// A wave-uniform pointer in scalar registers, where the compiler does not see
// that it is one.
__device__ inline const void* uniform(const void* p) {
    const uint64_t b = (uint64_t)p;
    return (const void*)((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) << 32 |
                         (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b));
}

// 16 bytes a lane from base + offset straight into LDS at `lds` + 16 * lane (lds
// and base wave-uniform; no register in between).  The compiler does not know of
// these loads: wait_loads_and_meet() before their first use.  Nor does it count
// wait states inside the block: the load needs one after M0, which takes its LDS
// address, is set, and five after a vector instruction (the v_readfirstlane of
// `base`, which may come right before the block) has written the scalar registers
// of its address.
__device__ inline void load_lds16(uint32_t lds, uint32_t offset, const void* base) {
    asm volatile(
        "s_nop 4\n\t"
        "global_load_lds_dwordx4 %0, %1"
        :
        : "v"(offset), "s"(uniform(base)), "{m0}"(__builtin_amdgcn_readfirstlane(lds))
        : "memory");
}
// This wave's loads into LDS have landed and its LDS reads are done (s_waitcnt
// vmcnt(0) lgkmcnt(0)), then the workgroup meets: the tile is whole and the
// other buffer is free.
__device__ inline void wait_loads_and_meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// Scheduling of one products step: READS LDS reads spread over its first PRODUCTS matrix instructions.
template <int READS, int PRODUCTS, int I = 0>
__device__ inline void spread_reads() {
    if constexpr (I < PRODUCTS) {
        constexpr int kPer = (READS + PRODUCTS - 1) / PRODUCTS;
        constexpr int n = READS - I * kPer < kPer ? READS - I * kPer : kPer;
        if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x100, n, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        spread_reads<READS, PRODUCTS, I + 1>();
    }
}
__device__ inline uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

// 16 bytes of an operand in its storage order: elements `in` .. +chunk of line
// `line` (along k: line is a row, in a column; across k the other way round),
// zero where the line or the element is past the end.
template <bool BF16>
__device__ inline u32x4 load_chunk(const void* p, int64_t ld, int64_t line, int64_t in, int64_t lines, int64_t ins) {
    typedef typename Elem<BF16>::raw raw;
    constexpr int E = Elem<BF16>::kChunk;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (line >= lines || in >= ins) return v;
    const raw* q = (const raw*)p + line * ld + in;
    if (in + E <= ins) return ((const Loose*)q)->v;
    raw e[E];
#pragma unroll
    for (int i = 0; i < E; i++) e[i] = in + i < ins ? q[i] : (raw)0;
    __builtin_memcpy(&v, e, 16);
    return v;
}

// Operands of one product of 16 columns for 32 rows: lane l holds row l % 32,
// columns 8 (l / 32) + 0..7, as they come from LDS (raw) and as the matrix cores
// take them.  bf16 is taken as it is.  fp32 is taken as three bf16 terms,
// x = a + b + c to 24 bits, and a product as the six products of terms that are
// above 2^-25 of it.  Measured, 2048 tokens through 1024 x 2048 forward: 102 us,
// 1.01 PFLOP/s of bf16 products, as many as the bf16 kernels reach at this size,
// 168 TFLOP/s of fp32 ones; with the fp32 matrix instruction the same tiles took
// 1.25 times as long.  Terms made once on the way into LDS (105 us, and 80 for 51
// where a CU has one workgroup, of which only one fits then) or between the
// products by hand (105) gained nothing.
template <bool BF16> struct Fragment;
template <> struct Fragment<true> {
    bf16x8 raw;
    __device__ void split() {}
};
template <> struct Fragment<false> {
    float raw[8];
    bf16x8 t[3];
    __device__ void split() { bf16_terms(raw, t); }
};
__device__ inline void mma(f32x16& acc, const Fragment<true>& a, const Fragment<true>& b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.raw, b.raw, acc, 0, 0, 0);
}
__device__ inline void mma(f32x16& acc, const Fragment<false>& a, const Fragment<false>& b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[2], b.t[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[0], b.t[2], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[1], b.t[1], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[1], b.t[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[0], b.t[1], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.t[0], b.t[0], acc, 0, 0, 0);
}

// Tile of BR rows by BK columns (BK elements fill 128 bytes) in LDS.  Along k:
// [BR][128 B], 16-byte chunk c of row r at c ^ (r / 2 % 8).  Across k: [BK][BR].
// bf16 lines are read back through the transposing LDS load: there the four
// lines of a 16-lane read are spread over the banks by xor of the chunk with
// 4 (k % 4).  fp32 lines are read a word a lane; the two halves of a wave read
// lines 8 apart, spread by xor with 8 (k / 8 % 2).
template <bool BF16, int BR, int LAY>
struct TileOf {
    static constexpr int E = Elem<BF16>::kChunk;
    static constexpr int BK = 8 * E;
    static constexpr int kBytes = BR * 128;
    static constexpr int kLineChunks = LAY == kAlongK ? 8 : BR / E;  // 16-byte chunks a line
    static constexpr int kChunks = kBytes / 16;
    static constexpr int kSteps = BK / 16;  // products steps of a tile
    static constexpr int kReads = (BF16 ? 1 : 2) * (LAY == kAlongK ? 1 : BF16 ? 2 : 4);  // LDS reads of one frag()

    __device__ static int chunk_at(int line, int c) {  // LDS byte offset
        if (LAY == kAlongK) return line * 128 + ((c ^ (line >> 1 & 7)) << 4);
        if (BF16) return (line * kLineChunks + (c ^ (line & 3) * (kLineChunks >= 16 ? 4 : 2))) << 4;
        return (line * kLineChunks + (c ^ (line >> 3 & 1) << 3)) << 4;
    }
    // Operand of the 32 rows at r0 for products step kk.
    __device__ static void frag(const char* lds, int r0, int kk, int lane, Fragment<true>& f) {
        if (LAY == kAlongK) {
            f.raw = *(const bf16x8*)(lds + chunk_at(r0 + (lane & 31), 2 * kk + (lane >> 5)));
        } else {
            const int k = 16 * kk + 8 * (lane >> 5) + (lane >> 2 & 3);
            const int col = r0 + 16 * (lane >> 4 & 1) + 4 * (lane & 3);
            s16x8 v;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                typedef __attribute__((address_space(3))) s16x4 lds4;
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds4*)(lds + chunk_at(k + 4 * h, col >> 3) + ((col & 7) << 1)));
#pragma unroll
                for (int i = 0; i < 4; i++) v[4 * h + i] = t[i];
            }
            f.raw = __builtin_bit_cast(bf16x8, v);
        }
    }
    __device__ static void frag(const char* lds, int r0, int kk, int lane, Fragment<false>& f) {
        const int r = r0 + (lane & 31);
        if (LAY == kAlongK) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const f32x4 v = *(const f32x4*)(lds + chunk_at(r, 4 * kk + 2 * (lane >> 5) + h));
#pragma unroll
                for (int i = 0; i < 4; i++) f.raw[4 * h + i] = v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                f.raw[i] = *(const float*)(lds + chunk_at(16 * kk + 8 * (lane >> 5) + i, r >> 2) + ((r & 3) << 2));
        }
    }
};

// The products are taken with the operands exchanged, so that a lane's result
// registers run along n: register i of a 32 x 32 block is row lane % 32 and
// column acc_col(lane, i), four at a time side by side.
__device__ inline int acc_col(int lane, int i) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// silu for a result that is rounded to bf16: hardware exp2 and reciprocal, a few
// fp32 steps of error (at g far below zero |g| of them, where the value vanishes).
__device__ inline float silu_fast(float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}

}  // namespace tile
}  // namespace moe
