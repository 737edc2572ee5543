// fp32 values as sums of three bf16 terms, for products on the bf16 matrix cores.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// v = t[0] + t[1] + t[2], each term the rounding of what the ones before leave:
// 24 bits, all of an fp32 value from 2^-110 up.  Of a smaller one what lies below
// bf16's least value, 2^-133, is rounded off: at most 2^-134.  (Past 3.39e38, the
// largest bf16, the first term is an infinity.)  What a term leaves is exact, so it may be taken as a
// dot product with (-1, 0) or (0, -1): one instruction in place of a shift and
// a subtraction, 3.5 a value in all.  The two constants pass through a register
// because the instruction reads an inline -1.0 as fp32's bits, the other half.
__device__ inline void bf16_terms(const float (&v)[8], bf16x8_t (&t)[3]) {
    uint32_t low = 0x0000BF80u, high = 0xBF800000u;
    asm("" : "+s"(low));
    asm("" : "+s"(high));
    const bf16x2_t first = __builtin_bit_cast(bf16x2_t, low), second = __builtin_bit_cast(bf16x2_t, high);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float a = v[i], b = v[i + 1];
#pragma unroll
        for (int c = 0; c < 3; c++) {
            bf16x2_t p;
            p[0] = (__bf16)a;
            p[1] = (__bf16)b;
            t[c][i] = p[0];
            t[c][i + 1] = p[1];
            if (c < 2) {
                a = __builtin_amdgcn_fdot2_f32_bf16(p, first, a, false);
                b = __builtin_amdgcn_fdot2_f32_bf16(p, second, b, false);
            }
        }
    }
}

}  // namespace moe
