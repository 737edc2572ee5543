// A word of a packed 4-bit matrix (dense.h) as eight bf16 values for the matrix cores.
#pragma once

#include "bf16_terms.h"

namespace moe {

// The 8 codes less their zero point (integers of 8 bits at most: exact), columns in order.
__device__ inline bf16x8_t codes_less_zero(uint32_t w, float z) {
    uint32_t lo = w & 0x0F0F0F0Fu, hi = w >> 4 & 0x0F0F0F0Fu;
    asm("" : "+v"(lo), "+v"(hi));  // (else each code is cut out by itself: 27 instructions for 22)
    bf16x8_t v;
#pragma unroll
    for (int e = 0; e < 8; e++)  // column e: pair e / 2, half e % 2 of the word
        v[e] = (__bf16)((float)(uint8_t)((e / 2 % 2 ? hi : lo) >> (16 * (e % 2) + 8 * (e / 4))) - z);
    return v;
}

}  // namespace moe
