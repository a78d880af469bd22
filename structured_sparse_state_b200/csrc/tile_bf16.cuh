// bf16 tiles in shared memory: rows of 128 bytes, 128-byte swizzle, and the
// pairs of values they are made of.
#pragma once

#include "common.cuh"

namespace pdssm {

// Byte offset of 16-byte piece q of row r in such a tile.
__device__ __forceinline__ uint32_t piece(int r, int q) {
    return (uint32_t)(r * 128 + ((q ^ (r & 7)) << 4));
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// two values rounded to bf16 in one word, and back
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace pdssm
