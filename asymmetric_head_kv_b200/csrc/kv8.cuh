// kv8.cuh -- device helpers of the 8-bit paged K/V cache (e4m3 codes, one power-of-two scale per
// block of positions and head).
#pragma once

#include "common.cuh"

namespace diffqkv {

// Exponents the writer gives a block.  2^e and 2^-e are normal binary32 numbers over this range, and
// an e4m3 code times 2^e is a finite bf16 number exactly (4 significant bits, from 2^-129 to 1.75 * 2^127).
constexpr int kKv8MinExp = -120;
constexpr int kKv8MaxExp = 119;

// A scale byte's exponent (2^(byte - 127)), held inside the range above whatever the byte.
__device__ __forceinline__ int kv8_exp(uint32_t byte) {
    return min(max((int)byte - 127, kKv8MinExp), kKv8MaxExp);
}

// 2^e as a binary32 number, -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// Two floats -> two e4m3 codes (lo in the low byte), to nearest even; magnitudes above 448,
// infinities among them, become 448 and NaN the NaN code.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (low 16 bits) -> two f16 values in one word (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}

__device__ __forceinline__ void f16x2_to_floats(uint32_t w, float &lo, float &hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.f32.f16 %0, l;\n\t"
        "cvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(w));
}

// One lane of a converged warp.  Instructions that take their operands from uniform registers (tcgen05.mma and commit,
// TMA) issue several times faster behind this than behind a test of the lane index, where the compiler cannot tell that
// one lane runs them: 45 against 239 clocks for an M 128, N 16, K 32 MMA on B200.  Their operands should be
// visibly uniform too (uniform() below for values that are not).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

}  // namespace diffqkv
