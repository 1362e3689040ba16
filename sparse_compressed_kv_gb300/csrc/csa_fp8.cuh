// csa_fp8.cuh -- e4m3 codes and their scales on the device.
#pragma once

#include "csa_device.cuh"

namespace csa {

constexpr int kFp8MaxExp = 60;      // scales are 2^-60 .. 2^60

// 2^k, -126 <= k <= 127
__device__ __forceinline__ float exponent_f32(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// two values to e4m3 (to nearest, ties to even, saturating; NaN stays NaN), the
// first in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | e4m3x2(c, d) << 16;
}

// two codes to f16, exactly
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return r;
}
__device__ __forceinline__ float2 f16x2_values(uint32_t h) {
    float2 v;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "r"(h));
    return v;
}
__device__ __forceinline__ void e4m3x4_values(uint32_t codes, float *v) {
    const float2 a = f16x2_values(e4m3x2_f16x2(codes)), b = f16x2_values(e4m3x2_f16x2(codes >> 16));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

// ---------------------------------------------------------------- tensor cores

// Instruction descriptor: kind::f8f6f4, A e4m3, B e4m3 or e5m2, f32 accumulator,
// M x N, A transposed (MN-major) or not.
template <int M, int N, bool kTransA, bool kE5m2B>
__device__ __forceinline__ constexpr uint32_t idesc_fp8() {
    return (1u << 4)                                // D: f32
           | ((kE5m2B ? 1u : 0u) << 10)             // (A: 0, e4m3)
           | ((kTransA ? 1u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// 8-bit operands from shared memory, K = 32
__device__ __forceinline__ void umma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same with A from tensor memory: row m in lane m, the 32 bytes of a K step in
// 8 columns.
__device__ __forceinline__ void umma_fp8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

}  // namespace csa
