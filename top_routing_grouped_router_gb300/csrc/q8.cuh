// q8.cuh -- values of the 8-bit cache: e4m3 codes, and the power of two of a block of tokens and head
// as a byte b that stands for 2^(b - 127) (255: NaN).  Four significant bits and a power of two are
// exact in bf16 as well as in fp16, so the tensor cores get the values as they are stored.
#pragma once

#include "attn.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace q8 {

// The exponents that an append writes: the smallest value other than 0 (2^-9 of the scale) and the
// largest (448 of it) are normal numbers of bf16.
constexpr int kLowest = -110, kHighest = 119;

__device__ __forceinline__ uint32_t ldp_byte(const uint8_t *p) {
    uint32_t v;
    asm volatile("ld.global.cg.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldp8b(const void *p) {
    uint2 v;
    asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
// 2^(b - 127); 2^-127 is no normal number, and 255 stands for NaN.
__device__ __forceinline__ float scale_of(uint32_t b) {
    return __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
}
// Two codes (the lower byte first) as fp16: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}
// Four codes as fp16, two and two.
__device__ __forceinline__ void to_f16x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
// The nearest codes of two values (ties to even, past 448 the largest; NaN stays NaN).
__device__ __forceinline__ uint32_t from_f32(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n\tcvt.u32.u16 %0, c;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint32_t from_f16x2(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f16x2 c, %1;\n\tcvt.u32.u16 %0, c;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
// Eight codes as floats times `scale`.
__device__ __forceinline__ void unpack8(const uint2 &w, float scale, float *v) {
    const uint32_t h[4] = {to_f16x2(w.x), to_f16x2(w.x >> 16), to_f16x2(w.y), to_f16x2(w.y >> 16)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        v[2 * i] = f.x * scale;
        v[2 * i + 1] = f.y * scale;
    }
}

}  // namespace q8
}  // namespace moe
