// q4_linear.cuh -- shared by the 4-bit linear's kernels: arguments, the unpacking of codes and
// scales, and the final write of a result.
#pragma once

#include "attn.cuh"

namespace moe {
namespace q4 {

struct Q4Args {
    const uint16_t *x;
    const uint8_t *codes;
    const uint16_t *scales;
    const uint16_t *res;
    void *out;
    int64_t x_stride, res_stride, out_stride;
    int T, K, N, q_block, out_f32;
    float codebook[16];
};

// (w & 0x00780078) | 0x41804180: two codes, already shifted to bits 3 .. 6 of each half, become
// the bf16 pair 16 + j, exactly.  Of a word's eight codes, << 3, >> 1, >> 5 and >> 9 give the
// pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t mask, uint32_t bias) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bias));
    return r;
}
// One 16-bit half of a word as a bf16 value: sel kLow the low one, kHigh the high one.
constexpr uint32_t kLow = 0x1044, kHigh = 0x3244;
__device__ __forceinline__ float half_of(uint32_t w, uint32_t sel) { return __uint_as_float(__byte_perm(w, 0, sel)); }

__device__ __forceinline__ bool q4_is_finite(float y) { return fabsf(y) < __builtin_inff(); }

// out[t][n] = y (+ residual[t][n]), rounded once.
__device__ __forceinline__ void q4_write(const Q4Args &a, int64_t t, int n, float y) {
    if (a.res) y += bf16_bits_to_f32(ldp(a.res + t * a.res_stride + n));
    if (a.out_f32)
        static_cast<float *>(a.out)[t * a.out_stride + n] = y;
    else
        static_cast<uint16_t *>(a.out)[t * a.out_stride + n] = f32_to_bf16_bits(y);
}

// A sum that the tensor cores left infinite or NaN is formed again, by its terms: (16 + j) x - (16 + j0) x of an
// infinite x is NaN where the sum is infinite, so is the zero low part of a general value times x, and
// x past 2^123 overflows on the way to a finite sum.  A wrong sum never comes out finite.  Inline: with a
// function call in its place 64 x 2048 x 131072 takes 127 us, so 125 (without the check 123), and 1 x 2048 x
// 5120 5.5, so 4.9.
__device__ __forceinline__ void q4_emit_by_terms(const Q4Args &a, int64_t t, int n) {
    const uint16_t *x = a.x + t * a.x_stride;
    for (int k = 0; k < a.K; k += 8) {  // a NaN decides, and is found without the weights
        float v[8];
        attn::ldp8(x + k, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (v[e] != v[e]) return q4_write(a, t, n, v[e]);
    }
    const uint8_t *codes = a.codes + (size_t)n * (a.K / 2);
    const uint16_t *scales = a.scales + (size_t)n * (a.K / a.q_block);
    float y = 0.f;
    for (int k = 0; k < a.K; k += 2) {  // q_block is even: a pair shares its scale
        const uint32_t c = codes[k / 2];
        const float s = bf16_bits_to_f32(scales[k / a.q_block]);
        y = fmaf(a.codebook[c & 15] * s, bf16_bits_to_f32(ldp(x + k)), y);
        y = fmaf(a.codebook[c >> 4] * s, bf16_bits_to_f32(ldp(x + k + 1)), y);
    }
    q4_write(a, t, n, y);
}

// Writes a finite sum; false, and nothing is written, for one that q4_emit_by_terms has to form.
__device__ __forceinline__ bool q4_emit(const Q4Args &a, int64_t t, int n, float y) {
    const bool finite = q4_is_finite(y);
    if (finite) q4_write(a, t, n, y);
    return finite;
}

bool run_tc(const Q4Args &a, float step, int twice_j0, int sms, cudaStream_t st, cudaError_t *err);
cudaError_t read_error(int32_t *code, cudaStream_t st);

}  // namespace q4
}  // namespace moe
