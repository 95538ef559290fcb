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

// out[t][n] = y (+ residual[t][n]), rounded once.
__device__ __forceinline__ void q4_emit(const Q4Args &a, int64_t t, int n, float y) {
    if (a.res) y += bf16_bits_to_f32(ldp(a.res + t * a.res_stride + n));
    if (a.out_f32)
        static_cast<float *>(a.out)[t * a.out_stride + n] = y;
    else
        static_cast<uint16_t *>(a.out)[t * a.out_stride + n] = f32_to_bf16_bits(y);
}

bool run_tc(const Q4Args &a, float step, int twice_j0, int sms, cudaStream_t st, cudaError_t *err);
cudaError_t read_error(int32_t *code, cudaStream_t st);

}  // namespace q4
}  // namespace moe
