// rope.cuh -- shared by the kernels that rotate new tokens' heads: their arguments, elements as they
// are loaded, and the layout of the cosines and sines in shared memory.
#pragma once

#include "attn.cuh"

namespace moe {

struct RopeArgs {
    attn::Args a;
    const void *k_in, *v_in;
    int64_t k_stride, v_stride;
    const int32_t *positions;
    const uint64_t *turns;
    const void *gq, *gk;
    int rot_dim, interleaved;
    float mscale, eps;
};

// Eight elements as loaded; get: as four pairs of floats.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = ldp16(p); }
    // through L1: weights that every row of the block reads (plain C++ loads: 1583 fp32 tokens 7.5 us, 6.6)
    __device__ __forceinline__ void load_cached(const uint16_t *p) {
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    }
    __device__ __forceinline__ void get(uint64_t *f) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = attn::pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = ldp16f(p);
        b = ldp16f(p + 4);
    }
    __device__ __forceinline__ void load_cached(const float *p) {
        asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w) : "l"(p));
        asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w) : "l"(p + 4));
    }
    __device__ __forceinline__ void get(uint64_t *f) const {
        f[0] = attn::pair(a.x, a.y);
        f[1] = attn::pair(a.z, a.w);
        f[2] = attn::pair(b.x, b.y);
        f[3] = attn::pair(b.z, b.w);
    }
};

// The 16-byte place of cosines and sines of pairs 2 q and 2 q + 1: rotated within eight places by
// q / 8, so that lanes eight (half layout: four places apart) or four pairs apart fall in
// different banks.
__device__ __forceinline__ int place_of(int q) { return (q & ~7) | ((q + (q >> 3)) & 7); }

}  // namespace moe
