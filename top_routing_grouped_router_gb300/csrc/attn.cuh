// attn.cuh -- shared by the attention kernels: the batch's device arrays with their
// checks, the mapping of row tiles onto ragged chunks, element conversions and launchers.
#pragma once

#include "moe_internal.cuh"

namespace moe {
namespace attn {

// What every kernel of this file set gets of a call, by value.
struct Args {
    const int32_t *cu_q, *kv_len, *table;
    const void *k, *v;
    int64_t page_stride, head_stride, token_stride;  // elements
    int32_t n_tokens, n_seqs, n_heads, n_kv_heads, head_dim, group;
    int32_t page_size, n_pages, max_pages, max_q;
    int32_t page_shift;  // log2(page_size), -1 if it is no power of two
    const void *q;
    void *out;
    float *lse;
    int64_t q_stride, out_stride;
    float scale;
    int32_t *err;
};

struct Seq {
    int q0;      // first row of the chunk
    int q_len;   // rows
    int kv_len;  // keys, the chunk's own included
    bool rows_ok;  // cu_q rises within [0, n_tokens] here
};

// Sequence b, forced into the arrays' bounds; a value that had to be forced is recorded.
// Read after griddep_wait: the caller's arrays may come from an earlier kernel.
__device__ __forceinline__ Seq load_seq(const Args &a, int b) {
    const int c0 = ldp(a.cu_q + b), c1 = ldp(a.cu_q + b + 1), kv = ldp(a.kv_len + b);
    Seq s;
    s.q0 = min(max(c0, 0), a.n_tokens);
    s.q_len = max(min(max(c1, 0), a.n_tokens) - s.q0, 0);
    s.kv_len = int(min((int64_t)max(kv, 0), (int64_t)a.max_pages * a.page_size));
    s.rows_ok = c0 == s.q0 && c1 == s.q0 + s.q_len;
    if (!s.rows_ok || kv != s.kv_len || s.q_len > a.max_q) record_error(a.err, MOE_ERR_DEVICE);
    return s;
}

// The page that holds place p of sequence b (0 and a recorded error if the table is wrong).
__device__ __forceinline__ int load_page(const Args &a, int b, int page_index) {
    const int p = ldp(a.table + (size_t)b * a.max_pages + page_index);
    if (p < 0 || p >= a.n_pages) {
        record_error(a.err, MOE_ERR_DEVICE);
        return 0;
    }
    return p;
}

// Rows of one sequence and key head: row r is query head r mod group of new token r / group.
// Tiles of `rows` such rows are numbered through the batch; block-wide (every thread calls
// it): the sequence and the tile within it of tile number `tile`, or b = -1 past the last.
// scratch: 4 + blockDim.x / 32 ints of shared memory.
struct TileAt {
    int b, tile;
};
__device__ __forceinline__ TileAt find_tile(const Args &a, int tile, int tokens_per_tile, int *scratch) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nwarp = (blockDim.x + 31) >> 5;
    if (a.n_seqs <= 32) {  // every warp for itself, without barriers
        int n = 0;
        if (lane < a.n_seqs) {
            const int c0 = min(max(ldp(a.cu_q + lane), 0), a.n_tokens), c1 = min(max(ldp(a.cu_q + lane + 1), 0), a.n_tokens);
            n = (max(c1 - c0, 0) + tokens_per_tile - 1) / tokens_per_tile;
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const int b = __ffs(__ballot_sync(0xffffffffu, tile < incl)) - 1;
        return {b, tile - __shfl_sync(0xffffffffu, incl - n, max(b, 0))};
    }
    if (tid == 0) scratch[0] = -1;
    int base = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += blockDim.x) {
        int n = 0;
        if (b0 + tid < a.n_seqs) {
            const int c0 = min(max(ldp(a.cu_q + b0 + tid), 0), a.n_tokens);
            const int c1 = min(max(ldp(a.cu_q + b0 + tid + 1), 0), a.n_tokens);
            n = (max(c1 - c0, 0) + tokens_per_tile - 1) / tokens_per_tile;
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        __syncthreads();
        if (lane == 31) scratch[4 + warp] = incl;
        __syncthreads();
        int before = base, total = 0;
        for (int w = 0; w < nwarp; ++w) {
            const int t = scratch[4 + w];
            before += w < warp ? t : 0;
            total += t;
        }
        before += incl - n;
        if (tile >= before && tile < before + n) {
            scratch[0] = b0 + tid;
            scratch[1] = tile - before;
        }
        base += total;
        if (tile < base) break;  // base is the same for every thread
    }
    __syncthreads();
    return {scratch[0], scratch[1]};
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ void from_f32(float v, float *o) { *o = v; }
__device__ __forceinline__ void from_f32(float v, uint16_t *o) { *o = f32_to_bf16_bits(v); }

// Eight consecutive elements, 16-byte aligned.  ldp8: data an earlier kernel may have written.
__device__ __forceinline__ void ldp8(const float *p, float *v) {
    const float4 a = ldp16f(p), b = ldp16f(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void unpack8(const uint4 &a, float *v) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void ldp8(const uint16_t *p, float *v) { unpack8(ldp16(p), v); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(float *p, const float *v) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t *p, const float *v) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                               pack_bf16(v[6], v[7]));
}

// Two floats in one 64-bit register, for the paired fp32 instructions: one issue slot for two.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

// Partial results of a row over a part of its keys, in the workspace after the header:
// unnormalised output [part][row][head_dim] fp32, then (max, sum) [part][row] float2, the
// max in log2 units (scale * log2 e applied).  row = token * n_heads + head.
struct Partials {
    float *o;
    float2 *ml;
    int parts;
};

size_t generic_ws_bytes(const moe_attn_shape &s);
cudaError_t launch_generic(const Args &a, int dtype, const moe_attn_shape &s, char *ws, cudaStream_t st);
bool decode_supported(const moe_attn_shape &s);
size_t decode_ws_bytes(const moe_attn_shape &s);
cudaError_t launch_decode(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int sms, cudaStream_t st);
bool chunk_supported(const moe_attn_shape &s);
size_t chunk_ws_bytes(const moe_attn_shape &s);
cudaError_t launch_chunk(const Args &a, const moe_attn_shape &s, char *ws, int sms, cudaStream_t st);
cudaError_t launch_combine(const Args &a, int dtype, const Partials &p, cudaStream_t st);

}  // namespace attn

cudaError_t launch_rope(const moe_attn_shape &s, const moe_rope &r, const attn::Args &a, const void *k, int64_t k_stride,
                        const void *v, int64_t v_stride, const int32_t *positions, cudaStream_t st);
cudaError_t launch_q4_linear(const moe_q4_linear_shape &s, const void *x, int64_t x_stride, const moe_q4_weight &w,
                             const void *res, int64_t res_stride, void *out, int64_t out_stride, int sms,
                             cudaStream_t st);

}  // namespace moe
