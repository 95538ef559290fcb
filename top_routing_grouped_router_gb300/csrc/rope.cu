// rope.cu -- rotary positions of the new tokens' q and k, with an optional RMS norm of each
// head before, and the write of k and v into the paged cache.
//
// One block works on one token: the cosines and sines of its rot_dim / 2 angles are shared by
// all its heads.  An angle is (turns_i * position) mod 2^64 in units of 2^-64 turn, an exact
// integer product, so no far position costs accuracy, and no range reduction is needed: the
// signed fraction of a turn goes to sincospi.
#include "attn.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

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

// A group of LG lanes (a power of two that covers head_dim / 8) holds one head, eight
// consecutive elements a lane, and goes over the token's n_heads + 2 n_kv_heads heads.
template <typename T, int LG>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs r) {
    __shared__ float2 cs[kMaxPairs];
    __shared__ int where[2];  // the token's sequence, its place
    griddep_wait();
    griddep_launch_dependents();
    const attn::Args &a = r.a;
    const int t = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) where[0] = -1;
    __syncthreads();
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const int c0 = ldp(a.cu_q + b), c1 = ldp(a.cu_q + b + 1);
        if (c0 <= t && t < c1) {
            where[0] = b;  // cu_q rises, so one b matches
            where[1] = ldp(a.kv_len + b) - (c1 - t);
        }
        if (t == 0 && (c0 < 0 || c1 < c0 || c1 > a.n_tokens)) record_error(a.err, MOE_ERR_DEVICE);
    }
    __syncthreads();
    const int b = where[0], place = where[1];
    if (b < 0) return;  // a padding row
    const int pairs = r.rot_dim / 2;
    if (tid < pairs) {
        const int64_t pos = r.positions ? ldp(r.positions + t) : place;
        const int64_t frac = int64_t(__ldg(reinterpret_cast<const unsigned long long *>(r.turns) + tid) * uint64_t(pos));
        float s, c;
        sincospif(__ll2float_rn(frac) * 0x1p-63f, &s, &c);  // half turns: 2 * frac / 2^64
        cs[tid] = make_float2(c * r.mscale, s * r.mscale);
    }
    __syncthreads();

    int64_t slot = -1;  // element offset of the token's slot of head 0, -1 if it has none
    if (place >= 0) {
        if (place < (int64_t)a.max_pages * a.page_size) {
            const int pi = place / a.page_size;
            const int page = ldp(a.table + (size_t)b * a.max_pages + pi);
            if (page >= 0 && page < a.n_pages)
                slot = page * a.page_stride + (int64_t)(place - pi * a.page_size) * a.token_stride;
        }
        if (slot < 0 && tid == 0) record_error(a.err, MOE_ERR_DEVICE);
    }

    const int chunk = tid % LG, d0 = chunk * 8, D = a.head_dim;
    const bool live = d0 < D;
    const int half = pairs / 8;  // chunks between the elements of a pair (half layout)
    const int heads = a.n_heads + 2 * a.n_kv_heads;
    for (int h0 = 0; h0 < heads; h0 += kThreads / LG) {
        const int h = h0 + tid / LG;
        const T *src = nullptr, *gamma = nullptr;
        T *dst = nullptr;
        bool rotate = true;
        if (live && h < a.n_heads) {
            src = static_cast<const T *>(a.q) + t * a.q_stride + (int64_t)h * D;
            dst = static_cast<T *>(a.out) + t * a.out_stride + (int64_t)h * D;
            gamma = static_cast<const T *>(r.gq);
        } else if (live && h < heads) {
            const bool is_v = h >= a.n_heads + a.n_kv_heads;
            const int kh = h - a.n_heads - (is_v ? a.n_kv_heads : 0);
            src = is_v ? static_cast<const T *>(r.v_in) + t * r.v_stride + (int64_t)kh * D
                       : static_cast<const T *>(r.k_in) + t * r.k_stride + (int64_t)kh * D;
            T *base = static_cast<T *>(const_cast<void *>(is_v ? a.v : a.k));
            dst = slot < 0 ? nullptr : base + slot + (int64_t)kh * a.head_stride;
            gamma = is_v ? nullptr : static_cast<const T *>(r.gk);
            rotate = !is_v;
        }
        float x[8] = {};
        if (src) attn::ldp8(src + d0, x);
        if (r.gq || r.gk) {  // every lane takes part in the shuffles
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (gamma) {
                const float rs = rsqrtf(ss / float(D) + r.eps);
                float g[8];
                attn::ldp8(gamma + d0, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * g[i];
            }
        }
        if (r.interleaved) {
            if (rotate && d0 < r.rot_dim) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 c = cs[d0 / 2 + i];
                    const float u = x[2 * i], w = x[2 * i + 1];
                    x[2 * i] = u * c.x - w * c.y;
                    x[2 * i + 1] = w * c.x + u * c.y;
                }
            }
        } else {
            const bool first = chunk < half;
            const int other = first ? chunk + half : chunk - half;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], other & (LG - 1), LG);
            if (rotate && d0 < r.rot_dim) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 c = cs[(first ? d0 : d0 - pairs) + i];
                    x[i] = first ? x[i] * c.x - y[i] * c.y : x[i] * c.x + y[i] * c.y;
                }
            }
        }
        if (dst) attn::store8(dst + d0, x);
    }
}

template <typename T>
cudaError_t launch_typed(const RopeArgs &r, cudaStream_t st) {
    const int chunks = r.a.head_dim / 8;
    const dim3 grid(r.a.n_tokens), block(kThreads);
    if (chunks <= 2) return launch_pdl(rope_kernel<T, 2>, grid, block, 0, st, r);
    if (chunks <= 4) return launch_pdl(rope_kernel<T, 4>, grid, block, 0, st, r);
    if (chunks <= 8) return launch_pdl(rope_kernel<T, 8>, grid, block, 0, st, r);
    if (chunks <= 16) return launch_pdl(rope_kernel<T, 16>, grid, block, 0, st, r);
    return launch_pdl(rope_kernel<T, 32>, grid, block, 0, st, r);
}

}  // namespace

cudaError_t launch_rope(const moe_attn_shape &s, const moe_rope &rp, const attn::Args &a, const void *k,
                        int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions, cudaStream_t st) {
    RopeArgs r{a, k, v, k_stride, v_stride, positions, rp.turns, rp.q_gamma, rp.k_gamma, rp.rot_dim, rp.interleaved,
               rp.mscale, rp.eps};
    return s.dtype == MOE_DT_F32 ? launch_typed<float>(r, st) : launch_typed<uint16_t>(r, st);
}

}  // namespace moe
