// rope.cu -- rotary positions of the new tokens' q and k, with an optional RMS norm of each
// head before, and the write of k and v into the paged cache.  Memory bound: every element is
// read once and written once.
//
// A block works on one token, or on four when there are plenty: the cosines and sines of a
// token's rot_dim / 2 angles are found once and shared by all its heads.  An angle is
// (turns_i * position) mod 2^64 in units of 2^-64 turn, an exact integer product, so no far
// position costs accuracy, and no range reduction is needed: the signed fraction of a turn goes
// to sincospi.  The first rows are requested before the tokens' places and angles are known.
// A lane holds both elements of its pairs (two pieces of eight elements, half the rotated part
// apart), so that the rotation needs no exchange between lanes: one lane an eighth of a head
// with a shuffle per element ran at 0.32 of the copy rate, bound by its instructions.
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

// Eight elements as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = ldp16(p); }
    __device__ __forceinline__ void load_const(const uint16_t *p) { v = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float *f) const { attn::unpack8(v, f); }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = ldp16f(p);
        b = ldp16f(p + 4);
    }
    __device__ __forceinline__ void load_const(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p + 4));
    }
    __device__ __forceinline__ void get(float *f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

// A group of LG lanes (a power of two that covers head_dim / 16) holds one head, two pieces of
// eight elements a lane: lane l < rot_dim / 16 pieces l and l + rot_dim / 16, the others the
// pieces past the rotated part.  The block's groups go over the n_heads + 2 n_kv_heads heads of
// its TB tokens.
template <typename T, int LG, int TB>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs r) {
    __shared__ __align__(16) float2 cs[TB][kMaxPairs];
    __shared__ int seq[TB], where[TB];     // the tokens' sequences (-1: none) and places
    __shared__ int64_t slots[TB];          // element offset of a token's slot of head 0, -1 if it has none
    const attn::Args &a = r.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = tid % LG;
    const int D = a.head_dim, pairs = r.rot_dim / 2, half = pairs / 8;
    const bool turned = l < half;
    const int da = (turned ? l : 2 * l) * 8, db = (turned ? l + half : 2 * l + 1) * 8;  // the lane's elements
    const bool on_a = da < D, on_b = db < D;
    const int heads = a.n_heads + 2 * a.n_kv_heads, q_heads = a.n_heads, qk_heads = a.n_heads + a.n_kv_heads;
    const int t0 = blockIdx.x * TB, tokens = min(TB, a.n_tokens - t0);
    constexpr int kGroups = kThreads / LG;

    // weights: no kernel of the library writes them
    constexpr int kTurns = (TB * kMaxPairs + kThreads - 1) / kThreads;
    uint64_t turn[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int at = tid + i * kThreads;
        if (at < TB * pairs) turn[i] = __ldg(reinterpret_cast<const unsigned long long *>(r.turns) + at % pairs);
    }
    griddep_wait();
    griddep_launch_dependents();

    Raw<T> xa, xb, na, nb;
    auto load = [&](int tk, int h) {
        if (tk >= tokens) return;
        const int64_t t = t0 + tk;
        const T *src = h < q_heads    ? static_cast<const T *>(a.q) + t * a.q_stride + h * D
                       : h < qk_heads ? static_cast<const T *>(r.k_in) + t * r.k_stride + (h - q_heads) * D
                                      : static_cast<const T *>(r.v_in) + t * r.v_stride + (h - qk_heads) * D;
        if (on_a) na.load(src + da);
        if (on_b) nb.load(src + db);
    };
    int tk = 0, h = tid / LG;
    auto next = [&](int &k, int &g) {
        for (g += kGroups; g >= heads; g -= heads) ++k;
    };
    for (; h >= heads; h -= heads) ++tk;
    load(tk, h);

    auto angles = [&](int i, int at, int k, int64_t pos) {
        float s, c;
        sincospif(__ll2float_rn(int64_t(turn[i] * uint64_t(pos))) * 0x1p-63f, &s, &c);  // half turns: 2 * frac / 2^64
        cs[k][at - k * pairs] = make_float2(c * r.mscale, s * r.mscale);
    };
    int32_t given[kTurns];
    if (r.positions) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int at = tid + i * kThreads;
            if (at < tokens * pairs) given[i] = ldp(r.positions + t0 + at / pairs);
        }
    }

    // places: the sequence b with cu_q[b] <= t < cu_q[b + 1]; cu_q rises, so one b matches
    if (tid < TB) seq[tid] = -1;
    __syncthreads();
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const int c0 = ldp(a.cu_q + b), c1 = ldp(a.cu_q + b + 1), kv = ldp(a.kv_len + b);
        if (blockIdx.x == 0 && (c0 < 0 || c1 < c0 || c1 > a.n_tokens)) record_error(a.err, MOE_ERR_DEVICE);
        if (c0 < t0 + tokens && c1 > t0) {
#pragma unroll
            for (int i = 0; i < TB; ++i)
                if (c0 <= t0 + i && t0 + i < c1) {
                    seq[i] = b;
                    where[i] = kv - (c1 - t0 - i);
                }
        }
    }
    if (r.positions) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int at = tid + i * kThreads;
            if (at < tokens * pairs) angles(i, at, at / pairs, given[i]);
        }
    }
    __syncthreads();
    if (warp == kThreads / 32 - 1 && lane < tokens && seq[lane] >= 0) {
        const int place = where[lane];
        int64_t slot = -1;
        if (place >= 0) {
            if (place < (int64_t)a.max_pages * a.page_size) {
                const int pi = place / a.page_size;
                const int page = ldp(a.table + (size_t)seq[lane] * a.max_pages + pi);
                if (page >= 0 && page < a.n_pages)
                    slot = page * a.page_stride + (int64_t)(place - pi * a.page_size) * a.token_stride;
            }
            if (slot < 0) record_error(a.err, MOE_ERR_DEVICE);
        }
        slots[lane] = slot;
    }
    if (!r.positions) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int at = tid + i * kThreads, k = at / pairs;
            if (at < tokens * pairs && seq[k] >= 0) angles(i, at, k, where[k]);
        }
    }
    __syncthreads();

    const float inv_d = 1.f / float(D);
    const bool norm = r.gq || r.gk;
    // every group makes the same number of turns: all lanes take part in the shuffles
    for (int left = (tokens * heads + kGroups - 1) / kGroups; left > 0; --left) {
        xa = na;
        xb = nb;
        int tk2 = tk, h2 = h;
        next(tk2, h2);
        load(tk2, h2);
        const bool on = tk < tokens && seq[tk < tokens ? tk : 0] >= 0;
        const bool is_q = h < q_heads, is_v = h >= qk_heads;
        float f[16] = {};
        if (on && on_a) xa.get(f);
        if (on && on_b) xb.get(f + 8);
        if (norm) {
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s0 = fmaf(f[e], f[e], s0);
                s1 = fmaf(f[8 + e], f[8 + e], s1);
            }
            float ss = s0 + s1;
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float rs = rsqrtf(ss * inv_d + r.eps);
            const T *gamma = static_cast<const T *>(is_q ? r.gq : is_v ? nullptr : r.gk);
            if (gamma) {
                float g[8];
                Raw<T> w;
                if (on_a) {
                    w.load_const(gamma + da);
                    w.get(g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = f[e] * rs * g[e];
                }
                if (on_b) {
                    w.load_const(gamma + db);
                    w.get(g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[8 + e] = f[8 + e] * rs * g[e];
                }
            }
        }
        if (turned && !is_v) {
            const float2 *ct = cs[tk < tokens ? tk : 0];
            if (r.interleaved) {  // pairs da / 2 .. + 3 and db / 2 .. + 3
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 c = *reinterpret_cast<const float4 *>(ct + ((e < 8 ? da : db) + (e & 7)) / 2);
                    const float u0 = f[e], w0 = f[e + 1], u1 = f[e + 2], w1 = f[e + 3];
                    f[e] = u0 * c.x - w0 * c.y;
                    f[e + 1] = w0 * c.x + u0 * c.y;
                    f[e + 2] = u1 * c.z - w1 * c.w;
                    f[e + 3] = w1 * c.z + u1 * c.w;
                }
            } else {  // element da + e pairs with db + e
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float4 c = *reinterpret_cast<const float4 *>(ct + da + e);
                    const float u0 = f[e], w0 = f[8 + e], u1 = f[e + 1], w1 = f[9 + e];
                    f[e] = u0 * c.x - w0 * c.y;
                    f[8 + e] = w0 * c.x + u0 * c.y;
                    f[e + 1] = u1 * c.z - w1 * c.w;
                    f[9 + e] = w1 * c.z + u1 * c.w;
                }
            }
        }
        T *dst = nullptr;
        if (on) {
            if (is_q)
                dst = static_cast<T *>(a.out) + (int64_t)(t0 + tk) * a.out_stride + h * D;
            else if (slots[tk] >= 0)
                dst = static_cast<T *>(const_cast<void *>(is_v ? a.v : a.k)) + slots[tk] +
                      (int64_t)(is_v ? h - qk_heads : h - q_heads) * a.head_stride;
        }
        if (dst && on_a) attn::store8(dst + da, f);
        if (dst && on_b) attn::store8(dst + db, f + 8);
        tk = tk2;
        h = h2;
    }
}

template <typename T, int LG>
cudaError_t launch_tokens(const RopeArgs &r, cudaStream_t st) {
    // four tokens a block once that leaves a block on each SM: 4043 tokens of 40 heads take 22.2 us
    // (one a block: 33.5), 1583 of 18 heads in fp32 7.4 us (10.5); 8 tokens 6.4 us (one: 4.3)
    if (r.a.n_tokens >= 4 * 152)
        return launch_pdl(rope_kernel<T, LG, 4>, dim3((r.a.n_tokens + 3) / 4), dim3(kThreads), 0, st, r);
    return launch_pdl(rope_kernel<T, LG, 1>, dim3(r.a.n_tokens), dim3(kThreads), 0, st, r);
}

template <typename T>
cudaError_t launch_typed(const RopeArgs &r, cudaStream_t st) {
    const int d = r.a.head_dim;
    if (d <= 16) return launch_tokens<T, 1>(r, st);
    if (d <= 32) return launch_tokens<T, 2>(r, st);
    if (d <= 64) return launch_tokens<T, 4>(r, st);
    if (d <= 128) return launch_tokens<T, 8>(r, st);
    return launch_tokens<T, 16>(r, st);
}

}  // namespace

cudaError_t launch_rope(const moe_attn_shape &s, const moe_rope &rp, const attn::Args &a, const void *k,
                        int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions, cudaStream_t st) {
    RopeArgs r{a, k, v, k_stride, v_stride, positions, rp.turns, rp.q_gamma, rp.k_gamma, rp.rot_dim, rp.interleaved,
               rp.mscale, rp.eps};
    return s.dtype == MOE_DT_F32 ? launch_typed<float>(r, st) : launch_typed<uint16_t>(r, st);
}

}  // namespace moe
