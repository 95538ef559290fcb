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
#include "rope.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

// A group of LG lanes (a power of two that covers head_dim / 16) holds one head, two pieces of
// eight elements a lane: lane l < rot_dim / 16 pieces l and l + rot_dim / 16, the others the
// pieces past the rotated part.  The block's groups go over the n_heads + 2 n_kv_heads heads of
// its TB tokens.
template <typename T, int LG, int TB>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs r) {
    __shared__ float4 cs[TB][kMaxPairs / 2];  // (cos, cos, sin, sin) of two pairs at place_of(pair / 2)
    __shared__ int seq[TB], where[TB];     // the tokens' sequences (-1: none) and places
    __shared__ int64_t slots[TB];          // element offset of a token's slot of head 0, -1 if it has none
    const attn::Args &a = r.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, l = tid % LG;
    const int D = a.head_dim, pairs = r.rot_dim / 2, half = pairs / 8;
    const bool turned = l < half;
    const int da = (turned ? l : 2 * l) * 8, db = (turned ? l + half : 2 * l + 1) * 8;  // the lane's elements
    const bool on_a = da < D, on_b = db < D;
    const int q_heads = a.n_heads;
    const int t0 = blockIdx.x * TB, tokens = min(TB, a.n_tokens - t0);
    constexpr int kGroups = kThreads / LG;

    // the table and the norms' weights too may be what the kernel before this one writes
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kTurns = (TB * kMaxPairs + kThreads - 1) / kThreads;
    uint64_t turn[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int at = tid + i * kThreads;
        if (at < TB * pairs) turn[i] = r.turns[at % pairs];
    }

    // Row i of the block: first the tokens' q heads, then their k and v heads.  A group takes rows
    // group, group + kGroups, ..; its place among a token's heads moves on without a division.
    Raw<T> na, nb;
    struct At {
        int tk, h;
    };
    const int group = tid / LG;
    auto start = [&](int per_token) {
        At at{0, group};
        for (; at.h >= per_token; at.h -= per_token) ++at.tk;
        return at;
    };
    auto next = [&](At at, int per_token) {
        for (at.h += kGroups; at.h >= per_token; at.h -= per_token) ++at.tk;
        return at;
    };
    const int kv_heads = 2 * a.n_kv_heads;
    auto load = [&](const T *src) {
        if (on_a) na.load(src + da);
        if (on_b) nb.load(src + db);
    };
    const T *q_in = static_cast<const T *>(a.q) + (int64_t)t0 * a.q_stride;
    const T *k_in = static_cast<const T *>(r.k_in) + (int64_t)t0 * r.k_stride;
    const T *v_in = static_cast<const T *>(r.v_in) + (int64_t)t0 * r.v_stride;
    const int q_row = int(a.q_stride), k_row = int(r.k_stride), v_row = int(r.v_stride), out_row = int(a.out_stride);
    auto load_q = [&](At at) {
        if (at.tk < tokens) load(q_in + (int64_t)at.tk * q_row + at.h * D);
    };
    auto load_kv = [&](At at) {
        if (at.tk < tokens)
            load(at.h < a.n_kv_heads ? k_in + (int64_t)at.tk * k_row + at.h * D
                                     : v_in + (int64_t)at.tk * v_row + (at.h - a.n_kv_heads) * D);
    };
    At at_q = start(q_heads);
    load_q(at_q);

    auto angles = [&](int i, int at, int k, int64_t pos) {
        float s, c;
        sincospif(__ll2float_rn(int64_t(turn[i] * uint64_t(pos))) * 0x1p-63f, &s, &c);  // half turns: 2 * frac / 2^64
        const int p = at - k * pairs;
        float *to = reinterpret_cast<float *>(&cs[k][place_of(p >> 1)]) + (p & 1);
        to[0] = c * r.mscale;
        to[2] = s * r.mscale;
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
        if (blockIdx.x == 0 && (c0 < 0 || c1 < c0 || c1 > a.n_tokens || c1 - c0 > a.max_q || kv < 0 ||
                                kv > (int64_t)a.max_pages * a.page_size))
            record_error(a.err, MOE_ERR_DEVICE);
        if (c0 < t0 + tokens && c1 > t0) {
#pragma unroll
            for (int i = 0; i < TB; ++i)
                if (c0 <= t0 + i && t0 + i < c1) {
                    seq[i] = b;
                    where[i] = max(kv, 0) - (c1 - t0 - i);
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
    // One row: the norm (gamma not null), the rotation, the store.  All lanes take part.
    auto row = [&](bool on, const T *gamma, bool rotate, const float4 *ct, T *dst) {
        uint64_t f[8] = {};
        if (on && on_a) na.get(f);
        if (on && on_b) nb.get(f + 4);
        return [=]() mutable {
            if (r.gq || r.gk) {
                uint64_t s2 = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) s2 = attn::fma2(f[e], f[e], s2);
                float lo, hi;
                attn::unpair(s2, lo, hi);
                float ss = lo + hi;
#pragma unroll
                for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (gamma) {
                    const float rs = rsqrtf(ss * inv_d + r.eps);
                    const uint64_t rs2 = attn::pair(rs, rs);
                    uint64_t g[4];
                    Raw<T> w;
                    if (on_a) {
                        w.load_cached(gamma + da);
                        w.get(g);
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = attn::mul2(attn::mul2(f[e], rs2), g[e]);
                    }
                    if (on_b) {
                        w.load_cached(gamma + db);
                        w.get(g);
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[4 + e] = attn::mul2(attn::mul2(f[4 + e], rs2), g[e]);
                    }
                }
            }
            if (rotate) {
                const uint64_t minus = attn::pair(-1.f, -1.f);
                if (r.interleaved) {  // pairs da / 2 .. + 3 and db / 2 .. + 3
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float4 c = ct[place_of(((e < 4 ? da : db) + 2 * (e & 3)) / 4)];
                        float u0, w0, u1, w1;
                        attn::unpair(f[e], u0, w0);
                        attn::unpair(f[e + 1], u1, w1);
                        f[e] = attn::pair(u0 * c.x - w0 * c.z, w0 * c.x + u0 * c.z);
                        f[e + 1] = attn::pair(u1 * c.y - w1 * c.w, w1 * c.y + u1 * c.w);
                    }
                } else {  // element da + e pairs with db + e
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 c = ct[place_of(da / 2 + e)];
                        const uint64_t co = attn::pair(c.x, c.y), si = attn::pair(c.z, c.w), u = f[e], w = f[4 + e];
                        f[e] = attn::fma2(w, attn::mul2(si, minus), attn::mul2(u, co));
                        f[4 + e] = attn::fma2(u, si, attn::mul2(w, co));
                    }
                }
            }
            float y[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) attn::unpair(f[e], y[2 * e], y[2 * e + 1]);
            if (dst && on_a) attn::store8(dst + da, y);
            if (dst && on_b) attn::store8(dst + db, y + 8);
        };
    };
    // every group makes the same number of turns: all lanes take part in the shuffles.  The next row
    // is requested before a row is worked on.
    At at_kv = start(kv_heads);
    T *out = static_cast<T *>(a.out) + (int64_t)t0 * a.out_stride;
    for (int left = (tokens * q_heads + kGroups - 1) / kGroups; left > 0; --left) {
        const int tk = at_q.tk < tokens ? at_q.tk : 0;
        const bool on = at_q.tk < tokens && seq[tk] >= 0;
        auto work = row(on, static_cast<const T *>(r.gq), turned, cs[tk], on ? out + (int64_t)tk * out_row + at_q.h * D : nullptr);
        at_q = next(at_q, q_heads);
        if (left > 1)
            load_q(at_q);
        else
            load_kv(at_kv);
        work();
    }
    for (int left = (tokens * kv_heads + kGroups - 1) / kGroups; left > 0; --left) {
        const int tk = at_kv.tk < tokens ? at_kv.tk : 0;
        const bool on = at_kv.tk < tokens && seq[tk] >= 0, is_v = at_kv.h >= a.n_kv_heads;
        T *dst = nullptr;
        if (on && slots[tk] >= 0)
            dst = static_cast<T *>(const_cast<void *>(is_v ? a.v : a.k)) + slots[tk] +
                  (int64_t)(is_v ? at_kv.h - a.n_kv_heads : at_kv.h) * a.head_stride;
        auto work = row(on, static_cast<const T *>(is_v ? nullptr : r.gk), turned && !is_v, cs[tk], dst);
        at_kv = next(at_kv, kv_heads);
        if (left > 1) load_kv(at_kv);
        work();
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
