// rope_q8.cu -- rotary positions of the new tokens' q and k, with an optional RMS norm of each head
// before, and the write of k and v into a paged cache of 8-bit values.
//
// A block of tokens shares a power of two a head: 2^e with e the smallest that keeps the block's
// largest value within 448.  The first new token of a sequence may fall into a block that holds old
// ones: if the new values need a larger scale, the old codes move down with it (their exponents
// shift; what falls below 2^-9 of the scale is rounded).
//
// One launch, two kinds of blocks of threads.  The first write k and v: a task is one head's k or v
// over one block of tokens.  Its warps keep the rotated values in shared memory while they agree on the
// largest, and then store the codes: k and v are read once.  (In registers, four tokens a lane, the kernel took
// 184 of them, and q's blocks waited for one another: 4043 tokens 44 us; two tokens a lane 28.)  The
// others rotate q, a token, four or sixteen at a time, and share a token's cosines and sines between its heads.
// 4043 tokens, 32 + 4 heads of 128 with a norm: 21 us on the GPU (the bytes alone 11.7), 14.7 for q alone and 10.7 for k and v.  The bound
// is latency: instructions (67 for a row of q of 128 elements) take 0.48 of the issue slots, in chains that 13.6 warps an SM do not
// cover.  One launch gives q's blocks, with one row in flight a group of lanes, the shared memory of k's and v's (two blocks an SM) and the
// registers of the larger part (113).  8 tokens: 3.6 us, latency.
#include "q8.cuh"
#include "rope.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;
constexpr int kMostKept = 64 << 10;  // bytes of shared memory for the values of a block of threads

struct Q8Args {
    RopeArgs r;
    uint8_t *k_scale, *v_scale;
    int64_t scale_page, scale_head;
    int32_t block;       // tokens of a scale
    int32_t warps;       // of a task
    int32_t groups;      // blocks of threads a block of tokens
    int32_t kv_blocks;   // blocks of threads that store k and v
    int32_t hold;        // tokens of a task that shared memory holds (0: they are worked out twice)
};

// What a lane of a group of LG lanes holds of a head: pieces of eight elements at da and db.
struct LaneOf {
    int D, da, db;
    bool turned, on_a, on_b;
    __device__ __forceinline__ LaneOf(const RopeArgs &r, int l) {
        D = r.a.head_dim;
        const int half = r.rot_dim / 16;
        turned = l < half;
        da = (turned ? l : 2 * l) * 8;
        db = (turned ? l + half : 2 * l + 1) * 8;
        on_a = da < D;
        on_b = db < D;
    }
    // the pair whose cosine is the first of c[e] (each c[e] holds two neighbours)
    __device__ __forceinline__ int pair_of(int e, bool interleaved) const {
        return interleaved ? (e < 2 ? da : db) / 2 + 2 * (e & 1) : da + 2 * e;
    }
};

// The lane's weights of a norm, as pairs like the values.
template <typename T>
__device__ __forceinline__ void load_gamma(uint64_t *g, const T *gamma, const LaneOf &at) {
    Raw<T> w;
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = 0;
    if (!gamma) return;
    if (at.on_a) {
        w.load_cached(gamma + at.da);
        w.get(g);
    }
    if (at.on_b) {
        w.load_cached(gamma + at.db);
        w.get(g + 4);
    }
}

// f[0..3], f[4..7]: the two pieces, as pairs of neighbouring elements.
template <int LG>
__device__ __forceinline__ void norm(uint64_t *f, const uint64_t *g, float inv_d, float eps) {
    uint64_t s2 = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) s2 = attn::fma2(f[e], f[e], s2);
    float lo, hi;
    attn::unpair(s2, lo, hi);
    float ss = lo + hi;
#pragma unroll
    for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rs = rsqrtf(ss * inv_d + eps);
    const uint64_t rs2 = attn::pair(rs, rs);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = attn::mul2(attn::mul2(f[e], rs2), g[e]);
}

__device__ __forceinline__ void rotate(uint64_t *f, const uint64_t *c, const uint64_t *s, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float c0, c1, s0, s1, u, w;
            attn::unpair(c[e / 2], c0, c1);
            attn::unpair(s[e / 2], s0, s1);
            attn::unpair(f[e], u, w);
            const float ce = e & 1 ? c1 : c0, se = e & 1 ? s1 : s0;
            f[e] = attn::pair(u * ce - w * se, w * ce + u * se);
        }
    } else {
        const uint64_t minus = attn::pair(-1.f, -1.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t u = f[e], w = f[4 + e];
            f[e] = attn::fma2(w, attn::mul2(s[e], minus), attn::mul2(u, c[e]));
            f[4 + e] = attn::fma2(u, s[e], attn::mul2(w, c[e]));
        }
    }
}

// The angle's cosine and sine times mscale.  turn * pos modulo 2^64 is the fraction of a turn in units of 2^-64,
// exact at every position; its upper half (pos as a signed number), in units of 2^-32 turn, is off by 1.5e-9
// radians at most.  Beside that fp32 rounds the angle, as it does in the append to a 16-bit cache: by up to 9.4e-8
// radians next to half a turn.
__device__ __forceinline__ void angle(uint64_t turn, int pos, float mscale, float &c, float &s) {
    const uint32_t lo = uint32_t(turn), hi = uint32_t(turn >> 32), p = uint32_t(pos);
    const uint32_t part = hi * p + __umulhi(lo, p) - (pos < 0 ? lo : 0u);
    sincospif(__int2float_rn(int(part)) * 0x1p-31f, &s, &c);  // half turns
    c *= mscale;
    s *= mscale;
}
__device__ __forceinline__ uint64_t ldp_turn(const uint64_t *p) {
    uint64_t v;
    asm volatile("ld.global.u64 %0, [%1];" : "=l"(v) : "l"(p));
    return v;
}

// One block of tokens of one sequence, as far as the call writes it.
struct Piece {
    int b, start;   // the sequence, the block's first place
    int lo, hi;     // places that the call writes, within the block
    int row;        // the row of the token at place lo
    int first;      // the chunk's first place (negative: its first tokens have none)
};

struct SeqSpan {
    int c0, first, p0, p1, count;
};
// How many blocks of tokens sequence b's chunk touches, and where.
__device__ __forceinline__ SeqSpan span_of(const attn::Args &a, int b, int block) {
    const int c0 = min(max(ldp(a.cu_q + b), 0), a.n_tokens), c1 = min(max(ldp(a.cu_q + b + 1), 0), a.n_tokens);
    const int kv = max(ldp(a.kv_len + b), 0), n = max(c1 - c0, 0);
    SeqSpan s;
    s.c0 = c0;
    s.first = kv - n;
    s.p0 = max(s.first, 0);
    s.p1 = int(min((int64_t)kv, (int64_t)a.max_pages * a.page_size));  // places past the table are not stored
    s.count = s.p1 > s.p0 && n > 0 ? (s.p1 - 1) / block - s.p0 / block + 1 : 0;
    return s;
}

// Piece number `at` of the batch; b = -1 past the last.  Every thread of the block calls it.
__device__ __forceinline__ Piece find_piece(const attn::Args &a, int at, int block, int *scratch) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto piece = [&](int b, int i, const SeqSpan &s) {
        Piece p;
        p.b = b;
        p.start = (s.p0 / block + i) * block;
        p.lo = max(p.start, s.p0);
        p.hi = min(s.p1 - p.start, block) + p.start;
        p.row = s.c0 + (p.lo - s.first);
        p.first = s.first;
        return p;
    };
    auto scan = [&](int n) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += u;
        }
        return n;
    };
    if (a.n_seqs <= 32) {  // every warp for itself, without barriers
        SeqSpan s{};
        if (lane < a.n_seqs) s = span_of(a, lane, block);
        const int incl = scan(s.count);
        const int b = __ffs(__ballot_sync(0xffffffffu, at < incl)) - 1, src = max(b, 0);
        const int i = at - __shfl_sync(0xffffffffu, incl - s.count, src);
        s.c0 = __shfl_sync(0xffffffffu, s.c0, src);
        s.first = __shfl_sync(0xffffffffu, s.first, src);
        s.p0 = __shfl_sync(0xffffffffu, s.p0, src);
        s.p1 = __shfl_sync(0xffffffffu, s.p1, src);
        return b < 0 ? Piece{-1, 0, 0, 0, 0, 0} : piece(b, i, s);
    }
    if (tid == 0) scratch[0] = -1;
    int base = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
        const int n = b0 + tid < a.n_seqs ? span_of(a, b0 + tid, block).count : 0, incl = scan(n);
        __syncthreads();
        if (lane == 31) scratch[2 + warp] = incl;
        __syncthreads();
        int before = base, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? scratch[2 + w] : 0;
            total += scratch[2 + w];
        }
        before += incl - n;
        if (at >= before && at - before < n) {
            scratch[0] = b0 + tid;
            scratch[1] = at - before;
        }
        base += total;
        if (at < base) break;  // base is the same for every thread
    }
    __syncthreads();
    const int b = scratch[0];
    return b < 0 ? Piece{-1, 0, 0, 0, 0, 0} : piece(b, scratch[1], span_of(a, b, block));
}

// The smallest e with top <= 448 2^e (448 = 1.75 * 2^8), kept within the range that is written.
__device__ __forceinline__ int exponent_of(float top) {
    const uint32_t u = __float_as_uint(top);
    const int e = int(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return top > 0.f ? min(max(e, q8::kLowest), q8::kHighest) : q8::kLowest;
}

template <typename T, int LG>
__device__ __forceinline__ void store_kv(const Q8Args &c) {
    constexpr int RPW = 32 / LG;  // tokens a warp works on at a time
    extern __shared__ float4 kept[];
    __shared__ int scratch[2 + kWarps];
    __shared__ uint32_t tops[kWarps];
    const RopeArgs &r = c.r;
    const attn::Args &a = r.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const LaneOf at(r, lane % LG);
    const Piece p = find_piece(a, blockIdx.x / c.groups, c.block, scratch);
    if (p.b < 0) return;  // the whole block
    const int W = c.warps, sub = warp & (W - 1), task = int(blockIdx.x % c.groups) * (kWarps / W) + warp / W;
    const bool on = task < 2 * a.n_kv_heads, is_v = task >= a.n_kv_heads;
    const int h = is_v ? task - a.n_kv_heads : task, n = p.hi - p.lo, old = p.lo - p.start;
    const int t0 = sub * RPW + lane / LG, stride_t = W * RPW;  // the lane's tokens of the piece: t0, t0 + stride_t, ..
    const int64_t row_stride = is_v ? r.v_stride : r.k_stride;
    const T *src = static_cast<const T *>(is_v ? r.v_in : r.k_in) + p.row * row_stride + h * at.D;
    const T *gamma = is_v ? nullptr : static_cast<const T *>(r.gk);
    const bool turn = !is_v && at.turned, held = n <= c.hold;
    const float inv_d = 1.f / float(at.D);
    // a lane's 16 values of a token lie lanes apart, so that a warp's stores and loads meet no bank twice
    float4 *mine = kept + (size_t)(warp / W) * c.hold * (LG * 4) + lane % LG;

    Raw<T> na, nb;
    auto load = [&](int t) {
        if (on && t < n) {
            if (at.on_a) na.load(src + t * row_stride + at.da);
            if (at.on_b) nb.load(src + t * row_stride + at.db);
        }
    };
    uint64_t turns[8];
    // token t's values: normed, rotated; an infinity becomes NaN (x + 0 x), which the maximum passes over and the
    // codes keep
    auto work = [&](int t, uint64_t *f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0;
        if (on && t < n) {
            if (at.on_a) na.get(f);
            if (at.on_b) nb.get(f + 4);
        }
        load(t + stride_t);
        if (gamma) {
            uint64_t g[8];
            load_gamma(g, gamma, at);
            norm<LG>(f, g, inv_d, r.eps);
        }
        if (turn && on && t < n) {
            const int pos = r.positions ? ldp(r.positions + p.row + t) : p.lo + t;
            uint64_t co[4], si[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float c0, c1, s0, s1;
                angle(turns[2 * e], pos, r.mscale, c0, s0);
                angle(turns[2 * e + 1], pos, r.mscale, c1, s1);
                co[e] = attn::pair(c0, c1);
                si[e] = attn::pair(s0, s1);
            }
            rotate(f, co, si, r.interleaved);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = attn::fma2(f[e], 0, f[e]);
    };
    load(t0);
    if (turn) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = at.pair_of(e, r.interleaved);
            turns[2 * e] = ldp_turn(r.turns + i);
            turns[2 * e + 1] = ldp_turn(r.turns + i + 1);
        }
    }
    const int pi = p.start / a.page_size, slot = p.start - pi * a.page_size;
    const int page = ldp(a.table + (size_t)p.b * a.max_pages + pi);

    uint32_t top = 0;  // the bits of the largest size: those of numbers of one sign are in the numbers' order
    for (int t = t0; t - lane / LG < n; t += stride_t) {
        uint64_t f[8];
        work(t, f);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float x, y;
            attn::unpair(f[e], x, y);
            m = fmaxf(m, fmaxf(fabsf(x), fabsf(y)));
        }
        top = max(top, __float_as_uint(m));
        if (held && t < n) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                float4 v;
                attn::unpair(f[e], v.x, v.y);
                attn::unpair(f[e + 1], v.z, v.w);
                mine[(t * 4 + e / 2) * LG] = v;
            }
        }
    }
    const bool page_ok = page >= 0 && page < a.n_pages;
    if (!page_ok && tid == 0) record_error(a.err, MOE_ERR_DEVICE);
    uint8_t *dst = static_cast<uint8_t *>(const_cast<void *>(is_v ? a.v : a.k)) + (page_ok ? page : 0) * a.page_stride +
                   h * a.head_stride + slot * a.token_stride;
    uint8_t *scale = (is_v ? c.v_scale : c.k_scale) + (page_ok ? page : 0) * c.scale_page + h * c.scale_head + slot / c.block;
    const int was = on && page_ok && old > 0 ? int(q8::ldp_byte(scale)) - 127 : q8::kLowest;
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    for (int w = warp - sub; w < warp - sub + W; ++w) top = max(top, tops[w]);
    if (!on || !page_ok) return;
    const int e_new = exponent_of(__uint_as_float(top)), e = old > 0 ? max(e_new, was) : e_new;

    if (old > 0 && e > was) {  // the old codes in units of the larger scale
        const int chunks = at.D / 16;
        const __half f16 = __float2half(q8::scale_of(uint32_t(max(127 + was - e, 1))));
        const __half2 down = __half2half2(f16);
        for (int i = sub * 32 + lane; i < old * chunks; i += W * 32) {
            uint8_t *q = dst + (i / chunks) * a.token_stride + (i % chunks) * 16;
            uint4 w = ldp16(q);
            uint32_t *x = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t lo, hi;
                q8::to_f16x4(x[j], lo, hi);
                const __half2 a0 = __hmul2(*reinterpret_cast<const __half2 *>(&lo), down);
                const __half2 a1 = __hmul2(*reinterpret_cast<const __half2 *>(&hi), down);
                x[j] = q8::from_f16x2(*reinterpret_cast<const uint32_t *>(&a0)) |
                       q8::from_f16x2(*reinterpret_cast<const uint32_t *>(&a1)) << 16;
            }
            *reinterpret_cast<uint4 *>(q) = w;
        }
    }
    if (sub == 0 && lane == 0) *scale = uint8_t(e + 127);
    const float up = q8::scale_of(uint32_t(min(max(127 - e, 0), 254)));
    const uint64_t up2 = attn::pair(up, up);
    dst += old * a.token_stride;
    if (!held) load(t0);
    for (int t = t0; t - lane / LG < n; t += stride_t) {
        uint64_t f[8];
        if (held) {
            if (t >= n) break;  // no shuffles here
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float4 v = mine[(t * 4 + e / 2) * LG];
                f[e] = attn::pair(v.x, v.y);
                f[e + 1] = attn::pair(v.z, v.w);
            }
        } else {
            work(t, f);
        }
        if (t >= n) continue;
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float x, y;
            attn::unpair(attn::mul2(f[k], up2), x, y);
            w[k] = q8::from_f32(x, y);
        }
        uint8_t *to = dst + t * a.token_stride;
        if (at.on_a) *reinterpret_cast<uint2 *>(to + at.da) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        if (at.on_b) *reinterpret_cast<uint2 *>(to + at.db) = make_uint2(w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}

template <typename T, int LG, int TB>
__device__ __forceinline__ void turn_q(const Q8Args &c) {
    __shared__ float4 cs[TB][kMaxPairs / 2];  // (cos, cos, sin, sin) of two pairs at place_of(pair / 2)
    __shared__ int seq[TB], where[TB];        // the tokens' sequences (-1: none) and places
    const RopeArgs &r = c.r;
    const attn::Args &a = r.a;
    const int tid = threadIdx.x, t0 = (int(blockIdx.x) - c.kv_blocks) * TB, tokens = min(TB, a.n_tokens - t0);
    const int pairs = r.rot_dim / 2, heads = a.n_heads;
    const LaneOf at(r, tid % LG);
    constexpr int kGroups = kThreads / LG;
    // a thread's pair in every token whose angles it finds: 32, 64 or 128 threads a token
    const int shift = pairs <= 32 ? 5 : pairs <= 64 ? 6 : 7, pair = tid & ((1 << shift) - 1);
    uint64_t turn = 0;
    if (pair < pairs) turn = ldp_turn(r.turns + pair);
    // a group takes heads group, group + kGroups, .. of the block's tokens; the next is requested ahead
    int tk = 0, h = tid / LG;
    auto settle = [&]() {
        for (; h >= heads; h -= heads) ++tk;
    };
    settle();
    Raw<T> na, nb;
    const T *q_in = static_cast<const T *>(a.q) + (int64_t)t0 * a.q_stride;
    T *out = static_cast<T *>(a.out) + (int64_t)t0 * a.out_stride;
    const int q_row = int(a.q_stride), out_row = int(a.out_stride);
    auto load = [&]() {
        if (tk < tokens) {
            const T *src = q_in + (int64_t)tk * q_row + h * at.D;
            if (at.on_a) na.load(src + at.da);
            if (at.on_b) nb.load(src + at.db);
        }
    };
    load();
    if (tid < TB) seq[tid] = -1;
    __syncthreads();
    for (int b = tid; b < a.n_seqs; b += kThreads) {
        const int c0 = ldp(a.cu_q + b), c1 = ldp(a.cu_q + b + 1), kv = ldp(a.kv_len + b);
        if (t0 == 0 && (c0 < 0 || c1 < c0 || c1 > a.n_tokens || c1 - c0 > a.max_q || kv < 0 ||
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
    __syncthreads();
    for (int k = tid >> shift; k < tokens; k += kThreads >> shift)
        if (pair < pairs && seq[k] >= 0) {
            float co, si;
            angle(turn, r.positions ? ldp(r.positions + t0 + k) : where[k], r.mscale, co, si);
            float *to = reinterpret_cast<float *>(&cs[k][place_of(pair >> 1)]) + (pair & 1);
            to[0] = co;
            to[2] = si;
        }
    __syncthreads();
    const float inv_d = 1.f / float(at.D);
    uint64_t gq[8];
    load_gamma(gq, static_cast<const T *>(r.gq), at);
    for (int left = (tokens * heads + kGroups - 1) / kGroups; left > 0; --left) {
        const int k = tk < tokens ? tk : 0;
        const bool on = tk < tokens && seq[k] >= 0;
        T *dst = out + (int64_t)k * out_row + h * at.D;
        uint64_t f[8] = {};
        if (on && at.on_a) na.get(f);
        if (on && at.on_b) nb.get(f + 4);
        h += kGroups;
        settle();
        if (left > 1) load();
        if (r.gq) norm<LG>(f, gq, inv_d, r.eps);
        if (at.turned) {
            uint64_t co[4], si[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v = cs[k][place_of(at.pair_of(e, r.interleaved) >> 1)];
                co[e] = attn::pair(v.x, v.y);
                si[e] = attn::pair(v.z, v.w);
            }
            rotate(f, co, si, r.interleaved);
        }
        float y[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) attn::unpair(f[e], y[2 * e], y[2 * e + 1]);
        if (on && at.on_a) attn::store8(dst + at.da, y);
        if (on && at.on_b) attn::store8(dst + at.db, y + 8);
    }
}

template <typename T, int LG, int TB>
__global__ void __launch_bounds__(kThreads, 2) rope_q8_kernel(const __grid_constant__ Q8Args c) {
    // the table and the norms' weights too may be what the kernel before this one writes
    griddep_wait();
    griddep_launch_dependents();
    if (int(blockIdx.x) < c.kv_blocks)
        store_kv<T, LG>(c);
    else
        turn_q<T, LG, TB>(c);
}

template <typename T, int LG, int TB>
cudaError_t launch_tokens(const Q8Args &c, int64_t grid, size_t smem, cudaStream_t st) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(rope_q8_kernel<T, LG, TB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKept);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    return launch_pdl(rope_q8_kernel<T, LG, TB>, dim3(unsigned(grid)), dim3(kThreads), smem, st, c);
}

template <typename T, int LG>
cudaError_t launch_lanes(Q8Args &c, const moe_attn_shape &s, cudaStream_t st) {
    constexpr int RPW = 32 / LG;
    // as many warps a task as leave each at least four turns on the new tokens of a block (one for every token it
    // works on at once: 4043 tokens 21.1 us, most of it the start of 8 x 552 warps)
    const int most = std::max(std::min(c.block, s.max_q), 1);
    for (c.warps = 1; c.warps < kWarps && c.warps * RPW * 4 < most;) c.warps *= 2;
    c.groups = (2 * s.n_kv_heads * c.warps + kWarps - 1) / kWarps;
    size_t smem = (size_t)(kWarps / c.warps) * most * LG * 64;
    c.hold = most;
    if (smem > kMostKept) c.hold = 0, smem = 0;
    // blocks of tokens that the chunks can touch: the host knows how many tokens and sequences there are
    const int64_t pieces = std::min<int64_t>(s.n_tokens, (int64_t)s.n_tokens / c.block + 2 * (int64_t)s.n_seqs);
    // tokens of a block that rotates q: more for fewer starts once that leaves a block on each SM
    const int tb = s.n_tokens >= 16 * 152 ? 16 : s.n_tokens >= 4 * 152 ? 4 : 1;
    const int64_t grid = pieces * c.groups + (s.n_tokens + tb - 1) / tb;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    c.kv_blocks = int(pieces * c.groups);
    if (tb == 16) return launch_tokens<T, LG, 16>(c, grid, smem, st);
    return tb == 4 ? launch_tokens<T, LG, 4>(c, grid, smem, st) : launch_tokens<T, LG, 1>(c, grid, smem, st);
}

template <typename T>
cudaError_t launch_typed(Q8Args &c, const moe_attn_shape &s, cudaStream_t st) {
    if (s.head_dim <= 16) return launch_lanes<T, 1>(c, s, st);
    if (s.head_dim <= 32) return launch_lanes<T, 2>(c, s, st);
    if (s.head_dim <= 64) return launch_lanes<T, 4>(c, s, st);
    if (s.head_dim <= 128) return launch_lanes<T, 8>(c, s, st);
    return launch_lanes<T, 16>(c, s, st);
}

}  // namespace

cudaError_t launch_rope_q8(const moe_attn_shape &s, const moe_rope &rp, const attn::Args &a, const moe_kv_cache_q8 &cache,
                           const void *k, int64_t k_stride, const void *v, int64_t v_stride, const int32_t *positions,
                           cudaStream_t st) {
    Q8Args c{};
    c.r = RopeArgs{a, k, v, k_stride, v_stride, positions, rp.turns, rp.q_gamma, rp.k_gamma, rp.rot_dim, rp.interleaved,
                   rp.mscale, rp.eps};
    c.k_scale = static_cast<uint8_t *>(cache.k_scale);
    c.v_scale = static_cast<uint8_t *>(cache.v_scale);
    c.scale_page = cache.scale_page_stride;
    c.scale_head = cache.scale_head_stride;
    c.block = cache.block;
    return s.dtype == MOE_DT_F32 ? launch_typed<float>(c, s, st) : launch_typed<uint16_t>(c, s, st);
}

}  // namespace moe
