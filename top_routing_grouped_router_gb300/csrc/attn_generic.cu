// attn_generic.cu -- attention of new tokens over the paged cache on CUDA cores: any head
// size, page size and both dtypes, in fp32 throughout; and the join of partial results.
//
// softmax in one pass: for each key tile m' = max(m, max s), l = l e^(m-m') + sum e^(s-m'),
// o = o e^(m-m') + sum e^(s-m') v, with everything in log2 units so that e^ is exp2.
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 16;      // query rows (token, head of the group) of a block: 4 a warp
constexpr int kKeys = 32;      // keys of a tile: one a lane
constexpr int kMaxParts = 32;
constexpr int kTargetBlocks = 1216;  // eight blocks of four warps on each of 152 SMs

int tokens_per_tile(int group) { return group >= kRows ? 1 : kRows / group; }
// A group wider than a tile is split into head slices of kRows.
int head_slices(int group) { return (group + kRows - 1) / kRows; }

int64_t max_tiles(const moe_attn_shape &s) {
    const int tt = tokens_per_tile(s.n_heads / s.n_kv_heads);
    const int64_t full = (s.n_tokens + tt - 1) / tt;
    const int64_t ragged = full + s.n_seqs;  // each sequence's last tile may be part full
    return ragged < s.n_tokens ? ragged : s.n_tokens;  // a tile holds at least one token
}

// Parts that each tile's keys are split into: enough blocks for the machine, at least two key
// tiles a part of the longest sequence that the block table allows.
int parts(const moe_attn_shape &s) {
    const int64_t blocks = max_tiles(s) * s.n_kv_heads * head_slices(s.n_heads / s.n_kv_heads);
    const int64_t keys = (int64_t)s.max_pages * s.page_size;
    int64_t p = blocks > 0 ? kTargetBlocks / blocks : 1;
    const int64_t most = (keys + 2 * kKeys - 1) / (2 * kKeys);
    if (p > most) p = most;
    if (p > kMaxParts) p = kMaxParts;
    return p < 1 ? 1 : int(p);
}

int smem_bytes(int D) { return (kRows * D + kKeys * (D + 4) + kKeys * D + 4 * kKeys * 4) * 4; }

// NJ: output elements of a lane, head_dim <= 32 NJ.
template <typename T, int NJ>
__global__ void __launch_bounds__(kThreads, NJ == 2 ? 5 : 1) generic_kernel(Args a, Partials part, int tt) {
    extern __shared__ float4 smem4[];
    __shared__ int scratch[4 + kThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const int D = a.head_dim, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *Q = reinterpret_cast<float *>(smem4), *K = Q + kRows * D, *V = K + kKeys * (D + 4);
    float *P = V + kKeys * D + warp * kKeys * 4;  // [key][row] of this warp
    // tiles from the last: with a causal mask the last tokens of a chunk have the most keys
    const TileAt at = find_tile(a, int(gridDim.x - 1 - blockIdx.x), tt, scratch);
    // wrong lengths of sequences without a tile are recorded too, by one block (of the number that all tiles may
    // need at most, the first is often idle)
    if (blockIdx.x + blockIdx.y + blockIdx.z == 0)
        for (int b = tid; b < a.n_seqs; b += kThreads) load_seq(a, b);
    if (at.b < 0) return;
    const Seq s = load_seq(a, at.b);
    const int slices = (a.group + kRows - 1) / kRows;
    const int hk = blockIdx.y / slices, g0 = (blockIdx.y % slices) * kRows;
    const int gw = min(a.group - g0, kRows);  // heads of the group in this block
    const int j0 = at.tile * tt, nj = min(tt, s.q_len - j0), rows = nj * gw;
    const int past = s.kv_len - s.q_len;

    // keys seen by each of the warp's rows, and by the block
    int seen[4];
    float m[4], l[4], o[4][NJ];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = warp * 4 + r;
        seen[r] = row < rows ? max(past + j0 + row / gw + 1, 0) : 0;
        m[r] = kNegInf;
        l[r] = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) o[r][j] = 0.f;
    }
    const int keys = max(past + j0 + nj, 0);
    const int64_t per = ((uint32_t(keys) + kKeys - 1) / kKeys + part.parts - 1) / part.parts * (int64_t)kKeys;
    const int64_t k_begin = blockIdx.z * per;
    const int k_end = int(min(k_begin + per, (int64_t)keys));

    // Tiles of keys: pieces of eight elements.  Small heads request the next tile before they work on
    // the one in hand, larger ones (which would not have the registers) two rounds of a tile at a time.
    constexpr int kRounds = (kKeys * NJ * 4 + kThreads - 1) / kThreads, kFly = kRounds < 2 ? kRounds : 2;
    constexpr bool kAhead = kFly == kRounds;
    const int pieces = D / 8;
    float kv[kFly][8], vv[kFly][8];
    // the cache offset of key lane, in every warp; slots past the last visible key are not read: they
    // may hold anything
    auto find_key = [&](int64_t k0) {
        const int64_t p = k0 + lane;
        if (p >= keys) return (int64_t)-1;
        const int pi = a.page_shift >= 0 ? int(p) >> a.page_shift : int(p) / a.page_size;
        return load_page(a, at.b, pi) * a.page_stride + hk * a.head_stride + (int64_t)(int(p) - pi * a.page_size) * a.token_stride;
    };
    auto load = [&](int64_t key_off, int i0) {
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const int item = (i0 + i) * kThreads + tid, kk = item / pieces, c = (item - kk * pieces) * 8;
            const int64_t off = __shfl_sync(0xffffffffu, key_off, kk & 31);
#pragma unroll
            for (int e = 0; e < 8; ++e) kv[i][e] = vv[i][e] = 0.f;
            if (kk < kKeys && off >= 0) {
                ldp8(static_cast<const T *>(a.k) + off + c, kv[i]);
                ldp8(static_cast<const T *>(a.v) + off + c, vv[i]);
            }
        }
    };
    auto store = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const int item = (i0 + i) * kThreads + tid, kk = item / pieces, c = (item - kk * pieces) * 8;
            if (kk >= kKeys) continue;
            // K rows are D + 4 floats apart, V rows D: both multiples of 16 bytes
            store8(K + kk * (D + 4) + c, kv[i]);
            store8(V + kk * D + c, vv[i]);
        }
    };
    if (kAhead && k_begin < k_end) load(find_key(k_begin), 0);

    // the rows of q, scaled, while those loads are in flight
    for (int i = tid; i < rows * (D / 8); i += kThreads) {
        const int r = i / (D / 8), c = i % (D / 8) * 8;
        float v[8];
        ldp8(static_cast<const T *>(a.q) + (s.q0 + j0 + r / gw) * a.q_stride + (int64_t)(hk * a.group + g0 + r % gw) * D + c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) Q[r * D + c + e] = v[e] * (a.scale * kLog2e);
    }
    for (int i = rows * D + tid; i < kRows * D; i += kThreads) Q[i] = 0.f;

    for (int64_t kb = k_begin; kb < k_end; kb += kKeys) {
        const int k0 = int(kb);
        if (kAhead) {
            __syncthreads();  // the tile before has been read
            store(0);
        } else {
            const int64_t key_off = find_key(kb);
            __syncthreads();
#pragma unroll
            for (int i0 = 0; i0 < kRounds; i0 += kFly) {
                load(key_off, i0);
                store(i0);
            }
        }
        __syncthreads();
        if (kAhead && kb + kKeys < k_end) load(find_key(kb + kKeys), 0);
        if (warp * 4 >= rows) continue;  // this warp only helps to load
        float sc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int d = 0; d < D; d += 4) {
            const float4 k4 = *reinterpret_cast<const float4 *>(K + lane * (D + 4) + d);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 q4 = *reinterpret_cast<const float4 *>(Q + (warp * 4 + r) * D + d);
                sc[r] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, sc[r]))));
            }
        }
        float pr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const bool on = k0 + lane < seen[r];
            float mx = on ? sc[r] : kNegInf;
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[r], mx);
            // a row that has seen nothing yet keeps m = -inf; 0 in its place makes its factor 2^-inf = 0, and
            // leaves a row whose scores are NaN what it is
            const float z = mn == kNegInf ? 0.f : mn, f = exp2f(m[r] - z);
            pr[r] = on ? exp2f(sc[r] - z) : 0.f;
            m[r] = mn;
            l[r] = l[r] * f + warp_sum(pr[r]);
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[r][j] *= f;
        }
        *reinterpret_cast<float4 *>(P + lane * 4) = make_float4(pr[0], pr[1], pr[2], pr[3]);
        __syncwarp();
#pragma unroll 8
        for (int kk = 0; kk < kKeys; ++kk) {
            const float4 p4 = *reinterpret_cast<const float4 *>(P + kk * 4);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if (lane + 32 * j < D) {
                    const float v = V[kk * D + lane + 32 * j];
                    o[0][j] = fmaf(p4.x, v, o[0][j]);
                    o[1][j] = fmaf(p4.y, v, o[1][j]);
                    o[2][j] = fmaf(p4.z, v, o[2][j]);
                    o[3][j] = fmaf(p4.w, v, o[3][j]);
                }
            }
        }
        __syncwarp();
    }

#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = warp * 4 + r;
        if (row >= rows) continue;
        const int t = s.q0 + j0 + row / gw, head = hk * a.group + g0 + row % gw;
        if (part.parts > 1) {
            const size_t idx = (size_t)blockIdx.z * a.n_tokens * a.n_heads + (size_t)t * a.n_heads + head;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                if (lane + 32 * j < D) part.o[idx * D + lane + 32 * j] = o[r][j];
            if (lane == 0) part.ml[idx] = make_float2(m[r], l[r]);
        } else {
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
            T *dst = static_cast<T *>(a.out) + t * a.out_stride + (int64_t)head * D;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                if (lane + 32 * j < D) from_f32(o[r][j] * inv, dst + lane + 32 * j);
            if (a.lse && lane == 0) a.lse[(size_t)t * a.n_heads + head] = l[r] == 0.f ? kNegInf : (m[r] + log2f(l[r])) * kLn2;
        }
    }
}

// Joins the parts of a row, one warp a row: o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p.
template <typename T>
__global__ void __launch_bounds__(kThreads) combine_kernel(Args a, Partials part) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t rows = (int64_t)a.n_tokens * a.n_heads;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, D = a.head_dim;
    if (row >= rows) return;
    const int t = int(row / a.n_heads), head = int(row % a.n_heads);
    if (t < ldp(a.cu_q) || t >= ldp(a.cu_q + a.n_seqs)) return;  // a padding row
    constexpr int kFly = 8;  // parts requested together; every part holds finite values (zeros for no keys)
    float4 v[kFly];
    auto load = [&](int d, int p0) {
#pragma unroll
        for (int p = 0; p < kFly; ++p) v[p] = ldp16f(part.o + (min(p0 + p, part.parts - 1) * rows + row) * D + d);
    };
    float2 ml = make_float2(kNegInf, 0.f);  // lane p: part p (at most 32)
    if (lane < part.parts) {
        const float *p = reinterpret_cast<const float *>(part.ml + lane * rows + row);
        ml = make_float2(ldp(p), ldp(p + 1));
    }
    load(min(lane * 4, D - 4), 0);
    float m = ml.x;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - m);
    const float l = warp_sum(ml.y * f);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *dst = static_cast<T *>(a.out) + t * a.out_stride + (int64_t)head * D;
    for (int d0 = 0; d0 < D; d0 += 128) {
        const int d = min(d0 + lane * 4, D - 4);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = 0; p0 < part.parts; p0 += kFly) {
            if (d0 + p0 > 0) load(d, p0);
#pragma unroll
            for (int p = 0; p < kFly; ++p) {
                const float fp = p0 + p < 32 ? __shfl_sync(0xffffffffu, f, (p0 + p) & 31) : 0.f;  // 0 past the last
                acc.x = fmaf(fp, v[p].x, acc.x);
                acc.y = fmaf(fp, v[p].y, acc.y);
                acc.z = fmaf(fp, v[p].z, acc.z);
                acc.w = fmaf(fp, v[p].w, acc.w);
            }
        }
        if (d0 + lane * 4 >= D) continue;
        from_f32(acc.x * inv, dst + d);
        from_f32(acc.y * inv, dst + d + 1);
        from_f32(acc.z * inv, dst + d + 2);
        from_f32(acc.w * inv, dst + d + 3);
    }
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
}

template <typename T, int NJ>
cudaError_t launch_typed(const Args &a, const Partials &p, dim3 grid, int tt, cudaStream_t st) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(generic_kernel<T, NJ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   smem_bytes(32 * NJ));
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    return launch_pdl(generic_kernel<T, NJ>, grid, dim3(kThreads), smem_bytes(a.head_dim), st, a, p, tt);
}

template <typename T>
cudaError_t launch_dim(const Args &a, const Partials &p, dim3 grid, int tt, cudaStream_t st) {
    if (a.head_dim <= 64) return launch_typed<T, 2>(a, p, grid, tt, st);
    if (a.head_dim <= 128) return launch_typed<T, 4>(a, p, grid, tt, st);
    return launch_typed<T, 8>(a, p, grid, tt, st);
}

}  // namespace

size_t generic_ws_bytes(const moe_attn_shape &s) {
    const int p = parts(s);
    return p > 1 ? (size_t)p * s.n_tokens * s.n_heads * (s.head_dim + 2) * 4 : 0;
}

cudaError_t launch_combine(const Args &a, int dtype, const Partials &p, cudaStream_t st) {
    const dim3 grid(unsigned(((int64_t)a.n_tokens * a.n_heads + 3) / 4));
    return dtype == MOE_DT_F32 ? launch_pdl(combine_kernel<float>, grid, dim3(kThreads), 0, st, a, p)
                               : launch_pdl(combine_kernel<uint16_t>, grid, dim3(kThreads), 0, st, a, p);
}

cudaError_t launch_generic(const Args &a, int dtype, const moe_attn_shape &s, char *ws, cudaStream_t st) {
    Partials p{};
    p.parts = parts(s);
    p.o = reinterpret_cast<float *>(ws);
    p.ml = reinterpret_cast<float2 *>(p.o + (size_t)p.parts * s.n_tokens * s.n_heads * s.head_dim);
    const dim3 grid(unsigned(max_tiles(s)), unsigned(s.n_kv_heads * head_slices(a.group)), unsigned(p.parts));
    const int tt = tokens_per_tile(a.group);
    const cudaError_t e = dtype == MOE_DT_F32 ? launch_dim<float>(a, p, grid, tt, st)
                                              : launch_dim<uint16_t>(a, p, grid, tt, st);
    if (e != cudaSuccess || p.parts == 1) return e;
    return launch_combine(a, dtype, p, st);
}

}  // namespace attn
}  // namespace moe
