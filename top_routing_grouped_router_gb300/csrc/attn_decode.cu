// attn_decode.cu -- attention of a few new tokens a sequence (decode, draft tokens) over the
// paged cache, bf16: the cache is read once, at the memory's rate.
//
// The query rows that share a key head (group x chunk, at most 16) fill one M = 16 tile of
// mma.sync, so a step of 16 keys is S = Q K^T, a running softmax, O += P V in one warp's
// registers; tcgen05's M = 128 would be 8 to 16 times padding here, and the matrix work is a
// twentieth of what the memory allows.  Each warp streams its own keys: cp.async copies of
// 16-byte pieces into a ring of its own (no barrier between warps), rows swizzled so that
// ldmatrix reads without bank conflicts.
//
// All (sequence, key head) pairs are laid end to end as steps of 16 keys, and every CTA takes
// an equal share of that line, whatever the lengths.  A pair that a CTA holds whole is written
// out at once; the others leave (max, sum, unnormalised O) in the workspace, and the CTA that
// arrives last joins them in order, so the bits do not depend on timing.
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kMaxGrid = 320;     // counters and partial slots (152 SMs x 2 = 304)
constexpr int kStep = 16;         // keys of a step
constexpr int kRows = 16;
constexpr size_t kCounters = 512;  // byte offset of the arrival counters in the workspace header
static_assert(kCounters + kMaxGrid * 4 <= kHdrBytes, "");

template <int D>
struct Cfg {
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kStageBytes = 2 * kStep * D * 2;  // K rows, V rows
    static constexpr int kRing = kStages * kStageBytes;
    static constexpr int kSmem = kWarps * kRing;  // also the join's buffers
    static_assert(kWarps * kRows * (D + 2) * 4 <= kSmem, "");
    static_assert(kMaxGrid * kRows * 4 <= kSmem, "");
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
// 16 bytes global -> shared; src_bytes = 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 2^x by the hardware unit (relative error about 2^-22; 0 for -inf).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int steps_of(const Seq &s) { return s.q_len ? max(1, (s.kv_len + kStep - 1) / kStep) : 0; }

// Sums (and with `mine` prefix-sums) one value a thread over the block.
__device__ __forceinline__ int64_t block_scan(int64_t n, int64_t *total, int64_t *scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? scratch[w] : 0;
        sum += scratch[w];
    }
    *total = sum;
    return before + incl - n;
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(Args a, int *counters, float *part_o, float2 *part_ml) {
    using C = Cfg<D>;
    constexpr int NT = D / 8;        // 8-column tiles of O
    constexpr int KS = D / 16;       // 16-element steps of the head dimension
    constexpr int CH = D / 8;        // 16-byte pieces of a row
    constexpr int RPI = 32 / CH;     // rows a warp copies per instruction
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t scratch[kWarps + 2];
    __shared__ int last_flag;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int G = a.group, Hkv = a.n_kv_heads;

    // this CTA's share of all steps
    int64_t n0 = 0, total = 0;
    for (int b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
        int64_t n = 0, sum;
        if (b0 + tid < a.n_seqs) n = (int64_t)steps_of(load_seq(a, b0 + tid)) * Hkv;
        if (b0 == 0) n0 = n;
        block_scan(n, &sum, scratch);
        total += sum;
    }
    // no more CTAs than leave every warp a step
    const int64_t ctas = max((int64_t)1, min((int64_t)gridDim.x, total / kWarps));
    const int64_t cta = blockIdx.x;
    if (cta >= ctas || total == 0) return;
    const int64_t u_end = (cta + 1) * total / ctas;
    int64_t u = cta * total / ctas;
    if (u >= u_end) return;
    int b = 0;
    int64_t base = 0;  // first step of sequence b
    for (int b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
        int64_t n = n0, sum;
        if (b0 > 0) n = b0 + tid < a.n_seqs ? (int64_t)steps_of(load_seq(a, b0 + tid)) * Hkv : 0;
        const int64_t before = base + block_scan(n, &sum, scratch);
        if (u >= before && u < before + n) {
            scratch[kWarps] = b0 + tid;
            scratch[kWarps + 1] = before;
        }
        if (u < base + sum) break;
        base += sum;
    }
    __syncthreads();
    b = int(scratch[kWarps]);
    base = scratch[kWarps + 1];

    const uint32_t ring = smem_addr(smem) + warp * C::kRing;
    const float sl2 = a.scale * kLog2e;
    Seq s = load_seq(a, b);
    int steps = steps_of(s);

    while (u < u_end) {
        while (u >= base + (int64_t)steps * Hkv) {  // the next sequence with a chunk
            base += (int64_t)steps * Hkv;
            s = load_seq(a, ++b);
            steps = steps_of(s);
        }
        const int h = int((u - base) / steps);
        const int64_t item = base + (int64_t)h * steps;  // its first step
        const int step0 = int(u - item), step1 = int(min((int64_t)steps, u_end - item));
        const int rows = min(s.q_len * G, kRows), past = s.kv_len - s.q_len;

        // the warp's keys: steps step0 + warp, + kWarps, ...  Lane r < 16 finds the cache offset of
        // key row r, one step before it is copied.
        const int mine = step1 - step0 > warp ? (step1 - step0 - warp + kWarps - 1) / kWarps : 0;
        auto find_row = [&](int i) -> int64_t {
            const int p = (step0 + warp + i * kWarps) * kStep + (lane & 15);
            if (i >= mine || p >= s.kv_len) return -1;
            const int pi = p / a.page_size;
            return load_page(a, b, pi) * a.page_stride + (int64_t)(p - pi * a.page_size) * a.token_stride;
        };
        const uint16_t *kc = static_cast<const uint16_t *>(a.k) + h * a.head_stride;
        const uint16_t *vc = static_cast<const uint16_t *>(a.v) + h * a.head_stride;
        auto copy = [&](int i, int64_t row_off) {
            if (i < mine) {
                const uint32_t dst = ring + (i % C::kStages) * C::kStageBytes;
#pragma unroll
                for (int it = 0; it < kStep / RPI; ++it) {
                    const int r = it * RPI + lane / CH, c = lane % CH;
                    const int64_t off = __shfl_sync(0xffffffffu, row_off, r);
                    const uint32_t at = dst + r * (D * 2) + ((c ^ (r & 7)) * 16);
                    const int n = off >= 0 ? 16 : 0;
                    cp16(at, kc + (n ? off + c * 8 : 0), n);
                    cp16(at + kStep * D * 2, vc + (n ? off + c * 8 : 0), n);
                }
            }
            cp_commit();
        };
        int64_t next = find_row(0);
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) {
            const int64_t cur = next;
            next = find_row(i + 1);
            copy(i, cur);
        }

        // Q as A fragments: rows g and g + 8, columns 16 ks + 2 t4 (+1) and + 8
        uint32_t q[KS][4];
        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (int64_t)s.q0 * a.q_stride + (int64_t)h * G * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = g + (e & 1) * 8, c = ks * 16 + t4 * 2 + (e >> 1) * 8;
                q[ks][e] = r < rows ? ldp(reinterpret_cast<const uint32_t *>(qp + (r / G) * a.q_stride + (r % G) * D + c)) : 0u;
            }
        const int seen0 = g < rows ? past + g / G + 1 : 0, seen1 = g + 8 < rows ? past + (g + 8) / G + 1 : 0;
        const int seen_all = past + 1;  // keys that every row sees
        float o[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;

        for (int i = 0; i < mine; ++i) {
            const int64_t cur = next;
            next = find_row(i + C::kStages);
            copy(i + C::kStages - 1, cur);
            cp_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t kb = ring + (i % C::kStages) * C::kStageBytes, vb = kb + kStep * D * 2;
            float sc[2][4] = {};
            {
                const int r = (lane & 7) + (lane >> 4) * 8;  // matrices: keys 0-7 (two pieces), keys 8-15
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t kf[4];
                    ldsm4(kb + r * (D * 2) + (((2 * ks + ((lane >> 3) & 1)) ^ (r & 7)) * 16), kf);
                    mma16816(sc[0], q[ks], kf[0], kf[1]);
                    mma16816(sc[1], q[ks], kf[2], kf[3]);
                }
            }
            const int key0 = (step0 + warp + i * kWarps) * kStep;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] *= sl2;
            if (key0 + kStep > seen_all) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + n * 8 + t4 * 2 + (e & 1);
                        if (key >= (e < 2 ? seen0 : seen1)) sc[n][e] = kNegInf;
                    }
            }
            float x0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
            float x1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
#pragma unroll
            for (int w = 1; w <= 2; w <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
            }
            const float n_0 = fmaxf(m0, x0), n_1 = fmaxf(m1, x1);
            // a row that has seen nothing keeps max -inf; 0 in its place makes its terms 2^-inf = 0
            const float z0 = n_0 == kNegInf ? 0.f : n_0, z1 = n_1 == kNegInf ? 0.f : n_1;
            if (__any_sync(0xffffffffu, n_0 != m0 || n_1 != m1)) {
                const float f0 = ex2(m0 - z0), f1 = ex2(m1 - z1);
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[j][0] *= f0;
                    o[j][1] *= f0;
                    o[j][2] *= f1;
                    o[j][3] *= f1;
                }
                m0 = n_0;
                m1 = n_1;
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                sc[n][0] = ex2(sc[n][0] - z0);
                sc[n][1] = ex2(sc[n][1] - z0);
                sc[n][2] = ex2(sc[n][2] - z1);
                sc[n][3] = ex2(sc[n][3] - z1);
                l0 += sc[n][0] + sc[n][1];  // this lane's columns; the quad's are added at the end
                l1 += sc[n][2] + sc[n][3];
            }
            const uint32_t p[4] = {pack_bf16(sc[0][0], sc[0][1]), pack_bf16(sc[0][2], sc[0][3]),
                                   pack_bf16(sc[1][0], sc[1][1]), pack_bf16(sc[1][2], sc[1][3])};
            {
                const int r = lane & 15;  // matrices: keys 0-7, 8-15 of one piece, then of the next
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t vf[4];
                    ldsm4t(vb + r * (D * 2) + (((j + (lane >> 4)) ^ (r & 7)) * 16), vf);
                    mma16816(o[j], p, vf[0], vf[1]);
                    mma16816(o[j + 1], p, vf[2], vf[3]);
                }
            }
            __syncwarp();  // the stage is read before a lane's next copy lands in it
        }
        cp_wait<0>();
#pragma unroll
        for (int w = 1; w <= 2; w <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, w);
            l1 += __shfl_xor_sync(0xffffffffu, l1, w);
        }

        // join the warps: [warp][row][D], then [warp][row] (max, sum)
        float *jo = reinterpret_cast<float *>(smem);
        float2 *jm = reinterpret_cast<float2 *>(jo + kWarps * kRows * D);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            *reinterpret_cast<float2 *>(jo + (warp * kRows + g) * D + j * 8 + t4 * 2) = make_float2(o[j][0], o[j][1]);
            *reinterpret_cast<float2 *>(jo + (warp * kRows + g + 8) * D + j * 8 + t4 * 2) = make_float2(o[j][2], o[j][3]);
        }
        if (t4 == 0) {
            jm[warp * kRows + g] = make_float2(m0, l0);
            jm[warp * kRows + g + 8] = make_float2(m1, l1);
        }
        __syncthreads();
        const int64_t c0 = ((item + 1) * ctas - 1) / total, c1 = ((item + steps) * ctas - 1) / total;
        const bool whole = c0 == c1;
        const size_t slot = (size_t)cta * 2 + (cta == c0 ? 1 : 0);
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            float m = kNegInf, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, jm[w * kRows + r].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = jm[w * kRows + r];
                const float f = ml.x == kNegInf ? 0.f : ex2(ml.x - m);
                const float4 v = *reinterpret_cast<const float4 *>(jo + (w * kRows + r) * D + d);
                l = fmaf(f, ml.y, l);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            const int tok = s.q0 + r / G, head = h * G + r % G;
            if (whole) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + tok * a.out_stride + (int64_t)head * D + d) =
                    make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
                if (a.lse && d == 0)
                    a.lse[(size_t)tok * a.n_heads + head] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(part_o + (slot * kRows + r) * D + d) = acc;
                if (d == 0) part_ml[slot * kRows + r] = make_float2(m, l);
            }
        }
        if (!whole) {
            __syncthreads();
            if (tid == 0) last_flag = arrive_acq_rel(counters + c0) == int(c1 - c0);
            __syncthreads();
            if (last_flag) {
                const int n = int(c1 - c0) + 1;
                if (tid == 0) counters[c0] = 0;  // as the next call expects it
                float *fac = reinterpret_cast<float *>(smem);  // [part][row]
                auto slot_of = [&](int i) { return (size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0); };
                for (int r = warp; r < rows; r += kWarps) {
                    float m = kNegInf, l = 0.f;
                    for (int i = lane; i < n; i += 32) m = fmaxf(m, ldp(&part_ml[slot_of(i) * kRows + r].x));
#pragma unroll
                    for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                    for (int i = lane; i < n; i += 32) {
                        const float *p = &part_ml[slot_of(i) * kRows + r].x;
                        const float f = ldp(p) == kNegInf ? 0.f : ex2(ldp(p) - m);
                        fac[i * kRows + r] = f;
                        l = fmaf(f, ldp(p + 1), l);
                    }
                    l = warp_sum(l);
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    for (int i = lane; i < n; i += 32) fac[i * kRows + r] *= inv;
                    if (a.lse && lane == 0)
                        a.lse[(size_t)(s.q0 + r / G) * a.n_heads + h * G + r % G] =
                            l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
                }
                __syncthreads();
                for (int i = tid; i < rows * (D / 4); i += kThreads) {
                    const int r = i / (D / 4), d = i % (D / 4) * 4;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int k = 0; k < n; ++k) {
                        const float4 v = ldp16f(part_o + (slot_of(k) * kRows + r) * D + d);
                        const float f = fac[k * kRows + r];
                        acc.x = fmaf(f, v.x, acc.x);
                        acc.y = fmaf(f, v.y, acc.y);
                        acc.z = fmaf(f, v.z, acc.z);
                        acc.w = fmaf(f, v.w, acc.w);
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + (s.q0 + r / G) * a.out_stride +
                                               (int64_t)(h * G + r % G) * D + d) =
                        make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
                }
            }
        }
        __syncthreads();  // the join's buffers become the ring again
        u = item + step1;
    }
}

template <int D>
cudaError_t launch_typed(const Args &a, char *hdr, char *ws, int grid, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    float *o = reinterpret_cast<float *>(ws);
    float2 *ml = reinterpret_cast<float2 *>(o + (size_t)kMaxGrid * 2 * kRows * D);
    return launch_pdl(decode_kernel<D>, dim3(grid), dim3(kThreads), Cfg<D>::kSmem, st, a,
                      reinterpret_cast<int *>(hdr + kCounters), o, ml);
}

}  // namespace

// bf16, head sizes 64 and 128, and at most 16 query rows a key head.
bool decode_supported(const moe_attn_shape &s) {
    return s.dtype == MOE_DT_BF16 && (s.head_dim == 64 || s.head_dim == 128) &&
           (int64_t)s.max_q * (s.n_heads / s.n_kv_heads) <= kRows;
}
size_t decode_ws_bytes(const moe_attn_shape &s) { return (size_t)kMaxGrid * 2 * kRows * (s.head_dim + 2) * 4; }

cudaError_t launch_decode(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int sms, cudaStream_t st) {
    const int grid = sms * kCtasPerSm < kMaxGrid ? sms * kCtasPerSm : kMaxGrid;
    return s.head_dim == 128 ? launch_typed<128>(a, hdr, ws, grid, st) : launch_typed<64>(a, hdr, ws, grid, st);
}

}  // namespace attn
}  // namespace moe
