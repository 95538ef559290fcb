// q4_linear_tc.cu -- out = x . W^T (+ residual) with 4-bit weights for batches of more rows than
// mma.sync keeps up with: the codes stream through the 5th-generation tensor cores.
//
// A CTA takes 128 outputs at a time; 128 inputs of their codes (8 KB) are a stage.
//   loads     TMA box of the codes, cp.async of the scales
//   unpack    eight warps, one output a thread: codes to the exact bf16 integers 16 + j (a shift and
//             a LOP3 for two of them), written to TMEM as the A operand
//   MMA       A (TMEM, outputs x inputs) times x (shared memory, rows x inputs), one fp32 product
//             P = sum (16 + j) x for each 64 inputs
//   add       eight warps, half the columns each: result += scale (P - (16 + j0) sum x), in fp32 registers
// No weight is rounded.  x lies in shared memory whole (or the CTA's share of the inputs, where a
// cluster splits them), in the order in which the codes are unpacked.
#include "attn.cuh"
#include "tc_common.cuh"

#include <algorithm>
#include <cmath>
#include <cooperative_groups.h>

#include "q4_linear.cuh"

namespace moe {
namespace q4 {
namespace {

using namespace tc;

constexpr int kLoadWarp = 0, kMmaWarp = 1, kUnpack0 = 2, kAdd0 = 10, kThreads = 18 * 32;
constexpr int kStagers = kThreads / 32 - kUnpack0;  // warps that bring x into place
constexpr int kOut = 128, kIn = 128;
// Stages of codes and scales: what fits next to x, from kMinRing to kMaxRing.  A stage lands 1.5 us
// after it is asked for under load: 6 stages (48 KB) held a 16 x 2048 x 131072 product at 61 us.
constexpr int kMinRing = 6, kMaxRing = 16;
constexpr int kCodeBytes = kOut * kIn / 2, kScaleBytes = kOut * 2 * 4, kStage = kCodeBytes + kScaleBytes;
constexpr int kA = 4;                                 // A operands in TMEM, 64 columns each
constexpr uint32_t kColD = kA * 64;
constexpr int kMaxSlices = 8, kMaxSmem = 232448, kCtrl = 512;

// Set if a wait ran out: read by moe_q4_linear_read_error.
__device__ int32_t g_err;

struct TcArgs {
    Q4Args a;
    int T0, rows;
    int slices, tiles, slice_stages, shift, ring;
    float centre, step;
    unsigned long long wait_ns;
    int extra_need;
};

__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// One arrival on the barrier when the thread's copies so far have landed.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// A stage's products, D = A B over its first 64 inputs and over the others (four MMAs each, A at
// TMEM columns a + 8 i, B 32 bytes further each; the second half of B at b2, of D at d2), and the
// commits to the two barriers: one election, one block of assembly, since the issuing warp shares
// its scheduler with warps that unpack and add.
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t d2, uint32_t a, uint64_t b, uint64_t b2, uint32_t idesc,
                                          uint32_t bar_d, uint32_t bar_a) {
    asm volatile(
        "{\n\t.reg .pred e, z, o;\n\t.reg .b64 v;\n\t.reg .b32 p;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 z, %5, %5;\n\tsetp.eq.b32 o, %5, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %3, %5, z;\n\t"
        "add.s32 p, %2, 8;\n\tadd.s64 v, %3, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %5, o;\n\t"
        "add.s32 p, %2, 16;\n\tadd.s64 v, %3, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %5, o;\n\t"
        "add.s32 p, %2, 24;\n\tadd.s64 v, %3, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %5, o;\n\t"
        "add.s32 p, %2, 32;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%1], [p], %4, %5, z;\n\t"
        "add.s32 p, %2, 40;\n\tadd.s64 v, %4, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%1], [p], v, %5, o;\n\t"
        "add.s32 p, %2, 48;\n\tadd.s64 v, %4, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%1], [p], v, %5, o;\n\t"
        "add.s32 p, %2, 56;\n\tadd.s64 v, %4, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%1], [p], v, %5, o;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];\n\t}"
        ::"r"(d), "r"(d2), "r"(a), "l"(b), "l"(b2), "r"(idesc), "r"(bar_d), "r"(bar_a)
        : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t ta, uint32_t *r);
template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t ta, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(ta) : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t ta, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(ta) : "memory");
}
template <int N>
__device__ __forceinline__ void ld_done(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// COLS: rows of x of a pass (the MMA's N), 16, 32 or 64.
template <int COLS>
__global__ void __launch_bounds__(kThreads, 1) q4_tc_kernel(const __grid_constant__ CUtensorMap map,
                                                            const __grid_constant__ TcArgs m) {
    namespace cg = cooperative_groups;
    constexpr int kD = COLS == 64 ? 2 : 4;  // products in TMEM, 2 COLS columns each
    constexpr int kHalf = COLS / 2;         // columns of an adding warp
    extern __shared__ __align__(1024) uint8_t smem[];
    const Q4Args &a = m.a;
    uint8_t *xs = smem;                                             // [64 inputs][COLS][128 bytes]
    uint8_t *ring = xs + (size_t)m.slice_stages * 2 * COLS * 128;   // [m.ring][codes, scales]
    float *starts = reinterpret_cast<float *>(ring + m.ring * kStage);  // [64 inputs][COLS]: -(16 + j0) sum x
    uint64_t *cf = reinterpret_cast<uint64_t *>(starts + (size_t)m.slice_stages * 2 * COLS);  // [kMaxRing]
    uint64_t *ce = cf + kMaxRing, *af = ce + kMaxRing, *ae = af + kA, *df = ae + kA, *de = df + kD, *xf = de + kD;
    uint64_t *drain = xf + 1;
    volatile int *abort = reinterpret_cast<volatile int *>(drain + 1);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1) + 1;
    static_assert((2 * kMaxRing + 2 * kA + 2 * 4 + 2) * 8 + 8 <= kCtrl, "");
    const Waits wt{&g_err, abort, m.wait_ns, smem_u32(const_cast<int *>(abort))};
    // the warp's number from one lane: known to be the same in all of them, so that the MMA warp's operands
    // stay in uniform registers
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (smem_u32(smem) & 1023u) {  // not seen: shared memory starts on such a boundary
        if (tid == 0) record_error(&g_err, MOE_ERR_DEVICE);
        return;
    }

    const int stages = (a.K + kIn - 1) / kIn;
    const int slice = int(blockIdx.x) % m.slices, group = int(blockIdx.x) / m.slices, groups = int(gridDim.x) / m.slices;
    const int s0 = int((int64_t)stages * slice / m.slices), s1 = int((int64_t)stages * (slice + 1) / m.slices);
    const int my_tiles = (m.tiles - group + groups - 1) / groups;

    if (tid == 0) {
        for (int i = 0; i < m.ring; ++i) {
            mbar_init(smem_u32(&cf[i]), 33);      // the TMA's arrival and 32 lanes' scales
            mbar_init(smem_u32(&ce[i]), 4 + 8);  // unpacking and adding warps
        }
        for (int i = 0; i < kA; ++i) {
            mbar_init(smem_u32(&af[i]), 4 + m.extra_need);
            mbar_init(smem_u32(&ae[i]), 1);
        }
        for (int i = 0; i < kD; ++i) {
            mbar_init(smem_u32(&df[i]), 1);
            mbar_init(smem_u32(&de[i]), 8);
        }
        mbar_init(smem_u32(xf), kStagers);
        mbar_init(smem_u32(drain), 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    const uint32_t blocks = uint32_t(a.K / a.q_block);
    bool ok = true;
    float acc[kHalf];  // adding warps: this output's sums

    // Codes and scales, as much as x, may be what the kernel before this one writes: every warp that
    // reads an array waits for that kernel first.
    if (warp >= kUnpack0) {
        // x, by the unpacking and adding warps before they have anything to do
        const int n8 = (s1 - s0) * (kIn / 8);
        auto put = [&](int c, int r, uint4 v) {  // 16-byte piece c of a row: 128-byte swizzle within 64 inputs
            *reinterpret_cast<uint4 *>(xs + ((size_t)(c >> 3) * COLS + r) * 128 + (((c & 7) ^ (r & 7)) * 16)) = v;
        };
        for (int r = m.rows + warp - kUnpack0; r < COLS; r += kStagers)  // rows past the last are zero
            for (int c = lane; c < n8; c += 32) {
                put(c, r, make_uint4(0, 0, 0, 0));
                if ((c & 7) == 0) starts[(c >> 3) * COLS + r] = 0.f;
            }
        griddep_wait();
        griddep_launch_dependents();
        constexpr int kBatch = 8;  // loads in flight a thread
        const int most = a.K - 8 - s0 * kIn, beside = m.rows < kStagers ? kStagers / m.rows : 1, mine = warp - kUnpack0;
        for (int r = mine / beside; r < m.rows && mine < kStagers / beside * beside; r += kStagers / beside) {
            const uint16_t *xr = a.x + (m.T0 + r) * a.x_stride + (int64_t)s0 * kIn;
            for (int w0 = mine % beside * 32; w0 < n8; w0 += kBatch * beside * 32) {
                const int c0 = w0 + lane;
                uint4 v[kBatch];
#pragma unroll
                for (int b = 0; b < kBatch; ++b) v[b] = ldp16(xr + min((c0 + b * beside * 32) * 8, most));
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const int c = c0 + b * beside * 32;
                    if (c * 8 > most) v[b] = make_uint4(0, 0, 0, 0);
                    float f[8];
                    attn::unpack8(v[b], f);
                    float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
#pragma unroll
                    for (int w = 1; w < 8; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                    const uint4 u = v[b];
                    if (c < n8) {
                        if ((c & 7) == 0) starts[(c >> 3) * COLS + r] = -m.centre * sum;
                        put(c, r, make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632),
                                             __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632)));
                    }
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read x
        asm volatile("bar.sync 1, %0;" ::"n"(kStagers * 32) : "memory");  // the adding warps read others' start values
        if (lane == 0) mbar_arrive(smem_u32(xf));
    }

    if (warp == kLoadWarp) {
        griddep_wait();
        int filled = 0;  // stages filled so far
        const int srow = lane >> 1, shalf = lane & 1;
        int slot = 0;
        uint32_t phase = 1;
        for (int k = 0; k < my_tiles && ok; ++k) {
            const int n0 = (group + k * groups) * kOut;
            for (int st = s0; st < s1; ++st) {
                ok = mbar_wait(smem_u32(&ce[slot]), phase, wt);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = smem_u32(&cf[slot]), dst = smem_u32(ring + slot * kStage);
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, kCodeBytes);
                    tma_load_2d(dst, &map, st * (kIn / 2), n0, bar);
                }
                // the aligned word that a scale lies in, 2 bytes of it at the array's end
                const bool in = st * kIn + shalf * 64 < a.K;
                uint32_t e = uint32_t(n0 + srow) * blocks + ((st * 2 + shalf) >> m.shift);
#pragma unroll
                for (int i = 0; i < kOut / 16; ++i, e += 16 * blocks) {
                    const bool on = in && n0 + srow + i * 16 < a.N;
                    cp4(dst + kCodeBytes + (i * 32 + lane) * 4, a.scales + (on ? e & ~1u : 0u), on ? 2 << (e & 1) : 0);
                }
                cp_arrive(bar);
                ++filled;
                if (++slot == m.ring) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {  // the copies in flight land before the CTA gives up its memory
            for (int i = max(0, filled - m.ring); i < filled; ++i)
                mbar_wait_drain(smem_u32(&cf[i % m.ring]), (i / m.ring) & 1, wt);
        }
    } else if (warp == kMmaWarp) {
        griddep_wait();  // or the limit of its first wait would count the time that the kernel before still runs
        const uint32_t idesc = instr_desc(kOut, COLS);
        int i = 0;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(xf), 0, wt));
        for (int k = 0; k < my_tiles && ok; ++k) {
            uint64_t b_desc = smem_desc(smem_u32(xs));
            for (int st = s0; st < s1; ++st, ++i) {
                ok = mbar_wait(smem_u32(&de[i % kD]), ((i / kD) & 1) ^ 1, wt) &&
                     mbar_wait(smem_u32(&af[i % kA]), (i / kA) & 1, wt);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + kColD + (i % kD) * 2 * COLS;
                mma_stage(d, d + COLS, tmem + (i % kA) * 64, b_desc, b_desc + COLS * 8, idesc, smem_u32(&df[i % kD]),
                          smem_u32(&ae[i % kA]));
                b_desc += 2 * COLS * 8;
            }
        }
        // every MMA and every arrival of its commits is over before the CTA ends
        mma_commit_warp(smem_u32(drain));
        mbar_wait_drain(smem_u32(drain), 0, wt);
    } else if (warp < kAdd0) {
        const int set = (warp - kUnpack0) >> 2, q = warp & 3, row = q * 32 + lane;
        const uint32_t mask = 0x00780078u, bias = 0x41804180u, ta = tmem + (uint32_t(q) << 21);
        const uint32_t row_at = row * 64, swz = (row >> 1) & 3;
        const int total = my_tiles * (s1 - s0);
        int slot = set;
        uint32_t phase = 0;
        for (int i = set; i < total; i += 2) {
            ok = mbar_wait(smem_u32(&cf[slot]), phase, wt);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t at = smem_u32(ring + slot * kStage) + row_at;
            uint32_t w[16], v[64];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint4 u = lds_v4(at + ((c ^ swz) * 16));
                w[4 * c] = u.x;
                w[4 * c + 1] = u.y;
                w[4 * c + 2] = u.z;
                w[4 * c + 3] = u.w;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                v[4 * c] = code_pair(w[c] << 3, mask, bias);
                v[4 * c + 1] = code_pair(w[c] >> 1, mask, bias);
                v[4 * c + 2] = code_pair(w[c] >> 5, mask, bias);
                v[4 * c + 3] = code_pair(w[c] >> 9, mask, bias);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ce[slot]));
            if ((slot += 2) >= m.ring) {
                slot -= m.ring;
                phase ^= 1;
            }
            ok = mbar_wait(smem_u32(&ae[i % kA]), ((i / kA) & 1) ^ 1, wt);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            tmem_st64(ta + (i % kA) * 64, v);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&af[i % kA]));
        }
        ok = __all_sync(0xffffffffu, ok);
    } else {
        const int set = (warp - kAdd0) >> 2, q = warp & 3, row = q * 32 + lane;
        const uint32_t ta = tmem + (uint32_t(q) << 21) + kColD + set * kHalf;
        const uint32_t odd = uint32_t(row) * blocks;  // tiles start on even rows: the same parity in all
        int i = 0, slot = 0;
        uint32_t phase = 0;
        for (int k = 0; k < my_tiles && ok; ++k) {
#pragma unroll
            for (int n = 0; n < kHalf; ++n) acc[n] = 0.f;
            for (int st = s0; st < s1; ++st, ++i) {
                ok = mbar_wait(smem_u32(&cf[slot]), phase, wt) &&
                     mbar_wait(smem_u32(&df[i % kD]), (i / kD) & 1, wt);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint2 words = lds_v2(smem_u32(ring + slot * kStage) + kCodeBytes + row * 8);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float sc = half_of(b ? words.y : words.x, (odd + ((st * 2 + b) >> m.shift)) & 1 ? kHigh : kLow);
                    const float4 *z = reinterpret_cast<const float4 *>(starts + ((size_t)(st - s0) * 2 + b) * COLS + set * kHalf);
#pragma unroll
                    for (int c = 0; c < kHalf; c += (kHalf < 16 ? kHalf : 16)) {
                        constexpr int W = kHalf < 16 ? kHalf : 16;
                        uint32_t p[W];
                        tmem_ld<W>(ta + ((i % kD) * 2 + b) * COLS + c, p);
                        ld_done(p);
#pragma unroll
                        for (int e = 0; e < W; e += 4) {
                            const float4 s = z[(c + e) / 4];
                            acc[c + e] = fmaf(sc, __uint_as_float(p[e]) + s.x, acc[c + e]);
                            acc[c + e + 1] = fmaf(sc, __uint_as_float(p[e + 1]) + s.y, acc[c + e + 1]);
                            acc[c + e + 2] = fmaf(sc, __uint_as_float(p[e + 2]) + s.z, acc[c + e + 2]);
                            acc[c + e + 3] = fmaf(sc, __uint_as_float(p[e + 3]) + s.w, acc[c + e + 3]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&de[i % kD]));
                    mbar_arrive(smem_u32(&ce[slot]));
                }
                if (++slot == m.ring) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (!ok || m.slices > 1) break;  // sliced: one tile a CTA, joined below
            const int n = (group + k * groups) * kOut + row;
            if (n < a.N) {
                bool finite = true;
#pragma unroll
                for (int c = 0; c < kHalf; ++c) {
                    acc[c] *= m.step;
                    finite = finite && q4_is_finite(acc[c]);
                }
                // rows past the last are zeros
                if (finite) {
#pragma unroll
                    for (int c = 0; c < kHalf; ++c)
                        if (set * kHalf + c < m.rows) q4_write(a, m.T0 + set * kHalf + c, n, acc[c]);
                } else {
                    uint32_t again = 0;
#pragma unroll
                    for (int c = 0; c < kHalf; ++c)
                        if (set * kHalf + c < m.rows) again |= uint32_t(!q4_emit(a, m.T0 + set * kHalf + c, n, acc[c])) << c;
                    for (; again; again &= again - 1) q4_emit_by_terms(a, m.T0 + set * kHalf + __ffs(again) - 1, n);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (m.slices > 1) {
        // the slices' sums added in order, the rows of x shared out over the cluster
        cg::cluster_group cl = cg::this_cluster();
        float *part = reinterpret_cast<float *>(ring);  // [COLS][kOut]: every stage has been read
        if (warp >= kAdd0) {
            const int set = (warp - kAdd0) >> 2, row = (warp & 3) * 32 + lane;
#pragma unroll
            for (int c = 0; c < kHalf; ++c) part[(set * kHalf + c) * kOut + row] = acc[c];
        }
        griddep_wait();  // the residual may be an earlier kernel's
        cl.sync();
        for (int idx = tid; idx < COLS * kOut; idx += kThreads) {
            const int r = idx / kOut, n = group * kOut + idx % kOut;
            if (r % m.slices != slice || r >= m.rows || n >= a.N) continue;
            float y = 0.f;
            for (int s = 0; s < m.slices; ++s) y += *cl.map_shared_rank(part + idx, s);
            if (!q4_emit(a, m.T0 + r, n, y * m.step)) q4_emit_by_terms(a, m.T0 + r, n);
        }
        cl.sync();  // no CTA leaves while another reads its sums
    }
}

template <int COLS>
int smem_bytes(int slice_stages, int ring) {
    return slice_stages * 2 * COLS * (128 + 4) + ring * kStage + kCtrl;
}

template <int COLS>
cudaError_t launch(const CUtensorMap &map, TcArgs m, int stages, int sms, cudaStream_t st) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(q4_tc_kernel<COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    m.slice_stages = (stages + m.slices - 1) / m.slices;
    m.ring = std::min(kMaxRing, (kMaxSmem - smem_bytes<COLS>(m.slice_stages, 0)) / kStage);
    const int groups = m.slices > 1 ? m.tiles : std::min(m.tiles, sms);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(m.slices);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(groups * m.slices));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(smem_bytes<COLS>(m.slice_stages, m.ring));
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = m.slices > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q4_tc_kernel<COLS>, map, m);
}

template <int COLS>
bool fits(int stages, int slices) { return smem_bytes<COLS>((stages + slices - 1) / slices, kMinRing) <= kMaxSmem; }

}  // namespace

// All rows in passes of up to 64 on the tensor cores; false if this shape is not theirs.
bool run_tc(const Q4Args &a, float step, int twice_j0, int sms, cudaStream_t st, cudaError_t *err) {
    if (a.q_block < 64 || a.K % 32) return false;
    const int stages = (a.K + kIn - 1) / kIn, tiles = (a.N + kOut - 1) / kOut;
    TcArgs m{};
    m.a = a;
    m.tiles = tiles;
    while ((64 << m.shift) < a.q_block) ++m.shift;
    m.centre = 16.f + 0.5f * float(twice_j0);
    m.step = step;
    m.wait_ns = wait_limit_ns();
    m.extra_need = debug_extra_need();
    // Rows of a pass and slices of the inputs, by the time they should take (us, measured at 2048
    // inputs): a stage 0.45, 0.5 or 0.7 for 16, 32 or 64 columns, 4 to bring 32768 elements of x into
    // place, 6 to start and end a CTA.  Unsliced CTAs go through several tiles with one x; sliced ones
    // hold one tile, and clusters of 8 and 4 find places for fewer CTAs than there are SMs.
    int cols_max = 0;
    double best = 1e30;
    for (int cols = 16; cols <= 64; cols *= 2)
        for (int slices = 1; slices <= kMaxSlices && (slices == 1 || stages >= 2 * slices); slices *= 2) {
            const bool ok = cols == 64 ? fits<64>(stages, slices) : cols == 32 ? fits<32>(stages, slices) : fits<16>(stages, slices);
            if (!ok || (cols > 16 && cols / 2 >= a.T)) continue;
            const double stage = cols == 64 ? 0.7 : cols == 32 ? 0.5 : 0.45;
            const double part = double((stages + slices - 1) / slices), x = 4.0 * cols * part * kIn / 32768;
            const int places = slices == 8 ? 96 : slices == 4 ? 128 : sms;
            const double rounds = std::ceil(double(tiles) * slices / places);
            const double t = std::ceil(double(a.T) / cols) * (slices == 1 ? rounds * part * stage + x + 6 : rounds * (part * stage + x + 6));
            if (t < best) {
                best = t;
                cols_max = cols;
                m.slices = slices;
            }
        }
    if (cols_max == 0) return false;
    CUtensorMap map;
    if (!make_map(&map, a.codes, (uint64_t)a.N, (uint64_t)a.K / 2, kOut, kIn / 2, true, true)) return false;
    *err = cudaSuccess;
    for (int t0 = 0; t0 < a.T && *err == cudaSuccess; t0 += cols_max) {
        m.T0 = t0;
        m.rows = std::min(a.T - t0, cols_max);
        *err = m.rows <= 16   ? launch<16>(map, m, stages, sms, st)
               : m.rows <= 32 ? launch<32>(map, m, stages, sms, st)
                              : launch<64>(map, m, stages, sms, st);
    }
    return true;
}

cudaError_t read_error(int32_t *code, cudaStream_t st) {
    void *p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_err);
    if (e == cudaSuccess) e = cudaMemcpyAsync(code, p, sizeof *code, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(p, 0, sizeof *code, st);
    return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

}  // namespace q4
}  // namespace moe
