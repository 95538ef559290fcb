// q4_linear.cu -- out = x . W^T (+ residual) with 4-bit weights (codes, one bf16 scale per
// q_block inputs, a 16-entry codebook), for batches of few rows.  What bounds it is the read of
// the codes, half a byte a weight, and next to it the instructions that unpack them.
//
// q4_mma_kernel: a CTA takes 16 outputs at a time.  Its eight warps split the inputs; each
// streams its part of the 16 code rows through a cp.async ring of its own, 64 inputs a stage,
// unpacks the codes in registers to the A operand of mma.sync (m16n8k16, outputs x inputs) and
// multiplies with the rows of x, which lie in shared memory in the order of the B fragments.
// A block of inputs that shares a scale is summed by the MMA alone, then added to the fp32
// result with the scale: the scales cost one multiply-add an output and block, and no weight is
// rounded.  The warps' sums are added in a fixed order.
#include "attn.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <cstring>

namespace moe {
namespace {

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

// ---------------------------------------------------------------- any q_block
constexpr int kAnyThreads = 128;
constexpr int kAnyRows = 8;  // rows of x of one pass over the weights

// One warp an output: lanes take 8-element words of the row, fp32 throughout.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads) q4_any_kernel(Q4Args a) {
    __shared__ float book[16];
    if (threadIdx.x < 16) book[threadIdx.x] = a.codebook[threadIdx.x];
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int n = blockIdx.x * (kAnyThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t0 = blockIdx.y * kAnyRows, rows = min(kAnyRows, a.T - t0);
    if (n >= a.N) return;
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(a.codes + (size_t)n * (a.K / 2));
    const uint16_t *scales = a.scales + (size_t)n * (a.K / a.q_block);
    float acc[kAnyRows] = {};
    for (int w = lane; w < a.K / 8; w += 32) {
        const uint32_t c = __ldg(codes + w);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {  // q_block is even: a pair shares its scale
            const float s = bf16_bits_to_f32(__ldg(scales + (w * 8 + e) / a.q_block));
            v[e] = book[(c >> (4 * e)) & 15] * s;
            v[e + 1] = book[(c >> (4 * e + 4)) & 15] * s;
        }
#pragma unroll
        for (int r = 0; r < kAnyRows; ++r) {
            if (r < rows) {
                float xv[8];
                attn::ldp8(a.x + (t0 + r) * a.x_stride + w * 8, xv);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[r] = fmaf(v[e], xv[e], acc[r]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kAnyRows; ++r) {
        if (r < rows) {
            float y = warp_sum(acc[r]);
            if (lane == 0) {
                if (a.res) y += bf16_bits_to_f32(ldp(a.res + (t0 + r) * a.res_stride + n));
                attn::from_f32(y, static_cast<T *>(a.out) + (t0 + r) * a.out_stride + n);
            }
        }
    }
}

cudaError_t launch_any(const Q4Args &a, int out_dtype, cudaStream_t st) {
    const dim3 block(kAnyThreads);
    // grid.y is at most 65535: 2^18 rows make 32768
    const dim3 grid((a.N + kAnyThreads / 32 - 1) / (kAnyThreads / 32), (a.T + kAnyRows - 1) / kAnyRows);
    return out_dtype == MOE_DT_F32 ? launch_pdl(q4_any_kernel<float>, grid, block, 0, st, a)
                                   : launch_pdl(q4_any_kernel<uint16_t>, grid, block, 0, st, a);
}

// ---------------------------------------------------------------- tensor cores, q_block a multiple of 32
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kOut = 16;         // outputs of a tile
constexpr int kIn = 64;          // inputs of a stage
constexpr int kDepth = 8;        // stages of a warp's ring
constexpr int kCodeBytes = kOut * kIn / 2, kScaleBytes = kOut * 2 * 4, kStageBytes = kCodeBytes + kScaleBytes;
constexpr int kRingBytes = kWarps * kDepth * kStageBytes;
constexpr int kLutBytes = 256 * 32 * 8;
constexpr int kMaxSlices = 8;    // CTAs of a cluster that split the inputs
constexpr int kMaxSmem = 232448;

struct MmaArgs {
    Q4Args a;
    int T0, rows;       // rows of x of this launch
    int slices;         // cluster size
    int tiles;          // output tiles
    int slice_stages;   // the most stages of 64 inputs that one CTA has
    uint64_t per_block; // ceil(2^32 / m), q_block = 32 m: 32-input part j lies in block (j * per_block) >> 32
    uint32_t centre;    // affine codebook: bf16x2 of 16 + j0
    float step;         // affine codebook: its step; else 1
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (w & 0x00780078) | 0x41804180: two codes, already shifted to bits 3 .. 6 of each half, become
// the bf16 pair 16 + j; minus 16 + j0 that is j - j0, every step exact.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t mask, uint32_t bias, uint32_t centre) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tlop3.b32 t, %1, %2, %3, 0xEA;\n\tsub.rn.bf16x2 %0, t, %4;\n\t}"
        : "=r"(r) : "r"(w), "r"(mask), "r"(bias), "r"(centre));
    return r;
}

// NT: 8-row tiles of x.  kFine: scales may change every 32 inputs (else every 64 or more).
// kAffine: codebook step * (j - j0); else a table in shared memory, each value as bf16 hi + lo.
template <int NT, bool kFine, bool kAffine>
__global__ void __launch_bounds__(kThreads) q4_mma_kernel(const __grid_constant__ MmaArgs m) {
    namespace cg = cooperative_groups;
    constexpr int kCols = NT * 8;
    constexpr int kRedBufs = NT <= 2 ? 2 : 1;
    extern __shared__ __align__(128) unsigned char smem[];
    const Q4Args &a = m.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    float *red = reinterpret_cast<float *>(smem);                        // [kRedBufs][kWarps][kCols][kOut]
    float *part = red + kRedBufs * kWarps * kCols * kOut;                // [2][kCols][kOut]
    unsigned char *ring_base = reinterpret_cast<unsigned char *>(part + 2 * kCols * kOut);
    unsigned char *lut = ring_base + kRingBytes;
    unsigned char *xs = lut + (kAffine ? 0 : kLutBytes);                 // [stage][NT][2][32] x 16 bytes
    const uint32_t ring = smem_addr(ring_base) + warp * kDepth * kStageBytes;

    // this CTA's stages of the inputs, and this warp's
    const int stages = (a.K + kIn - 1) / kIn;
    const int slice = int(blockIdx.x) % m.slices, group = int(blockIdx.x) / m.slices, groups = int(gridDim.x) / m.slices;
    const int s0 = int((int64_t)stages * slice / m.slices), s1 = int((int64_t)stages * (slice + 1) / m.slices);
    const int w0 = s0 + (s1 - s0) * warp / kWarps, w1 = s0 + (s1 - s0) * (warp + 1) / kWarps, mine = w1 - w0;
    const int my_tiles = (m.tiles - group + groups - 1) / groups;
    const int total = mine * my_tiles;

    // the block of inputs [32 j, 32 j + 32)
    auto block_of = [&](int j) { return uint32_t(uint64_t(j) * m.per_block >> 32); };

    // the ring: copies run kDepth - 1 stages ahead, across tiles
    const int blocks = a.K / a.q_block;
    int p_tile = group, p_stage = 0;
    const int crow = lane >> 1, chalf = lane & 1;
    auto copy = [&](int i) {
        if (i < total) {
            const uint32_t dst = ring + (i % kDepth) * kStageBytes;
            const int k = (w0 + p_stage) * kIn;
            const int n = p_tile * kOut + crow;
            const bool on = n < a.N && k + chalf * 32 < a.K;
            cp16(dst + lane * 16, a.codes + (on ? (size_t)n * (a.K / 2) + k / 2 + chalf * 16 : 0), on ? 16 : 0);
            // scales of the rows: one of each 32 inputs when they may differ there, else one a stage.
            // 2 bytes each; the copy writes 4, the rest zero
            if (kFine || chalf == 0) {
                const size_t e = (size_t)n * blocks + block_of(k / 32 + chalf);
                const size_t word = on ? e & ~size_t(1) : 0;
                cp4(dst + kCodeBytes + lane * 4, a.scales + word, on ? ((e & 1) ? 4 : 2) : 0);
            }
            if (++p_stage == mine) {
                p_stage = 0;
                p_tile += groups;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) copy(i);  // weights: no kernel of the library writes them

    if constexpr (!kAffine) {
        for (int v = warp; v < 256; v += kWarps) {
            const float c0 = a.codebook[v & 15], c1 = a.codebook[v >> 4];
            const uint32_t hi = attn::pack_bf16(c0, c1);
            const float l0 = c0 - __uint_as_float(hi << 16), l1 = c1 - __uint_as_float(hi & 0xffff0000u);
            *reinterpret_cast<uint2 *>(lut + v * 256 + lane * 8) = make_uint2(hi, attn::pack_bf16(l0, l1));
        }
    }
    griddep_wait();
    griddep_launch_dependents();
    // x into the order of the B fragments: 8 inputs of one row are one 16-byte piece, for lane
    // (row mod 8, t) of word wi.  A lane's two code words hold inputs 16 t + 8 wi (one scale a
    // stage) or 32 wi + 8 t (one each 32); the affine path unpacks codes i and i + 4 together.
    const int n8 = (s1 - s0) * (kIn / 8);
    for (int i = tid; i < n8 * kCols; i += kThreads) {
        const int c = i % n8, row = i / n8;
        const int k = s0 * kIn + c * 8, st = c / 8, o = c % 8;
        const int wi = kFine ? o / 4 : o & 1, tt = kFine ? o & 3 : o / 2;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < m.rows && k < a.K) v = ldp16(a.x + (m.T0 + row) * a.x_stride + k);
        if (kAffine)
            v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                           __byte_perm(v.y, v.w, 0x7632));
        *reinterpret_cast<uint4 *>(xs + ((((size_t)st * NT + row / 8) * 2 + wi) * 32 + (row & 7) * 4 + tt) * 16) = v;
    }
    __syncthreads();

    const uint32_t xa = smem_addr(xs) + lane * 16, la = smem_addr(lut) + lane * 8;
    const uint32_t mask = 0x00780078u, bias = 0x41804180u, centre = m.centre;
    int i = 0;
    for (int k = 0; k < my_tiles; ++k) {
        const int tile = group + k * groups;
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
        for (int st = w0; st < w1; ++st, ++i) {
            copy(i + kDepth - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            __syncwarp();
            const uint32_t at = ring + (i % kDepth) * kStageBytes;
            uint32_t w[2][2];  // [word][row g, g + 8]
            float sc[2][2];    // [word][row g, g + 8]
            if (kFine) {
#pragma unroll
                for (int wi = 0; wi < 2; ++wi)
#pragma unroll
                    for (int r = 0; r < 2; ++r) w[wi][r] = lds32(at + (g + 8 * r) * 32 + wi * 16 + t * 4);
            } else {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint2 v = lds64(at + (g + 8 * r) * 32 + t * 8);
                    w[0][r] = v.x;
                    w[1][r] = v.y;
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int wi = 0; wi < (kFine ? 2 : 1); ++wi) {
                    const uint32_t word = lds32(at + kCodeBytes + ((g + 8 * r) * 2 + wi) * 4);
                    // which half of the copied word: the parity of the scale's index
                    const uint32_t e = uint32_t(tile * kOut + g + 8 * r) * uint32_t(blocks) + block_of(st * 2 + wi);
                    sc[wi][r] = __uint_as_float((e & 1) ? word & 0xffff0000u : word << 16) * m.step;
                }
            float c[NT][4];
#pragma unroll
            for (int wi = 0; wi < 2; ++wi) {
                if (wi == 0 || kFine) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[n][e] = 0.f;
                }
                uint32_t p[2][4], q[2][4];  // [row][pair]; q: the low parts of a table's values
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t v = w[wi][r];
                    if (kAffine) {
                        p[r][0] = code_pair(v << 3, mask, bias, centre);
                        p[r][1] = code_pair(v >> 1, mask, bias, centre);
                        p[r][2] = code_pair(v >> 5, mask, bias, centre);
                        p[r][3] = code_pair(v >> 9, mask, bias, centre);
                    } else {
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const uint2 h = lds64(la + ((v >> (8 * b)) & 255u) * 256);
                            p[r][b] = h.x;
                            q[r][b] = h.y;
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 x = lds128(xa + (((st - s0) * NT + n) * 2 + wi) * 512);
                    mma16816(c[n], p[0][0], p[1][0], p[0][1], p[1][1], x.x, x.y);
                    mma16816(c[n], p[0][2], p[1][2], p[0][3], p[1][3], x.z, x.w);
                    if (!kAffine) {
                        mma16816(c[n], q[0][0], q[1][0], q[0][1], q[1][1], x.x, x.y);
                        mma16816(c[n], q[0][2], q[1][2], q[0][3], q[1][3], x.z, x.w);
                    }
                }
                if (kFine || wi == 1) {
                    const float f0 = sc[kFine ? wi : 0][0], f1 = sc[kFine ? wi : 0][1];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        acc[n][0] = fmaf(f0, c[n][0], acc[n][0]);
                        acc[n][1] = fmaf(f0, c[n][1], acc[n][1]);
                        acc[n][2] = fmaf(f1, c[n][2], acc[n][2]);
                        acc[n][3] = fmaf(f1, c[n][3], acc[n][3]);
                    }
                }
            }
            __syncwarp();  // the stage is read before the next copy lands in it
        }
        // the warps' sums, [column][output]; lane (g, t): outputs g and g + 8 of columns 2 t, 2 t + 1
        float *rb = red + (kRedBufs == 2 ? (k & 1) * kWarps * kCols * kOut : 0);
        if (kRedBufs == 1 && k > 0) __syncthreads();  // the tile before has been read
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                rb[(warp * kCols + n * 8 + 2 * t + (e & 1)) * kOut + g + 8 * (e >> 1)] = acc[n][e];
        __syncthreads();
        float *pb = part + (k & 1) * kCols * kOut;
        auto emit = [&](int idx, float y) {
            const int row = idx / kOut, n = tile * kOut + idx % kOut;
            if (row >= m.rows || n >= a.N) return;
            const int64_t tr = m.T0 + row;
            if (a.res) y += bf16_bits_to_f32(ldp(a.res + tr * a.res_stride + n));
            if (a.out_f32)
                static_cast<float *>(a.out)[tr * a.out_stride + n] = y;
            else
                static_cast<uint16_t *>(a.out)[tr * a.out_stride + n] = f32_to_bf16_bits(y);
        };
        for (int idx = tid; idx < kCols * kOut; idx += kThreads) {
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) y += rb[w * kCols * kOut + idx];
            if (m.slices == 1)
                emit(idx, y);
            else
                pb[idx] = y;
        }
        if (m.slices > 1) {
            // each CTA of the cluster adds the slices of its part of the outputs, in order; the
            // other buffer is written meanwhile, so one barrier a tile is enough
            cg::cluster_group cl = cg::this_cluster();
            cl.sync();
            for (int idx = slice * kThreads + tid; idx < kCols * kOut; idx += m.slices * kThreads) {
                float y = 0.f;
                for (int r = 0; r < m.slices; ++r) y += *cl.map_shared_rank(pb + idx, r);
                emit(idx, y);
            }
        }
    }
    if (m.slices > 1) cg::this_cluster().sync();  // no CTA leaves while another reads its sums
}

template <int NT, bool kFine, bool kAffine>
int mma_smem(int slice_stages) {
    const int red = (NT <= 2 ? 2 : 1) * kWarps * NT * 8 * kOut * 4, part = 2 * NT * 8 * kOut * 4;
    return red + part + kRingBytes + (kAffine ? 0 : kLutBytes) + slice_stages * NT * 2 * 32 * 16;
}

template <int NT, bool kFine, bool kAffine>
cudaError_t launch_mma(MmaArgs m, int sms, cudaStream_t st) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(q4_mma_kernel<NT, kFine, kAffine>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int smem = mma_smem<NT, kFine, kAffine>(m.slice_stages);
    const int per_sm = std::min(4, std::max(1, (kMaxSmem - 1024) / (smem + 1024)));
    const int groups = std::max(1, std::min(m.tiles, sms * per_sm / m.slices));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(m.slices);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(groups * m.slices));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = m.slices > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q4_mma_kernel<NT, kFine, kAffine>, m);
}

template <int NT>
cudaError_t launch_nt(const MmaArgs &m, bool fine, bool affine, int sms, cudaStream_t st) {
    if (affine) return fine ? launch_mma<NT, true, true>(m, sms, st) : launch_mma<NT, false, true>(m, sms, st);
    return fine ? launch_mma<NT, true, false>(m, sms, st) : launch_mma<NT, false, false>(m, sms, st);
}

// The most stages of x that fit next to the rest for NT tiles of 8 rows.
int max_stages(int nt, bool affine) {
    const int fixed = (nt <= 2 ? 2 : 1) * kWarps * nt * 8 * kOut * 4 + 2 * nt * 8 * kOut * 4 + kRingBytes +
                      (affine ? 0 : kLutBytes);
    return (kMaxSmem - fixed) / (nt * 1024);
}

// The rows in passes of up to 64 (fewer when x would not fit even split over a cluster); false
// if not even 8 rows fit.
bool run_mma(const Q4Args &a, int sms, cudaStream_t st, cudaError_t *err) {
    float step = 1.f;
    int twice = 0;
    const bool affine = q4_codebook_affine(a.codebook, &step, &twice);
    const bool fine = a.q_block % kIn != 0;
    const int stages = (a.K + kIn - 1) / kIn, tiles = (a.N + kOut - 1) / kOut;
    int nt_max = 8;
    while (nt_max > 0 && (stages + kMaxSlices - 1) / kMaxSlices > max_stages(nt_max, affine)) nt_max /= 2;
    if (nt_max == 0) return false;
    MmaArgs m{};
    m.a = a;
    m.tiles = tiles;
    m.step = affine ? step : 1.f;
    const uint32_t per = uint32_t(a.q_block / 32);
    m.per_block = ((uint64_t(1) << 32) + per - 1) / per;
    const float c = 16.f + 0.5f * float(twice);  // 6 significant bits: exact in bf16
    uint32_t bits;
    memcpy(&bits, &c, 4);
    m.centre = (bits & 0xffff0000u) | bits >> 16;
    *err = cudaSuccess;
    for (int t0 = 0; t0 < a.T && *err == cudaSuccess; t0 += nt_max * 8) {
        m.T0 = t0;
        m.rows = std::min(a.T - t0, nt_max * 8);
        const int nt = m.rows <= 8 ? 1 : m.rows <= 16 ? 2 : m.rows <= 32 ? 4 : 8;
        // slices: as many as x needs to fit; more while there are fewer CTAs than SMs and every
        // warp keeps two stages
        int slices = 1;
        while ((stages + slices - 1) / slices > max_stages(nt, affine)) slices *= 2;
        while (slices < kMaxSlices && tiles * slices * 2 <= sms * 2 && stages >= slices * 2 * 2 * kWarps) slices *= 2;
        m.slices = slices;
        m.slice_stages = (stages + slices - 1) / slices;
        *err = nt == 1   ? launch_nt<1>(m, fine, affine, sms, st)
               : nt == 2 ? launch_nt<2>(m, fine, affine, sms, st)
               : nt == 4 ? launch_nt<4>(m, fine, affine, sms, st)
                         : launch_nt<8>(m, fine, affine, sms, st);
    }
    return true;
}

}  // namespace

cudaError_t launch_q4_linear(const moe_q4_linear_shape &s, const void *x, int64_t x_stride, const moe_q4_weight &w,
                             const void *res, int64_t res_stride, void *out, int64_t out_stride, int sms, cudaStream_t st) {
    Q4Args a{};
    a.x = static_cast<const uint16_t *>(x);
    a.codes = static_cast<const uint8_t *>(w.codes);
    a.scales = static_cast<const uint16_t *>(w.scales);
    a.res = static_cast<const uint16_t *>(res);
    a.out = out;
    a.x_stride = x_stride;
    a.res_stride = res_stride;
    a.out_stride = out_stride;
    a.T = s.T;
    a.K = s.K;
    a.N = s.N;
    a.q_block = s.q_block;
    a.out_f32 = s.out_dtype == MOE_DT_F32;
    for (int i = 0; i < 16; ++i) a.codebook[i] = w.codebook[i];
    // code rows in 16-byte pieces, blocks that cover whole halves of a stage, 32-bit counts and an
    // exact division by the block's size (j m < 2^32)
    cudaError_t err;
    if (s.q_block % 32 == 0 && (uint64_t)(s.K / 32) * (s.q_block / 32) < (uint64_t(1) << 32) && (int64_t)((s.N + kOut - 1) / kOut) * ((s.K + kIn - 1) / kIn) < INT32_MAX &&
        run_mma(a, sms, st, &err))
        return err;
    return launch_any(a, s.out_dtype, st);
}

}  // namespace moe
