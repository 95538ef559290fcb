// q4_linear.cu -- out = x . W^T (+ residual) with 4-bit weights (codes, one bf16 scale per
// q_block inputs, a 16-entry codebook), for batches of few rows.  What bounds it is the read of
// the codes, half a byte a weight, and next to it the instructions that unpack them.
//
// q4_mma_kernel: a CTA takes 16 outputs at a time (16 to 128 where there are more, "side").  Its
// eight warps split the inputs; where there are many outputs, sixteen warps take pairs of 16 instead,
// each an equal piece of the line of all the CTA's pairs (16 rows x 2048 x 131072: 39.6 us; tiles whose inputs
// the warps split, with a barrier and a sum each, 54).  Each warp
// streams its part of the code rows through a cp.async ring of its own, 128 inputs a stage,
// unpacks the codes in registers to the A operand of mma.sync (m16n8k16, outputs x inputs) and
// multiplies with the rows of x, which lie in shared memory in the order of the B fragments.
// A block of inputs that shares a scale is summed by the MMA alone, then added to the fp32
// result with the scale: the scales cost one multiply-add an output and block, and no weight is
// rounded.  The warps' sums are added in a fixed order.
#include "q4_linear.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

namespace moe {
namespace q4 {
namespace {

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
        const uint32_t c = codes[w];
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {  // q_block is even: a pair shares its scale
            const float s = bf16_bits_to_f32(scales[(w * 8 + e) / a.q_block]);
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

// ---------------------------------------------------------------- tensor cores
constexpr int kStrip = 16;       // outputs of an MMA
constexpr int kIn = 128;         // inputs of a stage, two halves of 64
constexpr int kMaxSlices = 8;    // CTAs of a cluster that split the inputs
constexpr int kMaxSmem = 232448;
constexpr int kLutBytes = 256 * 32 * 8, kThirdBytes = 256 * 32 * 4;

// What a variant's shared memory holds.  NT: 8-row tiles of x; MT: strips of 16 outputs a warp works
// on, 1 or 2: two read each fragment of x once, and share the cost of a stage's copies.
template <int NT, int MT, bool kFine, int kParts>
struct Var {
    static constexpr bool kAffine = kParts == 0;
    static constexpr int kWarps = MT == 2 ? 16 : 8, kThreads = kWarps * 32;
    static constexpr int kDepth = MT == 2 || NT == 2 ? 3 : 4;  // stages of a warp's ring
    static constexpr int kOut = MT * kStrip;                 // outputs of a warp
    static constexpr int kCols = NT * 8;                     // rows of x
    static constexpr int kCodes = kOut * kIn / 2;            // code bytes of a stage
    static constexpr int kScalesRow = kFine ? 4 : 2;         // scale words of an output
    static constexpr int kStage = kCodes + kOut * kScalesRow * 4;
    static constexpr int kRedStride = kOut + 4;              // padded column of sums: no bank conflicts
    static constexpr int kRed = MT == 2 ? kWarps * MT * NT * 512 : kWarps * kCols * kRedStride * 4;
    static constexpr int kRing = kWarps * kDepth * kStage;
    static constexpr int kLut = kAffine ? 0 : kLutBytes + (kParts == 3 ? kThirdBytes : 0);
    static constexpr int kFixed = kRed + kRing + kLut;
    // 64 inputs of x: the fragments, and per block the start values (twice each, see below)
    static constexpr int kHalf = NT * 1024 + (kAffine ? (kFine ? 2 : 1) * NT * 64 : 0);
    static int part_bytes(int side) { return 2 * kCols * side * kOut * 4; }
    static int max_stages() { return (kMaxSmem - kFixed) / (2 * kHalf); }                           // of one CTA
    static int max_stages_sliced() { return (kMaxSmem - kFixed - part_bytes(kWarps)) / (2 * kHalf); }  // of a cluster's
};

constexpr int kMmaRows = 16;     // rows of x of a pass

struct MmaArgs {
    Q4Args a;
    int pass_rows;      // rows of x of a pass: grid.y passes read the weights side by side
    int slices;         // cluster size
    int side;           // output strips side by side in a CTA: its warps are side x (warps / side input parts)
    int tiles;          // tiles of side strips
    int slice_halves;   // the most 64-input halves that one CTA has
    int shift;          // log2(q_block / 64) (not fine)
    float centre;       // affine codebook: 16 + j0
    float step;         // affine codebook: its step; else 1
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// Plain loads and MMAs without `volatile`: the compiler may move them past one another (the waits
// for copies are barriers to it), so that a warp's loads, unpacking and products overlap.
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    return *reinterpret_cast<const uint32_t *>(__cvta_shared_to_generic(addr));
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    return *reinterpret_cast<const uint2 *>(__cvta_shared_to_generic(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    return *reinterpret_cast<const uint4 *>(__cvta_shared_to_generic(addr));
}
__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with another addend: starts a sum.
__device__ __forceinline__ void mma16816_from(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, const uint4 &z) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %11, %12, %13};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(__uint_as_float(z.x)),
                   "f"(__uint_as_float(z.y)), "f"(__uint_as_float(z.z)), "f"(__uint_as_float(z.w)));
}
// NT: 8-row tiles of x.  kFine: q_block 32, four blocks a stage; else 64 times a power of two.
// kParts 0, affine: codebook step * (j - j0).  The MMA multiplies the exact integers 16 + j, and each sum
// starts at -(16 + j0) sum x of its block (fp32, found once a CTA), which leaves sum (j - j0) x: the
// subtraction costs no instruction, and about a factor 5 of the fp32 sum's accuracy (16 + j
// against j - j0).  Else a table in shared memory, each value as kParts bf16 that add up to it: two
// (16 bits, 2^-17 of a value, for results that are rounded to bf16's 2^-8) or three (24 bits, for fp32).
template <int NT, int MT, bool kFine, int kParts>
__global__ void __launch_bounds__(Var<NT, MT, kFine, kParts>::kThreads)
q4_mma_kernel(const __grid_constant__ MmaArgs m) {
    namespace cg = cooperative_groups;
    using V = Var<NT, MT, kFine, kParts>;
    constexpr bool kAffine = V::kAffine;
    constexpr int kWarps = V::kWarps, kThreads = V::kThreads, kDepth = V::kDepth, kOut = V::kOut, kCols = V::kCols;
    constexpr int kStage = V::kStage, kRedStride = V::kRedStride, kRowBytes = kIn / 2;
    extern __shared__ __align__(128) unsigned char smem[];
    const Q4Args &a = m.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    float *red = reinterpret_cast<float *>(smem);  // [kWarps][kCols][kRedStride]
    unsigned char *ring_base = smem + V::kRed;
    unsigned char *lut = ring_base + V::kRing;
    unsigned char *xs = lut + V::kLut;  // [half][NT][2][32] x 16 bytes
    unsigned char *starts = xs + (size_t)m.slice_halves * NT * 1024;  // [block][NT][4] x 16 bytes (affine)
    float *part = reinterpret_cast<float *>(xs + (size_t)m.slice_halves * V::kHalf);  // [2][kCols][wide], slices > 1
    const uint32_t ring = smem_addr(ring_base) + warp * kDepth * kStage;

    const int T0 = blockIdx.y * m.pass_rows, rows = min(a.T - T0, m.pass_rows);

    const int stages = (a.K + kIn - 1) / kIn;
    // MT 1: this CTA's stages of the inputs, and this warp's, the same in each of the CTA's tiles.
    const int slice = int(blockIdx.x) % m.slices, group = int(blockIdx.x) / m.slices, groups = int(gridDim.x) / m.slices;
    const int s0 = int((int64_t)stages * slice / m.slices), s1 = int((int64_t)stages * (slice + 1) / m.slices);
    const int parts = kWarps / m.side, beside = warp % m.side, in_part = warp / m.side;
    const int wide = m.side * kOut, wide_log2 = __ffs(wide) - 1;
    // MT 2: the CTA's pairs of strips are a line of stages, and each warp takes an equal piece of it.
    // Its first pair may have been begun by the warps before, its last be ended by those after.
    const int pair0 = int((int64_t)m.tiles * blockIdx.x / gridDim.x);
    const int line = (int((int64_t)m.tiles * (blockIdx.x + 1) / gridDim.x) - pair0) * stages;
    auto line_at = [&](int w) { return int((int64_t)line * w / kWarps); };
    const int u0 = line_at(warp), u1 = line_at(warp + 1);
    const int w0 = MT == 2 ? u0 % stages : s0 + (s1 - s0) * in_part / parts;
    const int w1 = MT == 2 ? stages : s0 + (s1 - s0) * (in_part + 1) / parts, mine = w1 - w0;
    const int my_tiles = (m.tiles - group + groups - 1) / groups;

    // The ring: copies run kDepth - 1 stages ahead, across tiles.  Piece (lane mod 4) of row lane / 4
    // (+ 8 i) is 16 bytes; the pieces of a row are permuted so that the reads below have no bank
    // conflicts.  The scales of row lane / 2 (+ 16 i), half lane % 2 are copied with the aligned word
    // they lie in (2 bytes of it at the array's end), the reader picks the half by the index's parity.
    const uint32_t blocks = uint32_t(a.K / a.q_block);
    const size_t row_bytes = a.K / 2, row8 = 8 * row_bytes;
    const int crow = lane >> 2, cpiece = lane & 3, srow = lane >> 1, shalf = lane & 1;
    int p_n = MT == 2 ? (pair0 + u0 / stages) * kOut : group * wide + beside * kOut;
    int p_stage = w0, left = MT == 2 ? u1 - u0 : mine * my_tiles;
    const uint8_t *src = a.codes + (size_t)(p_n + crow) * row_bytes + (size_t)w0 * kRowBytes + cpiece * 16;
    const int tile_step = MT == 2 ? kOut : groups * wide, again = MT == 2 ? stages : mine;
    const size_t tile_skip = (size_t)tile_step * row_bytes - (size_t)again * kRowBytes;
    uint32_t sbase = uint32_t(p_n + srow) * blocks;
    const uint32_t ring_end = ring + kDepth * kStage;
    uint32_t dst = ring;
    const uint32_t code_at = crow * kRowBytes + ((cpiece ^ (crow >> 1 & 3)) * 16);  // row + 8: same permutation
    const int K = a.K, N = a.N, shift = m.shift;
    // whole stages of whole tiles with one or two scales a half advance by constants; what is cut by
    // the matrix's edge, or has wider blocks, is worked out
    const bool simple = K % kIn == 0 && (kFine || shift == 0);
    bool inside = simple && p_n + kOut <= N;
    constexpr int kScaleStep = kFine ? 8 : 4;  // bytes of a row's scales in a stage
    const char *scales = reinterpret_cast<const char *>(a.scales);
    const size_t strip_scales = (size_t)kStrip * blocks * 2;
    const uint32_t e0 = sbase + (kFine ? w0 * 4 + shalf * 2 : w0 * 2 + shalf);
    const char *ssrc = scales + (size_t)(e0 & ~1u) * 2;
    const size_t scale_skip = (size_t)tile_step * blocks * 2 - (size_t)again * kScaleStep;
    const int odd = e0 & 1;  // stages and tiles advance by even counts
    auto copy = [&]() {
        if (left > 0) {
            if (inside) {
                const uint8_t *s = src;
#pragma unroll
                for (int i = 0; i < kOut / 8; ++i, s += row8) cp16(dst + code_at + i * 8 * kRowBytes, s, 16);
                const char *q = ssrc;
#pragma unroll
                for (int i = 0; i < MT; ++i, q += strip_scales) {
                    const uint32_t to = dst + V::kCodes + (i * kStrip * 2 + lane) * (kFine ? 8 : 4);
                    cp4(to, q, odd ? 4 : 2);
                    if (kFine) cp4(to + 4, q + 4 * odd, odd ? 2 : 4);
                }
            } else {
                const bool in = p_stage * kIn + cpiece * 32 < K;
#pragma unroll
                for (int i = 0; i < kOut / 8; ++i) {
                    const bool ok = in && p_n + crow + i * 8 < N;
                    cp16(dst + code_at + i * 8 * kRowBytes, ok ? src + i * row8 : a.codes, ok ? 16 : 0);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int wi = 0; wi < (kFine ? 2 : 1); ++wi) {
                        const uint32_t e = sbase + i * kStrip * blocks +
                                           (kFine ? p_stage * 4 + shalf * 2 + wi : (p_stage * 2 + shalf) >> shift);
                        const bool ok = p_n + srow + i * kStrip < N && p_stage * kIn + shalf * 64 + wi * 32 < K;
                        cp4(dst + V::kCodes + (i * kStrip * 2 + lane) * (kFine ? 8 : 4) + wi * 4,
                            scales + (ok ? (size_t)(e & ~1u) * 2 : 0), ok ? 2 << (e & 1) : 0);
                    }
            }
            src += kRowBytes;
            ssrc += kScaleStep;
            dst += kStage;
            if (dst == ring_end) dst = ring;
            --left;
            if (++p_stage == w1) {
                p_stage = MT == 2 ? 0 : w0;
                p_n += tile_step;
                src += tile_skip;
                ssrc += scale_skip;
                sbase += uint32_t(tile_step) * blocks;
                inside = simple && p_n + kOut <= N;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (!kAffine) {
        for (int v = warp; v < 256; v += kWarps) {
            const float c0 = a.codebook[v & 15], c1 = a.codebook[v >> 4];
            const uint32_t hi = attn::pack_bf16(c0, c1);
            const float l0 = c0 - __uint_as_float(hi << 16), l1 = c1 - __uint_as_float(hi & 0xffff0000u);
            const uint32_t lo = attn::pack_bf16(l0, l1);
            *reinterpret_cast<uint2 *>(lut + v * 256 + lane * 8) = make_uint2(hi, lo);
            if (kParts == 3)
                *reinterpret_cast<uint32_t *>(lut + kLutBytes + v * 128 + lane * 4) =
                    attn::pack_bf16(l0 - __uint_as_float(lo << 16), l1 - __uint_as_float(lo & 0xffff0000u));
        }
    }
    // x in the order of the B fragments: 8 inputs of one row are one 16-byte piece, for lane (row mod 8,
    // t) of word wi of a 64-input half, inputs 32 wi + 8 t; the affine path unpacks codes i and i + 4
    // together.  Rows past the last are zero.
    const int n8 = (s1 - s0) * (kIn / 8);
    auto put = [&](int c, int row, uint4 v) {
        const int hf = c >> 3, wi = c >> 2 & 1, tt = c & 3;
        *reinterpret_cast<uint4 *>(xs + ((((size_t)hf * NT + row / 8) * 2 + wi) * 32 + (row & 7) * 4 + tt) * 16) = v;
    };
    // start values in the order of the accumulators: lane t, columns 2 t, 2 t + 1, for both rows
    constexpr int kPer = kFine ? 4 : 8;  // pieces of a block
    auto put_start = [&](int block, int row, float v) {
        float *z = reinterpret_cast<float *>(starts + ((size_t)block * NT + row / 8) * 64 + (row >> 1 & 3) * 16);
        z[row & 1] = z[2 + (row & 1)] = v;
    };
    for (int row = rows + warp; row < kCols; row += kWarps)
        for (int c = lane; c < n8; c += 32) {
            put(c, row, make_uint4(0, 0, 0, 0));
            if (kAffine && c % kPer == 0) put_start(c / kPer, row, 0.f);
        }
    // codes and scales too may be what the kernel before this one writes (a quantisation, a copy)
    griddep_wait();
    griddep_launch_dependents();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) copy();
    // the warps take the rows in turn, or where those are few, pieces of one: n8 is a multiple of 16,
    // so the lanes of a block stay together
    constexpr int kBatch = 4;  // loads in flight a thread
    const int beside_rows = rows < kWarps ? kWarps / rows : 1;  // warps on a row
    const int row_step = kWarps / beside_rows, c_step = beside_rows * 32;
    for (int row = warp / beside_rows; row < rows && warp < row_step * beside_rows; row += row_step) {
        const uint16_t *xr = a.x + (int64_t)(T0 + row) * a.x_stride + (int64_t)s0 * kIn;
        const int most = a.K - 8 - s0 * kIn;  // the last whole piece of the row
        for (int c0 = (warp % beside_rows) * 32 + lane; c0 < n8; c0 += kBatch * c_step) {
            uint4 v[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) v[b] = ldp16(xr + min((c0 + b * c_step) * 8, most));
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int c = c0 + b * c_step;
                if (c >= n8) break;  // whole groups of 16 lanes leave together
                if (c * 8 > most) v[b] = make_uint4(0, 0, 0, 0);
                if (kAffine) {
                    float f[8];
                    attn::unpack8(v[b], f);
                    float sum = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
                    const uint32_t group_mask = 0xffu << (lane & 24);
#pragma unroll
                    for (int w = 1; w < kPer; w <<= 1) sum += __shfl_xor_sync(group_mask, sum, w);
                    if (c % kPer == 0) put_start(c / kPer, row, -m.centre * sum);
                    const uint4 u = v[b];
                    v[b] = make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632),
                                      __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
                }
                put(c, row, v[b]);
            }
        }
    }
    __syncthreads();

    const uint32_t x0 = smem_addr(xs) + lane * 16, la = smem_addr(lut) + lane * 8,
                   l3 = smem_addr(lut) + kLutBytes + lane * 4;
    const uint32_t z0 = smem_addr(starts) + t * 16;
    const uint32_t mask = 0x00780078u, bias = 0x41804180u;
    // word wi of half hf of row g (+ 8): piece 2 hf + wi, word t
    uint32_t piece[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) piece[i] = g * kRowBytes + ((i ^ (g >> 1 & 3)) * 16) + t * 4;
    // The half of the copied word that holds a scale: by the parity of its index, the same for rows
    // g, g + 8, .. of every tile.
    const uint32_t g_odd = uint32_t(g) * blocks;
    uint32_t sel[2] = {g_odd & 1 ? kHigh : kLow, g_odd & 1 ? kLow : kHigh};  // q_block 32 or 64
    uint32_t at = ring;
    // Adds stage st (counted from the row's start) of the outputs in hand.
    auto stage = [&](int st, float (&acc)[MT][NT][4]) {
        const uint32_t xa = x0 + (st - s0) * (NT * 2048), za = z0 + (st - s0) * ((kFine ? 4 : 2) * NT * 64);
        copy();
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        __syncwarp();
        if (!kFine && shift > 0) sel[0] = sel[1] = (g_odd + ((st * 2) >> shift)) & 1 ? kHigh : kLow;
        float sc[MT][2][4];  // [strip][row g, g + 8][block of the stage]
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t sa = at + V::kCodes + (i * kStrip + g + 8 * r) * V::kScalesRow * 4;
                if (kFine) {
                    const uint4 v = lds128(sa);
                    sc[i][r][0] = half_of(v.x, sel[0]);
                    sc[i][r][1] = half_of(v.y, sel[1]);
                    sc[i][r][2] = half_of(v.z, sel[0]);
                    sc[i][r][3] = half_of(v.w, sel[1]);
                } else {
                    const uint2 v = lds64(sa);
                    sc[i][r][0] = half_of(v.x, sel[0]);
                    sc[i][r][1] = half_of(v.y, sel[1]);
                }
            }
        float c[MT][NT][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 32 inputs: word q & 1 of half q / 2
            const int block = kFine ? q : q / 2;
            const bool first = kFine || (q & 1) == 0, last = kFine || (q & 1) == 1;
            uint32_t p[MT][2][4], lo[MT][2][4], rest[MT][2][4];  // [strip][row][pair]; lo, rest: of a table's values
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t v = lds32(at + piece[q] + (i * kStrip + 8 * r) * kRowBytes);
                    if (kAffine) {
                        p[i][r][0] = code_pair(v << 3, mask, bias);
                        p[i][r][1] = code_pair(v >> 1, mask, bias);
                        p[i][r][2] = code_pair(v >> 5, mask, bias);
                        p[i][r][3] = code_pair(v >> 9, mask, bias);
                    } else {
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const uint2 h = lds64(la + ((v >> (8 * b)) & 255u) * 256);
                            p[i][r][b] = h.x;
                            lo[i][r][b] = h.y;
                            if (kParts == 3) rest[i][r][b] = lds32(l3 + ((v >> (8 * b)) & 255u) * 128);
                        }
                    }
                }
            uint4 x[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] = lds128(xa + (((q >> 1) * NT + n) * 2 + (q & 1)) * 512);
            // products on one accumulator are kept apart: each waits for the one before
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint4 z = make_uint4(0u, 0u, 0u, 0u);
                if (kAffine && first) z = lds128(za + (block * NT + n) * 64);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if (first)
                        mma16816_from(c[i][n], p[i][0][0], p[i][1][0], p[i][0][1], p[i][1][1], x[n].x, x[n].y, z);
                    else
                        mma16816(c[i][n], p[i][0][0], p[i][1][0], p[i][0][1], p[i][1][1], x[n].x, x[n].y);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    mma16816(c[i][n], p[i][0][2], p[i][1][2], p[i][0][3], p[i][1][3], x[n].z, x[n].w);
            if (!kAffine) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        mma16816(c[i][n], lo[i][0][0], lo[i][1][0], lo[i][0][1], lo[i][1][1], x[n].x, x[n].y);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        mma16816(c[i][n], lo[i][0][2], lo[i][1][2], lo[i][0][3], lo[i][1][3], x[n].z, x[n].w);
            }
            if (kParts == 3) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        mma16816(c[i][n], rest[i][0][0], rest[i][1][0], rest[i][0][1], rest[i][1][1], x[n].x, x[n].y);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        mma16816(c[i][n], rest[i][0][2], rest[i][1][2], rest[i][0][3], rest[i][1][3], x[n].z, x[n].w);
            }
            if (last) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[i][n][e] = fmaf(sc[i][e >> 1][block], c[i][n][e], acc[i][n][e]);
            }
        }
        at += kStage;
        if (at == ring_end) at = ring;
        __syncwarp();  // the stage is read before the next copy lands in it
    };
    auto clear = [](float (&acc)[MT][NT][4]) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;
    };
    if constexpr (MT == 2) {
        // A pair that one warp has whole goes out from its registers.  Of a pair that several share,
        // the one that begins it keeps its sums (they are its last), the others leave theirs in
        // `red`, and it adds those in order after the CTA's only barrier.
        float acc[MT][NT][4];
        auto emit_pair = [&](int n0) {
            bool finite = true;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        acc[i][n][e] *= m.step;
                        finite = finite && q4_is_finite(acc[i][n][e]);
                    }
            if (finite && !a.res && n0 + kOut <= N) {  // the usual case: one address a row
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int row = n * 8 + 2 * t + c;
                        if (row >= rows) continue;
                        const int64_t at_out = (T0 + row) * a.out_stride + n0 + g;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float y = acc[i][n][2 * r + c];
                                if (a.out_f32)
                                    static_cast<float *>(a.out)[at_out + i * kStrip + 8 * r] = y;
                                else
                                    static_cast<uint16_t *>(a.out)[at_out + i * kStrip + 8 * r] = f32_to_bf16_bits(y);
                            }
                    }
                return;
            }
            uint32_t again = 0;  // bit (n, c, i, r): a sum to be formed by its terms
            static_assert(NT * 4 * MT <= 32, "");
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = n * 8 + 2 * t + c;
                    if (row >= rows) continue;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int o = n0 + i * kStrip + 8 * r + g;
                            if (o < N && !q4_emit(a, T0 + row, o, acc[i][n][2 * r + c]))
                                again |= 1u << (((n * 2 + c) * MT + i) * 2 + r);
                        }
                }
            for (; again; again &= again - 1) {
                const int b = __ffs(again) - 1, r = b & 1, i = (b >> 1) % MT, c = (b >> 1) / MT & 1, n = (b >> 1) / MT / 2;
                q4_emit_by_terms(a, T0 + n * 8 + 2 * t + c, n0 + g + i * kStrip + 8 * r);
            }
        };
        int pending = -1, done = 0;  // the pair begun and not ended, and its stages
        for (int u = u0; u < u1;) {
            const int pair = u / stages, st0 = u - pair * stages, st1 = min(stages, st0 + u1 - u);
            clear(acc);
            for (int st = st0; st < st1; ++st) stage(st, acc);
            if (st0 > 0) {
                float4 *to = reinterpret_cast<float4 *>(red) + warp * (MT * NT * 32) + lane;
#pragma unroll
                for (int i = 0; i < MT * NT; ++i) {
                    const float *v = acc[i / NT][i % NT];
                    to[i * 32] = make_float4(v[0], v[1], v[2], v[3]);
                }
            } else if (st1 == stages) {
                emit_pair((pair0 + pair) * kOut);
            } else {
                pending = pair;
                done = st1;
            }
            u += st1 - st0;
        }
        __syncthreads();
        if (pending < 0) return;
        for (int w = warp + 1; done < stages; ++w) {
            const int theirs = line_at(w + 1) - line_at(w);
            if (theirs == 0) continue;
            const float4 *from = reinterpret_cast<const float4 *>(red) + w * (MT * NT * 32) + lane;
#pragma unroll
            for (int i = 0; i < MT * NT; ++i) {
                const float4 v = from[i * 32];
                float *to = acc[i / NT][i % NT];
                to[0] += v.x, to[1] += v.y, to[2] += v.z, to[3] += v.w;
            }
            done += theirs;
        }
        emit_pair((pair0 + pending) * kOut);
    } else {
        for (int k = 0; k < my_tiles; ++k) {
            const int n0 = (group + k * groups) * wide;
            float acc[MT][NT][4];
            clear(acc);
            for (int st = w0; st < w1; ++st) stage(st, acc);
            // the warps' sums, [column][output]; lane (g, t): outputs g and g + 8 of columns 2 t, 2 t + 1
            if (k > 0) __syncthreads();  // the tile before has been read
            float *rb = red + (warp * kCols + 2 * t) * kRedStride + g;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        rb[(n * 8 + (e & 1)) * kRedStride + i * kStrip + 8 * (e >> 1)] = acc[i][n][e];
            __syncthreads();
            float *pb = part + (k & 1) * kCols * wide;
            auto emit = [&](int row, int n, float y) {
                n += n0;
                if (row < rows && n < N && !q4_emit(a, T0 + row, n, y * m.step)) q4_emit_by_terms(a, T0 + row, n);
            };
            // output n of the tile is output n mod kOut of the warps beside = n / kOut, one an input part.
            // Threads are a multiple of the tile's outputs: a thread keeps its output, rows go by.
            {
                const uint32_t n = tid & (wide - 1), rows_step = kThreads >> wide_log2;
                const int cols = m.slices == 1 ? rows : kCols;
                const float *rr = red + (n / kOut * kCols) * kRedStride + n % kOut;
                const int part_step = m.side * kCols * kRedStride;
                for (int row = tid >> wide_log2; row < cols; row += rows_step) {
                    float y = rr[row * kRedStride];
                    for (int w = 1; w < parts; ++w) y += rr[row * kRedStride + w * part_step];
                    if (m.slices == 1)
                        emit(row, int(n), y);
                    else
                        pb[row * wide + n] = y;
                }
            }
            if (m.slices > 1) {
                // each CTA of the cluster adds the slices of its part of the outputs, in order; the
                // other buffer is written meanwhile, so one barrier a tile is enough
                cg::cluster_group cl = cg::this_cluster();
                cl.sync();
                for (int idx = slice * kThreads + tid; idx < kCols * wide; idx += m.slices * kThreads) {
                    float y = 0.f;
                    for (int r = 0; r < m.slices; ++r) y += *cl.map_shared_rank(pb + idx, r);
                    emit(idx >> wide_log2, idx & (wide - 1), y);
                }
            }
        }
        if (m.slices > 1) cg::this_cluster().sync();  // no CTA leaves while another reads its sums
    }
}

template <int NT, int MT, bool kFine, int kParts>
cudaError_t launch_mma(MmaArgs m, int stages, int sms, cudaStream_t st) {
    using V = Var<NT, MT, kFine, kParts>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(q4_mma_kernel<NT, MT, kFine, kParts>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int strips = (m.a.N + V::kOut - 1) / V::kOut;
    // slices: as many as x needs to fit; more while there are fewer CTAs than SMs and every warp
    // keeps a stage
    int slices = 1;
    if (stages > V::max_stages()) slices = 2;
    while (slices > 1 && (stages + slices - 1) / slices > V::max_stages_sliced()) slices *= 2;
    const int passes = (m.a.T + m.pass_rows - 1) / m.pass_rows;
    m.side = 1;
    if (MT == 1) {
        while (slices < kMaxSlices && (int64_t)strips * passes * slices * 2 <= sms * 2 && stages >= slices * 2 * V::kWarps) slices *= 2;
        // strips side by side: when there are plenty, each warp takes a longer part of the inputs, and
        // the sums over the parts cost less
        while (m.side < V::kWarps && strips * slices >= sms * 2 * m.side * 2 && stages / slices < 4 * V::kWarps / m.side) m.side *= 2;
    }
    m.slices = slices;
    m.tiles = (strips + m.side - 1) / m.side;
    m.slice_halves = 2 * ((stages + slices - 1) / slices);
    const int smem = V::kFixed + m.slice_halves * V::kHalf + (slices > 1 ? V::part_bytes(m.side) : 0);
    const int per_sm = std::min(MT == 2 ? 1 : 3, std::max(1, (kMaxSmem + 1024) / (smem + 1024)));
    const int groups = std::max(1, std::min(m.tiles, sms * per_sm / slices / std::min(passes, 4)));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(slices);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(groups * slices), unsigned(passes));
    cfg.blockDim = dim3(V::kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = slices > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q4_mma_kernel<NT, MT, kFine, kParts>, m);
}

// Whether warps take two strips: outputs for so many that every SM gets four pairs, or two where x has
// more than 8 rows (us with one strip and with two: 1 x 4096 x 10240 11.6, 13.5; 1 x 2048 x 20480 11.6,
// 10.2; 8 x 2048 x 20480 13.7, 10.5; 16 x 2048 x 10240 13.5, 10.6).
bool many(int64_t outputs, int sms, int nt) { return outputs >= (int64_t)sms * (nt == 2 ? 2 : 4) * 2 * kStrip; }

template <bool kFine, int kParts>
struct Rows {  // the variants by rows of x
    static bool fits(int nt, int stages) {
        const int s = (stages + kMaxSlices - 1) / kMaxSlices;
        return s <= (nt == 1 ? Var<1, 1, kFine, kParts>::max_stages_sliced() : Var<2, 1, kFine, kParts>::max_stages_sliced());
    }
    static int two_fit(int nt) {
        if (kParts == 3) return 0;  // one strip a warp: two would not have the registers
        return nt == 1 ? Var<1, 2, kFine, kParts>::max_stages() : Var<2, 2, kFine, kParts>::max_stages();
    }
    template <int NT>
    static cudaError_t launch_nt(const MmaArgs &m, int stages, int sms, cudaStream_t st) {
        // two strips a warp where there are plenty and x fits one CTA
        const int passes = (m.a.T + m.pass_rows - 1) / m.pass_rows;
        if constexpr (kParts != 3) {
            if (many((int64_t)m.a.N * passes, sms, NT) && stages <= Var<NT, 2, kFine, kParts>::max_stages())
                return launch_mma<NT, 2, kFine, kParts>(m, stages, sms, st);
        }
        return launch_mma<NT, 1, kFine, kParts>(m, stages, sms, st);
    }
    static cudaError_t launch(const MmaArgs &m, int stages, int sms, cudaStream_t st) {
        return m.pass_rows <= 8 ? launch_nt<1>(m, stages, sms, st) : launch_nt<2>(m, stages, sms, st);
    }
};

// Whether step (j - j0) stands for each codebook value well enough: within 2^-17 of the value for results
// that are rounded to bf16 (what the two parts of a general value keep), within 2^-20 for fp32 ones (values
// that were themselves computed in fp32, such as -1 + 2 j / 15 by steps, are off by up to 2^-20.6).  What
// rounding leaves in the place of a zero is taken as one.
bool affine_values(const float *book, float step, int twice_j0, bool out_f32) {
    double most = 0.0;
    for (int j = 0; j < 16; ++j) most = std::max(most, std::fabs(double(book[j])));
    for (int j = 0; j < 16; ++j) {
        const double v = book[j], off = std::fabs(v - double(step) * (j - 0.5 * twice_j0));
        if (off > std::fabs(v) * (out_f32 ? 0x1p-20 : 0x1p-17) + most * 0x1p-40) return false;
    }
    return true;
}

// The rows in passes of 16 (8 when x would not fit even split over a cluster), all in one launch;
// false if not even 8 rows fit.
bool run_mma(const Q4Args &a, int sms, cudaStream_t st, cudaError_t *err) {
    float step = 1.f;
    int twice = 0;
    const bool affine = q4_codebook_affine(a.codebook, &step, &twice) && affine_values(a.codebook, step, twice, a.out_f32);
    const bool fine = a.q_block == 32;
    const int stages = (a.K + kIn - 1) / kIn;
    // counted in 32 bits in the kernel
    if ((int64_t)(a.N + (1 << 20)) * (a.K / a.q_block) > UINT32_MAX || (int64_t)a.N * stages > INT32_MAX) return false;
    const int values = affine ? 0 : a.out_f32 ? 3 : 2;
    auto pick = [&](auto f) {
        if (values == 0) return fine ? f(Rows<true, 0>{}) : f(Rows<false, 0>{});
        if (values == 2) return fine ? f(Rows<true, 2>{}) : f(Rows<false, 2>{});
        return fine ? f(Rows<true, 3>{}) : f(Rows<false, 3>{});
    };
    auto two_fit = [&](int nt) {  // the most stages of two strips a warp
        return pick([&](auto v) { return decltype(v)::two_fit(nt); });
    };
    // where only 8 rows of x leave room for two strips a warp, passes of 8 (us in one pass and in two: 16 x
    // 4096 x 10240 24.9, 18.7; 16 x 2048 x 131072 with a general codebook in two parts 128, 102)
    const bool eights = a.T > 8 && two_fit(2) < stages && two_fit(1) >= stages && many((int64_t)a.N * ((a.T + 7) / 8), sms, 1);
    // tcgen05 for more rows than one pass where the weights are large enough that its longer start does
    // not count (us, tcgen05 and mma.sync): 64 x 2048 x 2048 14.6, 11.6; 40 x 512 x 20000 18.0, 15.1; 32 x 4096 x
    // 5120 16.0, 25.0; 64 x 4096 x 10240 51, 69.  For one pass of more than 8 rows only where neither side
    // of it has room for two strips: 16 x 2048 x 5120 10.2, 10.1; 16 x 4096 x 5120 12.1, 18.5; 16 x 8192 x 10240
    // 37, 52.
    const int64_t weights = (int64_t)a.N * a.K;
    const bool large = (a.K >= 2048 && weights >= (1 << 23)) || weights >= (1 << 26);
    if (affine && !fine && large && (a.T > kMmaRows || (a.T > 8 && two_fit(2) < stages && !eights)) &&
        run_tc(a, step, twice, sms, st, err))
        return true;
    auto fits = [&](int nt) {
        return pick([&](auto v) { return decltype(v)::fits(nt, stages); });
    };
    int nt_max = 2;
    while (nt_max > 0 && !fits(nt_max)) nt_max /= 2;
    if (nt_max == 0) return false;
    MmaArgs m{};
    m.a = a;
    m.step = affine ? step : 1.f;
    while (!fine && (64 << m.shift) < a.q_block) ++m.shift;
    m.centre = 16.f + 0.5f * float(twice);
    if (eights) nt_max = std::min(nt_max, 1);
    m.pass_rows = a.T <= 8 ? 8 : nt_max * 8;
    *err = pick([&](auto v) { return decltype(v)::launch(m, stages, sms, st); });
    return true;
}

}  // namespace
}  // namespace q4

cudaError_t launch_q4_linear(const moe_q4_linear_shape &s, const void *x, int64_t x_stride, const moe_q4_weight &w,
                             const void *res, int64_t res_stride, void *out, int64_t out_stride, int sms, cudaStream_t st) {
    q4::Q4Args a{};
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
    // q_block 32, or 64 times a power of two (a shift finds an input's block)
    const int q = s.q_block;
    cudaError_t err;
    if ((q == 32 || (q % 64 == 0 && (q & (q - 1)) == 0)) && q4::run_mma(a, sms, st, &err)) return err;
    return q4::launch_any(a, s.out_dtype, st);
}

}  // namespace moe
