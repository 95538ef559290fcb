// attn_decode.cuh -- attention of a few new tokens a sequence (decode, draft tokens) over the
// paged cache, bf16: the cache is read once, at the memory's rate.
//
// The query rows that share a key head (group x chunk, at most 16) fill one M = 16 tile of
// mma.sync, so a step of 16 keys is S = Q K^T, a running softmax, O += P V in one warp's
// registers; tcgen05's M = 128 would be 8 to 16 times padding here, and the matrix work is a
// sixth of what mma.sync does in the time that the memory takes (full decode batch: tensor pipe 18 %).  Each warp streams its own keys: cp.async copies of
// 16-byte pieces into a ring of its own (no barrier between warps), rows swizzled so that
// ldmatrix reads without bank conflicts.
//
// All (sequence, key head) pairs are laid end to end as steps of 16 keys.  Where the pairs are few,
// each is cut into parts of about the same number of steps, one part a CTA.  Where they are many,
// every CTA takes an equal share of the line, whatever the lengths, and may end one pair and
// begin the next: the shares are even, but a CTA pays the start and end of each piece (about
// kPiece steps' time).  A pair that a CTA holds whole is written out at once; the others leave (max, sum, unnormalised O) in the workspace, and the CTAs that
// arrive last join them in the order of the keys, so the bits do not depend on timing.
//
// Where the host sees that the pairs are few and no sequence can be long, a cluster of (sixteen,) eight, four
// or two CTAs (or one CTA) takes each pair: nothing is scheduled on the device, and the parts meet
// in shared memory (8 sequences of 150 to 1100 keys, 4 key heads: 7.5 us, 9.3 through the
// workspace; one sequence of 2000 keys 7.1 us, 9.3).
//
// With a window a pair's steps are those that hold a key that its first token sees: the first keys'
// steps, then, `skip` steps further on, the window's.  A window of 1024 over 64 sequences, 4 key heads of 128: 27.1 us, 0.74 of
// the measured copy rate; the start, a few dependent reads, is a quarter of it.
//
// Over an 8-bit cache (kQ8) a step is half as many bytes.  The codes become fp16 (exact: one
// instruction for two) as they leave shared memory and the products are fp16 ones: a row of q goes in
// units of a power of two that brings its largest element to 2^14 (fp16 then holds elements down to
// 2^-28 of that exactly; scores get the unit back), probabilities times 2^14.  A block's scale of k is
// a factor of its scores.  O is kept in units of a block's scale of v, and changes its unit when a block
// with a larger scale, or a much smaller one, comes; probabilities carry the rest.
// Up to 8 query rows a key head (kHalf) the products are turned round: keys, then values' columns, are the
// 16 rows of a tile and the queries its 8 columns, which halves the products, the softmax and O's registers
// (64 sequences, 537 k keys in all, groups of 8: 120 us as 16 x 8 tiles, half of them empty; 103 as here, two steps
// together, 0.81 of the measured copy rate).  The copies without the arithmetic take 92 us.  One sequence of 131071 keys takes 33.4 us, 20 of them the
// bytes and 12 the start and the join, as over a 16-bit cache.
#pragma once

#include "q8.cuh"

#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

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

template <int D, Mode kMode>
struct Cfg {
    static constexpr int kElem = kMode == kQ8 ? 1 : 2;  // bytes
    static constexpr int kStages = kMode == kQ8 ? (D == 128 ? 6 : 8) : D == 128 ? 3 : 6;
    static constexpr int kStageBytes = 2 * kStep * D * kElem;  // K rows, V rows
    static constexpr int kRing = kStages * kStageBytes;
    static constexpr int kSmem = kWarps * kRing;  // also the join's buffers
    static_assert((kWarps + 1) * kRows * (D + 2) * 4 <= kSmem, "");
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816h(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// An 8 x 8 matrix of 16-bit elements, two of a row a lane, with rows and columns exchanged.
__device__ __forceinline__ uint32_t turned(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// 2^e, -126 <= e <= 127; 0 for -127: what a sum in units of less than that of the new one becomes
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
// 2^x by the hardware unit (relative error about 2^-22; 0 for -inf).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The keys that a pair's rows do not all miss: places [0, cut) and from `low` on; and the steps between
// theirs, which are left out: step i of the pair is step i of the sequence below `sink_steps`, i + skip
// from there on.
template <Mode kMode>
struct Hole {
    uint32_t sink_steps = 0, skip = 0;
    int low = 0;
    __device__ __forceinline__ Hole(const Args &a, const Seq &s) {
        if (kMode == kAll) return;
        low = int(max((int64_t)s.kv_len - s.q_len + 1 - a.window, (int64_t)0));
        sink_steps = (uint32_t(min(a.sinks, low)) + kStep - 1) / kStep;
        const uint32_t from = uint32_t(low) / kStep;
        skip = from > sink_steps ? from - sink_steps : 0;
    }
    __device__ __forceinline__ uint32_t step(uint32_t i) const { return kMode == kAll || i < sink_steps ? i : i + skip; }
};

template <Mode kMode>
__device__ __forceinline__ int steps_of(const Args &a, const Seq &s) {
    if (s.q_len == 0) return 0;
    const int all = max(1, int((uint32_t(s.kv_len) + kStep - 1) / kStep));  // kv_len up to 2^31 - 1
    return kMode == kAll ? all : all - int(Hole<kMode>(a, s).skip);
}

// Exclusive prefix of one value a thread over the block, and the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t n, uint32_t *total, uint32_t *scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? scratch[w] : 0;
        sum += scratch[w];
    }
    *total = sum;
    return before + incl - n;
}

// The line of all steps cut into `ctas` shares that differ by at most one step: the first
// `more` shares hold each + 1.
struct Shares {
    uint32_t each, more;
    __device__ __forceinline__ uint32_t begin(uint32_t cta) const { return cta * each + min(cta, more); }
    __device__ __forceinline__ uint32_t owner(uint32_t step) const {
        const uint32_t edge = more * (each + 1);
        return step < edge ? step / (each + 1) : more + (step - edge) / each;
    }
};

constexpr uint32_t kPiece = 10;

// Partial results in the workspace.  A CTA leaves at most two: of the pair that its share
// begins inside (slot 2 cta) and of the pair that begins in its share and goes on (slot
// 2 cta + 1).  The CTAs of a pair are joined in groups of kGroup in the order of their keys,
// then the groups, so that no CTA reads hundreds of partial results alone.  Each arrival is a
// field of one word per CTA, the CTA that the pair or group starts in: bits 0-9 count the
// groups of the pair that starts there, 10-19 the members of that pair's first group, 20-29
// those of a later group that starts there.
constexpr uint32_t kGroup = 16;
constexpr int kJoinBatch = 8;  // parts whose outputs are requested together

struct Parts {
    uint32_t *words;
    float *o;     // [slot][row][D]
    float2 *ml;   // [slot][row]
};

// Adds one arrival; true for the last of n, which also puts the field back to 0.
__device__ __forceinline__ bool arrive_last(uint32_t *word, int shift, uint32_t n, int *flag) {
    __syncthreads();  // the block's partial results are written
    if (threadIdx.x == 0) {
        uint32_t old;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(word), "r"(1u << shift) : "memory");
        const bool last = ((old >> shift) & 1023u) == n - 1;
        if (last) atomicSub(word, n << shift);
        *flag = last;
    }
    __syncthreads();
    return *flag != 0;
}

// Joins parts [0, n) (their slots from slot_of) of `rows` <= kMost rows; emit(row, d, float4, m, l).
// sm: float2 [kJoinBatch][kRows].
template <int D, int kMost, typename SlotOf, typename Emit>
__device__ __forceinline__ void join_rows(const Parts &p, uint32_t n, int rows, float *sm, SlotOf slot_of, Emit emit) {
    constexpr int PER = kMost * D / 4 / kThreads;  // float4 positions of a thread
    const int tid = threadIdx.x;
    const int mr = tid & (kRows - 1), mi = tid / kRows;  // (row, part) whose (max, sum) the thread reads
    float4 acc[PER];
    float m[PER], l[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        m[e] = kNegInf;
        l[e] = 0.f;
    }
    float2 *sml = reinterpret_cast<float2 *>(sm);
    for (uint32_t k0 = 0; k0 < n; k0 += kJoinBatch) {
        float2 ml = make_float2(kNegInf, 0.f);
        if (k0 + mi < n && mr < rows) {
            const float *q = &p.ml[slot_of(k0 + mi) * kRows + mr].x;
            asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(ml.x), "=f"(ml.y) : "l"(q));
        }
        float4 v[PER][kJoinBatch];
#pragma unroll
        for (int k = 0; k < kJoinBatch; ++k) {
            const uint32_t kk = min(k0 + k, n - 1);  // past the last: read again, with factor 0
            const float *src = p.o + slot_of(kk) * kRows * D;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int i = e * kThreads + tid;
                v[e][k] = i < rows * (D / 4) ? ldp16f(src + i * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        __syncthreads();
        sml[mi * kRows + mr] = ml;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int r = (e * kThreads + tid) / (D / 4);
            float mn = m[e];
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) mn = fmaxf(mn, sml[k * kRows + r].x);
            const float f0 = m[e] == kNegInf ? 0.f : ex2(m[e] - mn);
            acc[e].x *= f0;
            acc[e].y *= f0;
            acc[e].z *= f0;
            acc[e].w *= f0;
            l[e] *= f0;
            m[e] = mn;
#pragma unroll
            for (int k = 0; k < kJoinBatch; ++k) {
                const float2 x = sml[k * kRows + r];
                const float f = x.x == kNegInf ? 0.f : ex2(x.x - mn);
                l[e] = fmaf(f, x.y, l[e]);
                acc[e].x = fmaf(f, v[e][k].x, acc[e].x);
                acc[e].y = fmaf(f, v[e][k].y, acc[e].y);
                acc[e].z = fmaf(f, v[e][k].z, acc[e].z);
                acc[e].w = fmaf(f, v[e][k].w, acc[e].w);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int i = e * kThreads + tid;
        if (i < rows * (D / 4)) emit(i / (D / 4), i % (D / 4) * 4, acc[e], m[e], l[e]);
    }
}

template <int D, typename SlotOf, typename Emit>
__device__ __forceinline__ void join_parts(const Parts &p, uint32_t n, int rows, float *sm, SlotOf slot_of, Emit emit) {
    if (rows <= 8)
        join_rows<D, 8>(p, n, rows, sm, slot_of, emit);
    else
        join_rows<D, 16>(p, n, rows, sm, slot_of, emit);
}

// kCluster: CTAs of a pair, 0 where the work is scheduled on the device.
template <int D, int kCluster, Mode kMode, bool kHalf>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(Args a, Parts parts) {
    namespace cg = cooperative_groups;
    using C = Cfg<D, kMode>;
    constexpr bool kClustered = kCluster > 0;
    constexpr int kC = kClustered ? kCluster : 1;
    // the join's buffers: [warp][row][D], [warp][row] (max, sum); clustered, after them [row][D], [row]
    constexpr int kJoinFloats = kWarps * kRows * (D + 2);
    static_assert((kJoinFloats + kRows * (D + 2)) * 4 <= C::kSmem, "");
    constexpr int NT = D / 8;        // 8-column tiles of O
    constexpr int KS = D / 16;       // 16-element steps of the head dimension
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint32_t scratch[kWarps];
    __shared__ uint32_t first[2];  // this CTA's first sequence and that sequence's first step
    __shared__ Seq first_seq;
    __shared__ int last_flag;
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const uint32_t G = a.group, Hkv = a.n_kv_heads;

    int b = 0;
    uint32_t base = 0, steps = 0, part = 0, at = 0, u = 0, u_end = 0;
    bool aligned = false;
    Shares sh{};
    Seq s{};
    const uint32_t cta = blockIdx.x;
    if constexpr (kClustered) {
        b = int(cta / kC / Hkv);
        s = load_seq(a, b);
        if (s.q_len == 0) return;  // the whole cluster
        steps = steps_of<kMode>(a, s);
    } else {
        // the line of all steps, and how it is cut.  Up to 32 sequences every warp scans by itself, without
        // barriers.
        const bool few = a.n_seqs <= 32;
        uint32_t n0 = 0, before0 = 0, total = 0, pairs = 0;
        auto warp_scan = [&](uint32_t n, uint32_t *sum) {
            uint32_t incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            *sum = __shfl_sync(0xffffffffu, incl, 31);
            return incl - n;
        };
        if (few) {
            if (lane < a.n_seqs) {
                s = load_seq(a, lane);
                n0 = steps_of<kMode>(a, s);
            }
            pairs = __popc(__ballot_sync(0xffffffffu, n0 > 0)) * Hkv;
            before0 = warp_scan(n0 * Hkv, &total);
        }
        for (int b0 = 0; !few && b0 < a.n_seqs; b0 += kThreads) {
            uint32_t n = 0, sum;
            if (b0 + tid < a.n_seqs) {
                const Seq x = load_seq(a, b0 + tid);
                n = steps_of<kMode>(a, x);
                if (b0 == 0) s = x;
            }
            pairs += uint32_t(__syncthreads_count(n > 0)) * Hkv;
            const uint32_t before = block_scan(n * Hkv, &sum, scratch);
            if (b0 == 0) {
                n0 = n;
                before0 = before;
            }
            total += sum;
        }
        const uint32_t grid = gridDim.x;
        // parts of at most `part` steps make at most total / part + pairs <= grid CTAs; each warp keeps
        // two steps
        part = pairs < grid ? max(2u * kWarps, (total + grid - pairs - 1) / (grid - pairs)) : 0u;
        aligned = part > 0 && part <= max(2u * kWarps, total / grid + kPiece);
        // no more CTAs than leave every warp two steps: fewer parts to join
        const uint32_t ctas = max(1u, min(grid, total / (2 * kWarps)));
        sh = Shares{total / ctas, total % ctas};
        if (!aligned) {
            if (cta >= ctas) return;
            u = sh.begin(cta);
            u_end = sh.begin(cta + 1);
            if (u >= u_end) return;
        }
        // places of a sequence: its parts (aligned), or its steps, of all heads
        auto places_of = [&](uint32_t n) { return (aligned ? (n + part - 1) / part : n) * Hkv; };
        at = aligned ? cta : u;  // its place on the line of parts or steps
        if (few) {
            uint32_t sum;
            const uint32_t n = places_of(n0), before = aligned ? warp_scan(n, &sum) : before0;
            const uint32_t here = __ballot_sync(0xffffffffu, at >= before && at - before < n);
            if (here == 0) return;  // past the last part: every warp of the block
            b = __ffs(here) - 1;
            base = __shfl_sync(0xffffffffu, before, b);
            s.q0 = __shfl_sync(0xffffffffu, s.q0, b);
            s.q_len = __shfl_sync(0xffffffffu, s.q_len, b);
            s.kv_len = __shfl_sync(0xffffffffu, s.kv_len, b);
        } else {
            if (tid == 0) first[0] = ~0u;
            auto found = [&](uint32_t i, uint32_t before, uint32_t n, const Seq &x) {
                if (at >= before && at - before < n) {
                    first[0] = i;
                    first[1] = before;
                    first_seq = x;
                }
            };
            if (a.n_seqs <= kThreads) {
                uint32_t sum;
                const uint32_t n = places_of(n0), before = aligned ? block_scan(n, &sum, scratch) : before0;
                __syncthreads();
                found(tid, before, n, s);
            } else {
                for (int b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
                    uint32_t n = 0, sum;
                    Seq x{};
                    if (b0 + tid < a.n_seqs) {
                        x = load_seq(a, b0 + tid);
                        n = places_of(steps_of<kMode>(a, x));
                    }
                    const uint32_t before = base + block_scan(n, &sum, scratch);
                    found(b0 + tid, before, n, x);
                    base += sum;
                    if (at < base) break;
                }
            }
            __syncthreads();
            if (first[0] == ~0u) return;  // past the last part
            b = int(first[0]);
            base = first[1];
            s = first_seq;
        }
        steps = steps_of<kMode>(a, s);
    }

    const uint32_t ring = smem_addr(smem) + warp * C::kRing;
    const float sl2 = a.scale * kLog2e;

    for (bool more = true; more;) {
        uint32_t h, c0 = 0, n_parts = 1, step0, step1, item = 0;
        if (kClustered) {
            h = cta / kC % Hkv;
            const uint32_t rank = cta % kC;
            const Shares even{steps / kC, steps % kC};
            step0 = even.begin(rank);
            step1 = even.begin(rank + 1);
            more = false;
        } else if (aligned) {
            const uint32_t per = (steps + part - 1) / part;
            h = (at - base) / per;
            const uint32_t i = at - base - h * per;
            // even parts of the pair
            const Shares even{steps / per, steps % per};
            step0 = even.begin(i);
            step1 = even.begin(i + 1);
            c0 = cta - i;
            n_parts = per;
            more = false;
        } else {
            while (u - base >= steps * Hkv) {  // the next sequence with a chunk
                base += steps * Hkv;
                if (++b >= a.n_seqs) return;  // not seen: the line ends with the last sequence
                s = load_seq(a, b);
                steps = steps_of<kMode>(a, s);
            }
            h = (u - base) / steps;
            item = base + h * steps;  // its first step
            step0 = u - item;
            step1 = min(steps, u_end - item);
            c0 = step0 == 0 ? cta : sh.owner(item);
            n_parts = (step1 == steps ? cta : sh.owner(item + steps - 1)) - c0 + 1;
            u = item + step1;
            more = u < u_end;
        }
        const int rows = min(s.q_len * int(G), kHalf ? kRows / 2 : kRows), past = s.kv_len - s.q_len;

        // the warp's keys: steps step0 + warp, + kWarps, ...  The cache offset of lane r's key row (r <
        // 16), or of the first row where a step lies within a page, is found a step before the copy.
        const int mine = step1 - step0 > uint32_t(warp) ? int(step1 - step0 - warp + kWarps - 1) / kWarps : 0;
        const bool in_page = kMode == kQ8 || a.page_size % kStep == 0;
        const Hole<kMode> hole(a, s);
        auto key_of = [&](int i) { return int(hole.step(step0 + warp + i * kWarps)) * kStep; };
        // whether a row sees key p (those past the last are not asked about), and every key of a step
        auto wanted = [&](int p) { return kMode == kAll || p < a.sinks || p >= hole.low; };
        auto all_wanted = [&](int p) { return kMode == kAll || p >= hole.low || a.sinks - p >= kStep; };
        auto find_row = [&](int i) -> int64_t {
            const int p = i < mine ? key_of(i) + (in_page ? 0 : lane & 15) : 0;
            if (i >= mine || p >= s.kv_len || (!in_page && !wanted(p))) return -1;
            const int pi = a.page_shift >= 0 ? p >> a.page_shift : p / a.page_size;
            return load_page(a, b, pi) * a.page_stride + (int64_t)(p - pi * a.page_size) * a.token_stride;
        };
        constexpr int E = C::kElem, CHB = D * E / 16, RPB = 32 / CHB;  // 16-byte pieces of a row, rows an instruction
        const uint8_t *kc = static_cast<const uint8_t *>(a.k) + (int64_t)h * a.head_stride * E + lane % CHB * 16;
        const uint8_t *vc = static_cast<const uint8_t *>(a.v) + (int64_t)h * a.head_stride * E + lane % CHB * 16;
        const int64_t lane_row = (int64_t)(lane / CHB) * a.token_stride * E, next_row = (int64_t)RPB * a.token_stride * E;
        // where piece c of row r lies: ldmatrix reads a piece of eight rows at a time, the codes of k are read
        // as four pieces of two rows
        auto at_k = [&](int r, int c) {
            return kMode != kQ8 ? c ^ (r & 7) : D == 128 ? c ^ ((r & 1) << 2) : c;
        };
        auto at_v = [&](int r, int c) { return kMode != kQ8 || D == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3); };
        auto copy = [&](int i, int64_t row_off) {
            if (i < mine) {
                const uint32_t dst = ring + (i % C::kStages) * C::kStageBytes + lane / CHB * (D * E);
                const int p = key_of(i);
                if (in_page && s.kv_len - p >= kStep && all_wanted(p)) {
                    const uint8_t *ks = kc + row_off * E + lane_row, *vs = vc + row_off * E + lane_row;
#pragma unroll
                    for (int it = 0; it < kStep / RPB; ++it, ks += next_row, vs += next_row) {
                        const int r = it * RPB + lane / CHB;
                        const uint32_t to = dst + it * RPB * (D * E);
                        cp16(to + at_k(r, lane % CHB) * 16, ks, 16);
                        cp16(to + kStep * D * E + at_v(r, lane % CHB) * 16, vs, 16);
                    }
                } else {
#pragma unroll
                    for (int it = 0; it < kStep / RPB; ++it) {
                        const int r = it * RPB + lane / CHB;
                        int64_t off = __shfl_sync(0xffffffffu, row_off, in_page ? 0 : r);
                        if (in_page) off += r * a.token_stride;
                        // rows past the last key, and those that no row sees: zeros, nothing is read
                        const int n = p + r < s.kv_len && wanted(p + r) ? 16 : 0;
                        const uint32_t to = dst + it * RPB * (D * E);
                        cp16(to + at_k(r, lane % CHB) * 16, kc + (n ? off * E : 0), n);
                        cp16(to + kStep * D * E + at_v(r, lane % CHB) * 16, vc + (n ? off * E : 0), n);
                    }
                }
            }
            cp_commit();
        };
        int64_t next = kMode == kQ8 ? 0 : find_row(0);

        // Q as A fragments: rows g and g + 8, columns 16 ks + 2 t4 (+1) and + 8; a row past the
        // last reads the first one's and is zeroed, so that all loads go out together.  Over 8-bit keys, whose
        // lane t4 holds 16 consecutive codes, the columns of step ks are four of those.
        uint32_t q[KS][4];
        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (int64_t)s.q0 * a.q_stride + (int64_t)h * G * D +
                             (kMode == kQ8 ? t4 * 16 : t4 * 2);
        const bool on0 = g < rows, on1 = g + 8 < rows;
        const uint32_t r0 = on0 ? g : 0, r1 = on1 ? g + 8 : 0, j0 = r0 / G, j1 = r1 / G;
        const uint16_t *q0 = qp + j0 * a.q_stride + (r0 - j0 * G) * D, *q1 = qp + j1 * a.q_stride + (r1 - j1 * G) * D;
        auto load_q = [&](const uint16_t *from, int e) {
            if constexpr (kMode == kQ8) {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    const uint4 v = ldp16(from + ks / 4 * 64 + ks % 4 * 4);
                    q[ks][e] = v.x;
                    q[ks][e + 2] = v.y;
                    q[ks + 1][e] = v.z;
                    q[ks + 1][e + 2] = v.w;
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    q[ks][e] = ldp(reinterpret_cast<const uint32_t *>(from + ks * 16));
                    q[ks][e + 2] = ldp(reinterpret_cast<const uint32_t *>(from + ks * 16 + 8));
                }
            }
        };
        load_q(q0, 0);
        if (!kHalf && rows > 8) {
            load_q(q1, 1);
        } else {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) q[ks][1] = q[ks][3] = 0u;
        }
        // 8-bit keys: the pages and scales of 32 steps at a time, a lane each.  `_cur` is what copies read now, the
        // batch after it is on its way (its pages half a batch before its scales, which need them)
        int64_t off_cur = 0, off_next = 0;
        uint32_t sc_cur = 0, sc_prev = 0, sc_next = 0;  // a step's bytes: k, v << 8
        int page_next = 0;
        auto batch_page = [&](int i) {
            const int p = i < mine ? key_of(i) : 0;
            if (i >= mine || p >= s.kv_len) return -1;
            return load_page(a, b, a.page_shift >= 0 ? p >> a.page_shift : p / a.page_size);
        };
        auto batch_rest = [&](int i, int page, int64_t &off, uint32_t &sc) {
            off = 0;
            sc = 127 | 127 << 8;
            if (page < 0) return;
            const int p = key_of(i), slot = a.page_shift >= 0 ? p & (a.page_size - 1) : p % a.page_size;
            off = page * a.page_stride + (int64_t)slot * a.token_stride;
            const int64_t of = page * a.scale_page + h * a.scale_head + (a.block_shift >= 0 ? slot >> a.block_shift : slot / a.block);
            sc = q8::ldp_byte(a.k_scale + of) | q8::ldp_byte(a.v_scale + of) << 8;
        };
        auto copy_q8 = [&](int i) {
            if (i % 32 == 0 && i > 0) {
                sc_prev = sc_cur;
                sc_cur = sc_next;
                off_cur = off_next;
                page_next = batch_page(i + 32 + lane);
            }
            if (i % 32 == 16) batch_rest(i + 16 + lane, page_next, off_next, sc_next);
            copy(i, __shfl_sync(0xffffffffu, off_cur, i & 31));
        };
        if constexpr (kMode == kQ8) {
            batch_rest(lane, batch_page(lane), off_cur, sc_cur);
            page_next = batch_page(32 + lane);
        }
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) {
            if constexpr (kMode == kQ8) {
                copy_q8(i);
            } else {
                const int64_t cur = next;
                next = find_row(i + 1);
                copy(i, cur);
            }
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[ks][e] = ((e & 1) ? on1 : on0) ? q[ks][e] : 0u;
        float sl2_0 = sl2, sl2_1 = sl2;  // of the rows g and g + 8
        if constexpr (kMode == kQ8) {
            // the unit of a row: 2^-x with x from its largest exponent (an infinity counts as the largest number)
            uint32_t top0 = 0, top1 = 0;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                top0 = __vmaxu2(top0, __vmaxu2(q[ks][0] & 0x7fff7fffu, q[ks][2] & 0x7fff7fffu));
                top1 = __vmaxu2(top1, __vmaxu2(q[ks][1] & 0x7fff7fffu, q[ks][3] & 0x7fff7fffu));
            }
#pragma unroll
            for (int w = 1; w <= 2; w <<= 1) {
                top0 = __vmaxu2(top0, __shfl_xor_sync(0xffffffffu, top0, w));
                top1 = __vmaxu2(top1, __shfl_xor_sync(0xffffffffu, top1, w));
            }
            auto unit = [](uint32_t top) { return min(127 + 14 - min(int(max(top & 0xffffu, top >> 16) >> 7), 254), 126); };
            const int x0 = unit(top0), x1 = unit(top1);
            sl2_0 *= pow2(-x0);
            sl2_1 *= pow2(-x1);
            if constexpr (kHalf) {  // of the rows 2 t4 and 2 t4 + 1
                const float own = sl2_0;
                sl2_0 = __shfl_sync(0xffffffffu, own, t4 * 8);
                sl2_1 = __shfl_sync(0xffffffffu, own, t4 * 8 + 4);
            }
            auto to_f16 = [](uint32_t v, float f) {
                return pack_f16(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
            };
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e) q[ks][e] = to_f16(q[ks][e], (e & 1) ? pow2(x1) : pow2(x0));
        }
        // keys that the lane's two rows of scores see: g and g + 8, or 2 t4 and 2 t4 + 1
        const bool see0 = kHalf ? t4 * 2 < rows : on0, see1 = kHalf ? t4 * 2 + 1 < rows : on1;
        const int seen0 = see0 ? past + int(kHalf ? t4 * 2 / G : j0) + 1 : 0;
        const int seen1 = see1 ? past + int(kHalf ? (t4 * 2 + 1) / G : j1) + 1 : 0;
        const int seen_all = past + 1;  // keys that every row sees
        constexpr int OT = kHalf ? D / 16 : NT;
        float o[OT][4];
#pragma unroll
        for (int j = 0; j < OT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;
        int unit_v = -1, most_v = 0;  // 8-bit values: O is in units of 2^(unit_v - 127 - 14); the largest byte so far

        // the products turned round, N steps at a time (of an 8-bit cache, whose steps have one scale each)
        auto half_steps = [&](auto count, int i, int copied) {
            constexpr int N = decltype(count)::value;
            float sc[N][4], odd[N][4];
            uint32_t bytes[N], kb[N];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                bytes[n] = __shfl_sync(0xffffffffu, ((i + n) ^ copied) < 32 ? sc_cur : sc_prev, (i + n) & 31);
                kb[n] = ring + ((i + n) % C::kStages) * C::kStageBytes;
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] = odd[n][e] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < KS / 4; ++c)
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint4 w0 = lds16(kb[n] + g * D + at_k(g, c * 4 + t4) * 16), w1 = lds16(kb[n] + (g + 8) * D + at_k(g + 8, c * 4 + t4) * 16);
                    const uint32_t y0[4] = {w0.x, w0.y, w0.z, w0.w}, y1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t k4[4];  // keys g and g + 8, two columns each, then the next two
                        q8::to_f16x4(y0[e], k4[0], k4[2]);
                        q8::to_f16x4(y1[e], k4[1], k4[3]);
                        mma16816h(e & 1 ? odd[n] : sc[n], k4, q[c * 4 + e][0], q[c * 4 + e][2]);
                    }
                }
            float x0 = m0, x1 = m1;  // of the rows 2 t4 and 2 t4 + 1
            int top = -1;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const float ks = q8::scale_of(bytes[n] & 255), f0 = sl2_0 * ks, f1 = sl2_1 * ks;
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] = (sc[n][e] + odd[n][e]) * (e & 1 ? f1 : f0);
                const int key0 = key_of(i + n);
                if (key0 > seen_all - kStep || (key0 < s.kv_len - a.window && key0 > a.sinks - kStep)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + (e >> 1) * 8 + g, seen = e & 1 ? seen1 : seen0;
                        if (key >= seen || (key >= a.sinks && key < seen - a.window)) sc[n][e] = kNegInf;
                    }
                }
                x0 = fmaxf(x0, fmaxf(sc[n][0], sc[n][2]));
                x1 = fmaxf(x1, fmaxf(sc[n][1], sc[n][3]));
                const int ev = bytes[n] >> 8;
                top = max(top, ev < 255 ? ev : -1);
            }
#pragma unroll
            for (int w = 4; w <= 16; w <<= 1) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
            }
            const float z0 = x0 == kNegInf ? 0.f : x0, z1 = x1 == kNegInf ? 0.f : x1;
            const int old_unit = unit_v < 0 ? top : unit_v;
            most_v = max(most_v, top);
            if (top > unit_v || (top >= 0 && top < unit_v - 6 && top >= most_v - 60)) unit_v = top;
            if (__any_sync(0xffffffffu, x0 != m0 || x1 != m1) || unit_v != old_unit) {
                const float u = pow2(max(old_unit - unit_v, -127));
                float f0 = ex2(m0 - z0), f1 = ex2(m1 - z1);
                l0 *= f0;
                l1 *= f1;
                f0 *= u;
                f1 *= u;
#pragma unroll
                for (int j = 0; j < OT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][e] *= e & 1 ? f1 : f0;
                m0 = x0;
                m1 = x1;
            }
            uint32_t p[N][2];
#pragma unroll
            for (int n = 0; n < N; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] = ex2(sc[n][e] - (e & 1 ? z1 : z0));
                l0 += sc[n][0] + sc[n][2];  // this lane's keys; the others' are added at the end
                l1 += sc[n][1] + sc[n][3];
                // in fp16, as below; turned, the tiles' second operand
                const int ev = bytes[n] >> 8;
                const float f = ev == 255 ? q8::scale_of(255) : pow2(max(14 + ev - max(unit_v, 0), -126));
                p[n][0] = turned(pack_f16(sc[n][0] * f, sc[n][1] * f));
                p[n][1] = turned(pack_f16(sc[n][2] * f, sc[n][3] * f));
            }
            const int r = lane & 15;
#pragma unroll
            for (int c = 0; c < D / 16; c += 2)
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    uint32_t vf[4];
                    ldsm4t(kb[n] + kStep * D + r * D + at_v(r, c + (lane >> 4)) * 16, vf);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t v4[4];  // columns 2 g and 2 g + 1 of keys 2 t4 (+ 1), then of the keys 8 further on
                        q8::to_f16x4(__byte_perm(vf[2 * e], 0, 0x3120), v4[0], v4[1]);
                        q8::to_f16x4(__byte_perm(vf[2 * e + 1], 0, 0x3120), v4[2], v4[3]);
                        mma16816h(o[c + e], v4, p[n][0], p[n][1]);
                    }
                }
        };
        if constexpr (kHalf) {
            // two steps together, for more independent instructions and half the reductions (one at a time: a full
            // batch 108 us)
            int i = 0;
            for (; i + 2 <= mine; i += 2) {
                copy_q8(i + C::kStages - 1);
                cp_wait<C::kStages - 2>();
                __syncwarp();
                half_steps(std::integral_constant<int, 2>{}, i, i + C::kStages - 1);
                __syncwarp();  // the stages are read before a lane's next copy lands in them
                copy_q8(i + C::kStages);
            }
            if (i < mine) {
                cp_wait<C::kStages - 2>();
                __syncwarp();
                half_steps(std::integral_constant<int, 1>{}, i, i + C::kStages - 2);
            }
        }
        for (int i = 0; i < (kHalf ? 0 : mine); ++i) {
            uint32_t bytes = 0;  // the step's scales
            if constexpr (kMode == kQ8) {
                copy_q8(i + C::kStages - 1);
                bytes = __shfl_sync(0xffffffffu, (i ^ (i + C::kStages - 1)) < 32 ? sc_cur : sc_prev, i & 31);
            } else {
                const int64_t cur = next;
                next = find_row(i + C::kStages);
                copy(i + C::kStages - 1, cur);
            }
            cp_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t kb = ring + (i % C::kStages) * C::kStageBytes, vb = kb + kStep * D * E;
            float sc[2][4] = {};
            if constexpr (kMode == kQ8) {
                float odd[2][4] = {};
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int r = n * 8 + g;
#pragma unroll
                    for (int c = 0; c < KS / 4; ++c) {
                        const uint4 w = lds16(kb + r * D + at_k(r, c * 4 + t4) * 16);
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t lo, hi;
                            q8::to_f16x4(x[e], lo, hi);
                            mma16816h(e & 1 ? odd[n] : sc[n], q[c * 4 + e], lo, hi);
                        }
                    }
                }
                const float ks = q8::scale_of(bytes & 255), f0 = sl2_0 * ks, f1 = sl2_1 * ks;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    sc[n][0] = (sc[n][0] + odd[n][0]) * f0;
                    sc[n][1] = (sc[n][1] + odd[n][1]) * f0;
                    sc[n][2] = (sc[n][2] + odd[n][2]) * f1;
                    sc[n][3] = (sc[n][3] + odd[n][3]) * f1;
                }
            } else {
                const int r = (lane & 7) + (lane >> 4) * 8;  // matrices: keys 0-7 (two pieces), keys 8-15
                float odd[2][4] = {};  // a second chain of dependent products, half as long each
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t kf[4];
                    ldsm4(kb + r * (D * 2) + (((2 * ks + ((lane >> 3) & 1)) ^ (r & 7)) * 16), kf);
                    mma16816(ks & 1 ? odd[0] : sc[0], q[ks], kf[0], kf[1]);
                    mma16816(ks & 1 ? odd[1] : sc[1], q[ks], kf[2], kf[3]);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[n][e] += odd[n][e];
            }
            const int key0 = key_of(i);
            if constexpr (kMode != kQ8) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[n][e] *= sl2;
            }
            if (key0 > seen_all - kStep) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + n * 8 + t4 * 2 + (e & 1);
                        if (key >= (e < 2 ? seen0 : seen1)) sc[n][e] = kNegInf;
                    }
            }
            if (kMode != kAll && key0 < s.kv_len - a.window && key0 > a.sinks - kStep) {  // before a row's window
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + n * 8 + t4 * 2 + (e & 1);
                        if (key >= a.sinks && key < (e < 2 ? seen0 : seen1) - a.window) sc[n][e] = kNegInf;
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
            // O's unit: that of this block where its scale is larger than O's, or smaller by more than 2^6 (fp16
            // then still holds probabilities of 2^-22 as normal numbers), down to 2^-60 of the largest seen
            int old_unit = unit_v;
            if constexpr (kMode == kQ8) {
                const int ev = bytes >> 8;
                if (ev < 255) {
                    most_v = max(most_v, ev);
                    if (unit_v < 0) old_unit = ev;
                    if (ev > unit_v || (ev < unit_v - 6 && ev >= most_v - 60)) unit_v = ev;
                }
            }
            if (__any_sync(0xffffffffu, n_0 != m0 || n_1 != m1) || (kMode == kQ8 && unit_v != old_unit)) {
                float f0 = ex2(m0 - z0), f1 = ex2(m1 - z1);
                l0 *= f0;
                l1 *= f1;
                if constexpr (kMode == kQ8) {
                    const float u = pow2(max(old_unit - unit_v, -127));
                    f0 *= u;
                    f1 *= u;
                }
#pragma unroll
                for (int j = 0; j < OT; ++j) {
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
            if constexpr (kMode == kQ8) {
                // probabilities in fp16, in units that take in the difference of the block's scale to O's
                const int ev = bytes >> 8;
                const float f = ev == 255 ? q8::scale_of(255) : pow2(max(14 + ev - max(unit_v, 0), -126));
                const uint32_t p[4] = {pack_f16(sc[0][0] * f, sc[0][1] * f), pack_f16(sc[0][2] * f, sc[0][3] * f),
                                       pack_f16(sc[1][0] * f, sc[1][1] * f), pack_f16(sc[1][2] * f, sc[1][3] * f)};
                const int r = lane & 15;
#pragma unroll
                for (int c = 0; c < D / 16; c += 2) {
                    // a register of a matrix: two codes of one key, the same two of the next
                    uint32_t vf[4];
                    ldsm4t(vb + r * D + at_v(r, c + (lane >> 4)) * 16, vf);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t even0, odd0, even1, odd1;
                        q8::to_f16x4(__byte_perm(vf[2 * e], 0, 0x3120), even0, odd0);
                        q8::to_f16x4(__byte_perm(vf[2 * e + 1], 0, 0x3120), even1, odd1);
                        mma16816h(o[2 * (c + e)], p, even0, even1);
                        mma16816h(o[2 * (c + e) + 1], p, odd0, odd1);
                    }
                }
            } else {
                // probabilities in bf16 for the product: up to 2^-8 of each, of either sign, where the output is rounded to
                // as much anyway (error of a decode batch against 64 bits 0.0019 of the outputs' size, with fp32
                // probabilities 0.0017); the sum that divides is of the unrounded ones
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
            }
            __syncwarp();  // the stage is read before a lane's next copy lands in it
        }
        cp_wait<0>();
#pragma unroll
        for (int w = kHalf ? 4 : 1; w <= (kHalf ? 16 : 2); w <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, w);
            l1 += __shfl_xor_sync(0xffffffffu, l1, w);
        }

        if constexpr (kMode == kQ8) {
            const float u = q8::scale_of(max(unit_v, 0));
#pragma unroll
            for (int j = 0; j < OT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = o[j][e] * pow2(-14) * u;
        }

        // join the warps: [warp][row][D], then [warp][row] (max, sum)
        float *jo = reinterpret_cast<float *>(smem);
        float2 *jm = reinterpret_cast<float2 *>(jo + kWarps * kRows * D);
        __syncthreads();
        if constexpr (kHalf) {
#pragma unroll
            for (int c = 0; c < OT; ++c) {
                float *to = jo + (warp * kRows + t4 * 2) * D + c * 16 + g * 2;
                *reinterpret_cast<float2 *>(to) = make_float2(o[c][0], o[c][2]);
                *reinterpret_cast<float2 *>(to + D) = make_float2(o[c][1], o[c][3]);
            }
        } else if constexpr (kMode == kQ8) {  // tiles of even and of odd columns
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                float *to = jo + (warp * kRows + g) * D + j * 8 + t4 * 4;
                *reinterpret_cast<float4 *>(to) = make_float4(o[j][0], o[j + 1][0], o[j][1], o[j + 1][1]);
                if (rows > 8)
                    *reinterpret_cast<float4 *>(to + 8 * D) = make_float4(o[j][2], o[j + 1][2], o[j][3], o[j + 1][3]);
            }
        }
#pragma unroll
        for (int j = 0; j < (kMode == kQ8 ? 0 : NT); ++j) {
            *reinterpret_cast<float2 *>(jo + (warp * kRows + g) * D + j * 8 + t4 * 2) = make_float2(o[j][0], o[j][1]);
            if (rows > 8)
                *reinterpret_cast<float2 *>(jo + (warp * kRows + g + 8) * D + j * 8 + t4 * 2) = make_float2(o[j][2], o[j][3]);
        }
        if (kHalf ? g == 0 : t4 == 0) {
            jm[warp * kRows + (kHalf ? t4 * 2 : g)] = make_float2(m0, l0);
            jm[warp * kRows + (kHalf ? t4 * 2 + 1 : g + 8)] = make_float2(m1, l1);
        }
        __syncthreads();
        auto write_out = [&](int r, int d, float4 v, float m, float l) {
            const uint32_t j = uint32_t(r) / G, head = h * G + (r - j * G);
            const int64_t tok = s.q0 + j;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + tok * a.out_stride + (int64_t)head * D + d) =
                make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            if (a.lse && d == 0) a.lse[tok * a.n_heads + head] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
        };
        auto write_part = [&](size_t slot, int r, int d, float4 v, float m, float l) {
            *reinterpret_cast<float4 *>(parts.o + (slot * kRows + r) * D + d) = v;
            if (d == 0) parts.ml[slot * kRows + r] = make_float2(m, l);
        };
        const bool whole = n_parts == 1;
        float *cj = jo + kJoinFloats;  // clustered: this CTA's part for the others
        float2 *cm = reinterpret_cast<float2 *>(cj + kRows * D);
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
            if (kC > 1) {
                *reinterpret_cast<float4 *>(cj + r * D + d) = acc;
                if (d == 0) cm[r] = make_float2(m, l);
            } else if (whole) {
                write_out(r, d, acc, m, l);
            } else {
                write_part(slot, r, d, acc, m, l);
            }
        }
        if constexpr (kC > 1) {
            // each CTA joins its share of the outputs, the parts in the order of the keys
            cg::cluster_group cl = cg::this_cluster();
            cl.sync();
            const int all = rows * (D / 4), each = (all + kC - 1) / kC, from = int(cta % kC) * each;
            for (int i = from + tid; i < min(from + each, all); i += kThreads) {
                const int r = i / (D / 4), d = i % (D / 4) * 4;
                float2 ml[kC];
                float4 v[kC];
                float m = kNegInf, l = 0.f;
#pragma unroll
                for (int k = 0; k < kC; ++k) {
                    ml[k] = *cl.map_shared_rank(cm + r, k);
                    v[k] = *cl.map_shared_rank(reinterpret_cast<float4 *>(cj + r * D + d), k);
                }
#pragma unroll
                for (int k = 0; k < kC; ++k) m = fmaxf(m, ml[k].x);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kC; ++k) {
                    const float f = ml[k].x == kNegInf ? 0.f : ex2(ml[k].x - m);
                    l = fmaf(f, ml[k].y, l);
                    acc.x = fmaf(f, v[k].x, acc.x);
                    acc.y = fmaf(f, v[k].y, acc.y);
                    acc.z = fmaf(f, v[k].z, acc.z);
                    acc.w = fmaf(f, v[k].w, acc.w);
                }
                write_out(r, d, acc, m, l);
            }
            cl.sync();  // no CTA leaves while another reads its part
            return;
        }
        if (!whole) {
            const uint32_t n = n_parts, groups = (n + kGroup - 1) / kGroup, k = (cta - c0) / kGroup;
            const uint32_t first_cta = c0 + k * kGroup, members = min(kGroup, n - k * kGroup);
            auto slot_of = [&](uint32_t i) { return (size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0); };  // i-th CTA of the pair
            float *sm = reinterpret_cast<float *>(smem);
            if (arrive_last(parts.words + first_cta, k == 0 ? 10 : 20, members, &last_flag)) {
                auto member = [&](uint32_t i) { return slot_of(k * kGroup + i); };
                if (groups == 1) {
                    join_parts<D>(parts, members, rows, sm, member, write_out);
                } else {
                    const size_t to = slot_of(k * kGroup);  // in the place of the group's first
                    join_parts<D>(parts, members, rows, sm, member,
                                  [&](int r, int d, float4 v, float m, float l) { write_part(to, r, d, v, m, l); });
                    if (arrive_last(parts.words + c0, 0, groups, &last_flag))
                        join_parts<D>(parts, groups, rows, sm, [&](uint32_t i) { return slot_of(i * kGroup); }, write_out);
                }
            }
        }
        __syncthreads();  // the join's buffers become the ring again
    }
}

// CTAs of a pair's cluster, or 0: as many clusters as the machine holds at two CTAs an SM (a little
// fewer than their number says: eight CTAs find places within one part of the chip only), and no
// sequence with more than 8 steps a warp (104 pairs of up to 1819 keys, 14 steps: 13.8 us with
// clusters of two, 12.2 scheduled; 40 pairs of up to 1989, clusters of four: 9.3, 9.6).
// Where a window bounds the keys most pairs have as many, and a warp may have more steps: 12, and 40 if there are more
// than 16 pairs.  us of a call with clusters (their size), and scheduled:
//   pairs  window   16 bits                8 bits
//     256    2048   46.9 (1)      51.3     27.7    31.1
//      64    9000   50.4 (4)      55.0     28.8    36.4
//       4    9000   18.4 (8)      16.1     12.4    11.7      why eight stop at 12 steps (sixteen go on, below)
// With a window or over an 8-bit cache up to eight pairs may have clusters of sixteen, which few parts of the chip hold
// two of (16 pairs, window 300: 10.8 us, clusters of eight 5.4).  us of a call with sixteen, and with eight (from 12000 on:
// scheduled):
//   pairs  window   16 bits                8 bits
//       4     300   5.2            4.8     4.8      4.7
//       4    1000   5.5            6.1     5.0      5.5      sixteen from 600 keys on
//       4    4097   8.5           11.3     6.8      8.4
//       4   12000   14.3          16.7     10.3    12.1
//       1   14000   15.6          14.5     -        -        why sixteen stop at 12 steps too
//       8    2500   9.4            8.8     7.2      7.1
//       8    4097   10.9          11.5     8.0      8.5      sixteen from 3200 keys on
//       8   12000   16.4          17.4     12.1    13.3
template <Mode kMode>
int cluster_of(const moe_attn_shape &s, int64_t keys) {
    const int64_t pairs = (int64_t)s.n_seqs * s.n_kv_heads;
    if (kMode != kAll && pairs <= 8 && keys > (pairs <= 4 ? 600 : 3200)) {
        const int steps = keys >= (int64_t)s.max_pages * s.page_size ? 8 : 12;
        if (keys <= steps * kWarps * kStep * 16) return 16;
    }
    const int steps = keys >= (int64_t)s.max_pages * s.page_size ? 8 : pairs > 16 ? 40 : 12;
    const int sizes[4] = {8, 4, 2, 1}, most[4] = {32, 72, 152, 304};
    for (int i = 0; i < 4; ++i)
        if (pairs <= most[i]) return keys <= steps * kWarps * kStep * sizes[i] ? sizes[i] : 0;
    return 0;
}

template <int D, int kCluster, Mode kMode, bool kHalf>
cudaError_t launch_typed(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int grid, cudaStream_t st) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, kCluster, kMode, kHalf>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (Cfg<D, kMode>::kSmem));
        if (e != cudaSuccess) return e;
        if (kCluster > 8) {
            const cudaError_t e =
                cudaFuncSetAttribute(decode_kernel<D, kCluster, kMode, kHalf>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
        }
        attr_set[dev] = true;
    }
    float *o = reinterpret_cast<float *>(ws);
    float2 *ml = reinterpret_cast<float2 *>(o + (size_t)kMaxGrid * 2 * kRows * D);
    const Parts p{reinterpret_cast<uint32_t *>(hdr + kCounters), o, ml};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster > 0 ? kCluster : 1;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kCluster > 0 ? unsigned(s.n_seqs * s.n_kv_heads * kCluster) : unsigned(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (Cfg<D, kMode>::kSmem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, decode_kernel<D, kCluster, kMode, kHalf>, a, p);
}

template <int kCluster, Mode kMode, bool kHalf>
cudaError_t launch_dim(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int grid, cudaStream_t st) {
    return s.head_dim == 128 ? launch_typed<128, kCluster, kMode, kHalf>(a, s, hdr, ws, grid, st)
                             : launch_typed<64, kCluster, kMode, kHalf>(a, s, hdr, ws, grid, st);
}

template <Mode kMode, bool kHalf = false>
cudaError_t launch(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int sms, cudaStream_t st) {
    const int grid = sms * kCtasPerSm < kMaxGrid ? sms * kCtasPerSm : kMaxGrid;
    int64_t keys = (int64_t)s.max_pages * s.page_size;  // of a pair, at most: with a window its steps' only
    if (kMode != kAll) keys = std::min(keys, (int64_t)a.window + a.sinks + s.max_q + 2 * kStep);
    const int cluster = cluster_of<kMode>(s, keys);
    if constexpr (kMode != kAll) {
        if (cluster == 16) return launch_dim<16, kMode, kHalf>(a, s, hdr, ws, grid, st);
    }
    switch (cluster) {
    case 8: return launch_dim<8, kMode, kHalf>(a, s, hdr, ws, grid, st);
    case 4: return launch_dim<4, kMode, kHalf>(a, s, hdr, ws, grid, st);
    case 2: return launch_dim<2, kMode, kHalf>(a, s, hdr, ws, grid, st);
    case 1: return launch_dim<1, kMode, kHalf>(a, s, hdr, ws, grid, st);
    default: return launch_dim<0, kMode, kHalf>(a, s, hdr, ws, grid, st);
    }
}

}  // namespace
}  // namespace attn
}  // namespace moe
