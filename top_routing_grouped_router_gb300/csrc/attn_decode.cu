// attn_decode.cu -- attention of a few new tokens a sequence (decode, draft tokens) over the
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
// Where the host sees that the pairs are few and no sequence can be long, a cluster of eight, four
// or two CTAs (or one CTA) takes each pair: nothing is scheduled on the device, and the parts meet
// in shared memory (8 sequences of 150 to 1100 keys, 4 key heads: 7.5 us, 9.3 through the
// workspace; one sequence of 2000 keys 7.1 us, 9.3).
#include "attn.cuh"

#include <cooperative_groups.h>

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
// 2^x by the hardware unit (relative error about 2^-22; 0 for -inf).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int steps_of(const Seq &s) {
    return s.q_len ? max(1, int((uint32_t(s.kv_len) + kStep - 1) / kStep)) : 0;  // kv_len up to 2^31 - 1
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
template <int D, int kCluster>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(Args a, Parts parts) {
    namespace cg = cooperative_groups;
    using C = Cfg<D>;
    constexpr bool kClustered = kCluster > 0;
    constexpr int kC = kClustered ? kCluster : 1;
    // the join's buffers: [warp][row][D], [warp][row] (max, sum); clustered, after them [row][D], [row]
    constexpr int kJoinFloats = kWarps * kRows * (D + 2);
    static_assert((kJoinFloats + kRows * (D + 2)) * 4 <= C::kSmem, "");
    constexpr int NT = D / 8;        // 8-column tiles of O
    constexpr int KS = D / 16;       // 16-element steps of the head dimension
    constexpr int CH = D / 8;        // 16-byte pieces of a row
    constexpr int RPI = 32 / CH;     // rows a warp copies per instruction
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
        steps = steps_of(s);
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
                n0 = steps_of(s);
            }
            pairs = __popc(__ballot_sync(0xffffffffu, n0 > 0)) * Hkv;
            before0 = warp_scan(n0 * Hkv, &total);
        }
        for (int b0 = 0; !few && b0 < a.n_seqs; b0 += kThreads) {
            uint32_t n = 0, sum;
            if (b0 + tid < a.n_seqs) {
                const Seq x = load_seq(a, b0 + tid);
                n = steps_of(x);
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
                        n = places_of(steps_of(x));
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
        steps = steps_of(s);
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
                steps = steps_of(s);
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
        const int rows = min(s.q_len * int(G), kRows), past = s.kv_len - s.q_len;

        // the warp's keys: steps step0 + warp, + kWarps, ...  The cache offset of lane r's key row (r <
        // 16), or of the first row where a step lies within a page, is found a step before the copy.
        const int mine = step1 - step0 > uint32_t(warp) ? int(step1 - step0 - warp + kWarps - 1) / kWarps : 0;
        const bool in_page = a.page_size % kStep == 0;
        auto find_row = [&](int i) -> int64_t {
            const int p = int(step0 + warp + i * kWarps) * kStep + (in_page ? 0 : lane & 15);
            if (i >= mine || p >= s.kv_len) return -1;
            const int pi = a.page_shift >= 0 ? p >> a.page_shift : p / a.page_size;
            return load_page(a, b, pi) * a.page_stride + (int64_t)(p - pi * a.page_size) * a.token_stride;
        };
        const uint16_t *kc = static_cast<const uint16_t *>(a.k) + h * a.head_stride + lane % CH * 8;
        const uint16_t *vc = static_cast<const uint16_t *>(a.v) + h * a.head_stride + lane % CH * 8;
        const int64_t lane_row = (int64_t)(lane / CH) * a.token_stride, next_row = (int64_t)RPI * a.token_stride;
        // rows it * RPI + lane / CH: the swizzle's row bits repeat every 8 rows
        auto copy = [&](int i, int64_t row_off) {
            if (i < mine) {
                const uint32_t dst = ring + (i % C::kStages) * C::kStageBytes + lane / CH * (D * 2);
                const int p = int(step0 + warp + i * kWarps) * kStep;
                if (in_page && s.kv_len - p >= kStep) {
                    const uint16_t *ks = kc + row_off + lane_row, *vs = vc + row_off + lane_row;
#pragma unroll
                    for (int it = 0; it < kStep / RPI; ++it, ks += next_row, vs += next_row) {
                        const uint32_t to = dst + it * RPI * (D * 2) + (((lane % CH) ^ ((it * RPI + lane / CH) & 7)) * 16);
                        cp16(to, ks, 16);
                        cp16(to + kStep * D * 2, vs, 16);
                    }
                } else {
#pragma unroll
                    for (int it = 0; it < kStep / RPI; ++it) {
                        const int r = it * RPI + lane / CH;
                        int64_t off = __shfl_sync(0xffffffffu, row_off, in_page ? 0 : r);
                        if (in_page) off += r * a.token_stride;
                        const int n = p + r < s.kv_len ? 16 : 0;  // rows past the last key: zeros, nothing is read
                        const uint32_t to = dst + it * RPI * (D * 2) + (((lane % CH) ^ (r & 7)) * 16);
                        cp16(to, kc + (n ? off : 0), n);
                        cp16(to + kStep * D * 2, vc + (n ? off : 0), n);
                    }
                }
            }
            cp_commit();
        };
        int64_t next = find_row(0);

        // Q as A fragments: rows g and g + 8, columns 16 ks + 2 t4 (+1) and + 8; a row past the
        // last reads the first one's and is zeroed, so that all loads go out together
        uint32_t q[KS][4];
        const uint16_t *qp = static_cast<const uint16_t *>(a.q) + (int64_t)s.q0 * a.q_stride + (int64_t)h * G * D + t4 * 2;
        const bool on0 = g < rows, on1 = g + 8 < rows;
        const uint32_t r0 = on0 ? g : 0, r1 = on1 ? g + 8 : 0, j0 = r0 / G, j1 = r1 / G;
        const uint16_t *q0 = qp + j0 * a.q_stride + (r0 - j0 * G) * D, *q1 = qp + j1 * a.q_stride + (r1 - j1 * G) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            q[ks][0] = ldp(reinterpret_cast<const uint32_t *>(q0 + ks * 16));
            q[ks][2] = ldp(reinterpret_cast<const uint32_t *>(q0 + ks * 16 + 8));
        }
        if (rows > 8) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                q[ks][1] = ldp(reinterpret_cast<const uint32_t *>(q1 + ks * 16));
                q[ks][3] = ldp(reinterpret_cast<const uint32_t *>(q1 + ks * 16 + 8));
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) q[ks][1] = q[ks][3] = 0u;
        }
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) {
            const int64_t cur = next;
            next = find_row(i + 1);
            copy(i, cur);
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[ks][e] = ((e & 1) ? on1 : on0) ? q[ks][e] : 0u;
        const int seen0 = on0 ? past + int(j0) + 1 : 0, seen1 = on1 ? past + int(j1) + 1 : 0;
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
            const int key0 = int(step0 + warp + i * kWarps) * kStep;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[n][e] *= sl2;
            if (key0 > seen_all - kStep) {
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
            if (rows > 8)
                *reinterpret_cast<float2 *>(jo + (warp * kRows + g + 8) * D + j * 8 + t4 * 2) = make_float2(o[j][2], o[j][3]);
        }
        if (t4 == 0) {
            jm[warp * kRows + g] = make_float2(m0, l0);
            jm[warp * kRows + g + 8] = make_float2(m1, l1);
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
int cluster_of(const moe_attn_shape &s) {
    const int64_t pairs = (int64_t)s.n_seqs * s.n_kv_heads, keys = (int64_t)s.max_pages * s.page_size;
    const int sizes[4] = {8, 4, 2, 1}, most[4] = {32, 72, 152, 304};
    for (int i = 0; i < 4; ++i)
        if (pairs <= most[i]) return keys <= 8 * kWarps * kStep * sizes[i] ? sizes[i] : 0;
    return 0;
}

template <int D, int kCluster>
cudaError_t launch_typed(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int grid, cudaStream_t st) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, kCluster>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
        if (e != cudaSuccess) return e;
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
    cfg.dynamicSmemBytes = Cfg<D>::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, decode_kernel<D, kCluster>, a, p);
}

template <int kCluster>
cudaError_t launch_dim(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int grid, cudaStream_t st) {
    return s.head_dim == 128 ? launch_typed<128, kCluster>(a, s, hdr, ws, grid, st)
                             : launch_typed<64, kCluster>(a, s, hdr, ws, grid, st);
}

}  // namespace

// bf16, head sizes 64 and 128, at most 16 query rows a key head, and a line of steps that
// 32 bits count even if every sequence fills its row of the block table.
bool decode_supported(const moe_attn_shape &s) {
    const double steps = double(s.n_seqs) * s.n_kv_heads * ((double)s.max_pages * s.page_size / kStep + 1);
    return s.dtype == MOE_DT_BF16 && (s.head_dim == 64 || s.head_dim == 128) &&
           (int64_t)s.max_q * (s.n_heads / s.n_kv_heads) <= kRows && steps < 2147483648.0;
}
size_t decode_ws_bytes(const moe_attn_shape &s) { return (size_t)kMaxGrid * 2 * kRows * (s.head_dim + 2) * 4; }

cudaError_t launch_decode(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int sms, cudaStream_t st) {
    const int grid = sms * kCtasPerSm < kMaxGrid ? sms * kCtasPerSm : kMaxGrid;
    switch (cluster_of(s)) {
    case 8: return launch_dim<8>(a, s, hdr, ws, grid, st);
    case 4: return launch_dim<4>(a, s, hdr, ws, grid, st);
    case 2: return launch_dim<2>(a, s, hdr, ws, grid, st);
    case 1: return launch_dim<1>(a, s, hdr, ws, grid, st);
    default: return launch_dim<0>(a, s, hdr, ws, grid, st);
    }
}

}  // namespace attn
}  // namespace moe
