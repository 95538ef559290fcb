// attn_chunk.cu -- attention of chunks of new tokens over the paged cache on the 5th-generation
// tensor cores (bf16, head sizes 64 and 128).
//
// The query rows that share a key head (tokens x heads of the group) form tiles of up to 128
// rows.  A CTA works on two tiles at a time ("item": a sequence, a key head, 2 x 128 rows) and
// goes over the keys in steps of 128:
//   S_t = Q_t K^T      M = 128, N = 128, into TMEM
//   P_t = 2^(S_t - m)  by four warps per tile, one row a thread, to TMEM as bf16
//   O_t += P_t V       A = P_t from TMEM, V as it lies in the cache (keys x head: N-major)
// Heads of 128: P_t takes the place of S_t (TMEM is full), and one warp issues P0 V, S0', P1 V, S1':
// while one tile's softmax runs, the tensor cores work on the other's products.  What bounds it is
// that chain: 1400 cycles of softmax and 1024 of products a tile, 2890 a step of both tiles where the
// products alone are 2048 (2048 tokens over 16384 keys, 32 heads: 333 us by itself, 1550 TFLOP/s; 360 with its
// join in a row of calls, when the clocks fall).  Multiplying the first half of P while the softmax works on the
// second made it slower (by 6 %).
// Heads of 64: P_t lies beside S_t, the next scores are computed while the softmax works, and each
// tile has an MMA warp of its own.
// The running maximum m may lag behind: only when a row's maximum grows by more than 2^8 is O
// rescaled (by the softmax warps, in TMEM); until then the larger probabilities are exact in bf16
// terms all the same, since the scale of a row cancels.
//
// K and V tiles come by TMA through the block table, one box a page.  All items are laid end
// to end as steps of 128 keys and each CTA takes an equal share of that line; items cut by a
// share's end leave fp32 partial results that a second kernel joins.
#include "attn.cuh"
#include "tma_nd.cuh"

namespace moe {
namespace attn {
namespace {

using namespace tc;

// Warps 0-3, 4-7: softmax of tile 0, 1; the third warpgroup: MMAs, loads, the list of
// segments, and with heads of 64 the MMAs of tile 1.  It gives up registers that the softmax takes: 8 x 32 x 208 + 4 x 32 x 80 is within the launch's
// 12 x 32 x 168.
constexpr int kThreads = 384, kLaunchRegs = 168, kSoftmaxRegs = 208, kOtherRegs = 80;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kListWarp = 10, kMma1Warp = 11;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "");
constexpr int kM = 128, kKeys = 128;
constexpr int kMaxCtas = 160;   // one per SM (152)
constexpr int kMaxSegs = 16;    // segments prepared at a time
constexpr float kLag = 8.f;     // log2 of the growth of a row's maximum that O tolerates
constexpr int kJoinRows = 16;   // rows of a block of the join kernel

template <int D>
struct Cfg {
    static constexpr int kTile = kM * D * 2;                  // one Q tile, one K or V stage
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kSmem = 2 * kTile + kStages * kTile + 1024 + 2048;
    static_assert(kSmem <= 232448, "");
    // TMEM columns of tile t: S at 128 t, P and O here.  Heads of 64 leave room for P beside S: the scores
    // of the next step are computed while the softmax works on this one's, which the softmax holds in
    // registers.  Heads of 128 do not: P takes the place of S.
    static constexpr bool kEarly = D == 64;
    // Warps that issue MMAs, each for its tiles.  With heads of 128 one, in the order of the tiles, which
    // keeps one tile's products beside the other's softmax (two: 420 us for a chunk of 2048, one at the time: 341);
    // with heads of 64, whose products are half as long, two (a mixed batch 48.4 us, with one 51).
    static constexpr int kMmaWarps = D == 64 ? 2 : 1;
    static constexpr uint32_t col_p(int t) { return kEarly ? 256 + 64 * t : 128 * t; }
    static constexpr uint32_t col_o(int t) { return kEarly ? 384 + 64 * t : 256 + 128 * t; }
};

// One item, or the part of it in this CTA's share.
struct Seg {
    int b, h, tok0, q0, q_len, kv_len;  // tok0: first token of the chunk in the item
    int step0, step1;                   // key steps of this share
    int slot;                           // -1: whole item; else the slot of the partial results
    int tiles;                          // 1 or 2
};
// What the join kernel needs of an item that starts in a CTA's share and goes on past it.
struct Rec {
    int n, h, tok0, q0, q_len;  // n: parts (0: none)
};

// sum_{i < n} floor((a i + b) / m), m > 0, as Euclid's algorithm goes: whole multiples of m are taken out of a and b,
// then rows and columns of the lattice points under the line change places (reciprocity of such sums: Graham,
// Knuth, Patashnik, Concrete Mathematics, chapter 3).  The sum and a n + m fit 32 bits.
__device__ __forceinline__ uint32_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
    uint32_t sum = 0;
    while (n > 0) {
        if (a >= m) {
            sum += uint32_t(uint64_t(n) * (n - 1) / 2) * (a / m);
            a %= m;
        }
        if (b >= m) {
            sum += n * (b / m);
            b %= m;
        }
        const uint32_t y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const uint32_t t = a;
        a = m;
        m = t;
    }
    return sum;
}

// Tokens of an item, and their logarithm (-1 if they are no power of two).
struct Item {
    uint32_t tokens;
    int shift;
    __device__ __forceinline__ uint32_t div(uint32_t x) const { return shift >= 0 ? x >> shift : x / tokens; }
};

// sum_{i < n} floor((tokens i + b) / kKeys).  Tokens that are a power of two need no division: below
// kKeys, floor((i + floor(b / tokens)) / p) with p = kKeys / tokens.
__device__ __forceinline__ uint32_t step_sum(uint32_t n, Item it, uint32_t b) {
    constexpr int kLog = 7;
    static_assert(kKeys == 1 << kLog, "");
    if (it.shift < 0) return floor_sum(n, kKeys, it.tokens, b);
    if (n == 0) return 0;
    if (it.shift >= kLog) return (uint32_t((uint64_t)n * (n - 1) / 2) << (it.shift - kLog)) + n * (b >> kLog);
    const int lp = kLog - it.shift;
    const uint32_t b1 = b >> it.shift;
    auto f = [lp](uint32_t x) {  // sum_{j < x} floor(j / p)
        const uint32_t q = x >> lp;
        return ((q * (q - 1) / 2) << lp) + q * (x - (q << lp));
    };
    return f(b1 + n) - f(b1);
}

// Steps of item i of a chunk: the keys that its last token sees, at least one step.
__device__ __forceinline__ uint32_t item_steps(const Seq &s, uint32_t i, Item it) {
    const int64_t keys = min((int64_t)s.kv_len - s.q_len + (int64_t)(i + 1) * it.tokens, (int64_t)s.kv_len);
    return keys <= kKeys ? 1u : (uint32_t(keys) + kKeys - 1) / kKeys;
}
__device__ __forceinline__ uint32_t items_of(const Seq &s, Item it) { return it.div(s.q_len + it.tokens - 1); }

// Steps of items [0, i) of a chunk.
__device__ __forceinline__ uint32_t steps_before(const Seq &s, uint32_t i, Item it) {
    if (i == 0) return 0;
    const uint32_t n = items_of(s, it);
    const uint32_t last = i == n ? item_steps(s, n - 1, it) : 0;
    const uint32_t full = i == n ? n - 1 : i;  // items that hold all their tokens
    const int64_t past = (int64_t)s.kv_len - s.q_len;
    // items that see no key have one step each
    const uint32_t none = past < 0 ? min(full, it.div(uint32_t(-past))) : 0;
    const uint32_t b = uint32_t(past + (int64_t)(none + 1) * it.tokens + kKeys - 1);  // > kKeys - 1
    return none + step_sum(full - none, it, b) + last;
}

// On the line of all steps an item takes kSetup places more than its steps, at its front: what
// starting and ending an item costs, about two steps' time (a mixed batch of short and long
// items: 85 us with none, the slowest CTA 1.45 times the mean).
constexpr uint32_t kSetup = 2;
__device__ __forceinline__ uint32_t places_before(const Seq &s, uint32_t i, Item it, bool whole) {
    return whole ? i : steps_before(s, i, it) + i * kSetup;
}
// Where no sequence can hold more keys than this, items are not cut (each takes one place on the
// line), and the join is not launched.
constexpr int kWholeKeys = 512;

struct Shares {
    uint32_t each, more;
    __device__ __forceinline__ uint32_t begin(uint32_t cta) const { return cta * each + min(cta, more); }
    __device__ __forceinline__ uint32_t owner(uint32_t step) const {
        const uint32_t edge = more * (each + 1);
        return step < edge ? step / (each + 1) : more + (step - edge) / each;
    }
};


__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 columns of this thread's TMEM lane, no wait; the wait is tmem_ld_done.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t ta, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(ta)
        : "memory");
}
// Waits for every load of the thread; r passes through so that no use moves above the wait.
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[128]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 128; ++i) asm volatile("" : "+r"(r[i]));
}

// Matrix descriptor of a V tile as the B operand of P V: keys x 64-element slabs of the head,
// 128-byte rows (one key's 64 elements), 128-byte swizzle, N-major: 8-key groups 1024 B apart
// (stride offset), slabs kKeys * 128 B apart (leading offset).
__device__ __forceinline__ uint64_t v_desc(uint32_t addr) {
    return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t((kKeys * 128) >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// The MMAs of one product in one block of assembly: one election, and descriptors that differ by
// constants, so that the issuing warp needs few of the issue slots that the softmax warps fill.
// (Written as separate calls an MMA took 147 cycles to issue next to them, 64 to run.)
// S: D / 16 MMAs over the 64-element slabs of Q and K (128 rows x 128 bytes each), then a commit.
template <int D>
__device__ __forceinline__ void mma_s(uint32_t d, uint64_t q, uint64_t k, uint32_t idesc, uint32_t bar) {
    if constexpr (D == 128) {
        asm volatile(
            "{\n\t.reg .pred e, z;\n\t.reg .b64 q, k;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 z, %3, %3;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, z;\n\tsetp.eq.b32 z, %3, %3;\n\t"
            "add.s64 q, %1, 2;\n\tadd.s64 k, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "add.s64 q, %1, 4;\n\tadd.s64 k, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "add.s64 q, %1, 6;\n\tadd.s64 k, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "add.s64 q, %1, 1024;\n\tadd.s64 k, %2, 1024;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "add.s64 q, %1, 1026;\n\tadd.s64 k, %2, 1026;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "add.s64 q, %1, 1028;\n\tadd.s64 k, %2, 1028;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "add.s64 q, %1, 1030;\n\tadd.s64 k, %2, 1030;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}"
            ::"r"(d), "l"(q), "l"(k), "r"(idesc), "r"(bar)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, z;\n\t.reg .b64 q, k;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 z, %3, %3;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, z;\n\tsetp.eq.b32 z, %3, %3;\n\t"
            "add.s64 q, %1, 2;\n\tadd.s64 k, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "add.s64 q, %1, 4;\n\tadd.s64 k, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "add.s64 q, %1, 6;\n\tadd.s64 k, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], q, k, %3, z;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}"
            ::"r"(d), "l"(q), "l"(k), "r"(idesc), "r"(bar)
            : "memory");
    }
}
// O (+)= P V over 128 keys: 8 MMAs, P at TMEM columns p + 8 i, V 2048 bytes (16 keys) further each.
__device__ __forceinline__ void mma_o(uint32_t d, uint32_t p, uint64_t v, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, z;\n\t.reg .b64 v;\n\t.reg .b32 p;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 z, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, z;\n\tsetp.eq.b32 z, %3, %3;\n\t"
        "add.s32 p, %1, 8;\n\tadd.s64 v, %2, 128;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %3, z;\n\t"
        "add.s32 p, %1, 16;\n\tadd.s64 v, %2, 256;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %3, z;\n\t"
        "add.s32 p, %1, 24;\n\tadd.s64 v, %2, 384;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %3, z;\n\t"
        "add.s32 p, %1, 32;\n\tadd.s64 v, %2, 512;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %3, z;\n\t"
        "add.s32 p, %1, 40;\n\tadd.s64 v, %2, 640;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %3, z;\n\t"
        "add.s32 p, %1, 48;\n\tadd.s64 v, %2, 768;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %3, z;\n\t"
        "add.s32 p, %1, 56;\n\tadd.s64 v, %2, 896;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [p], v, %3, z;\n\t}"
        ::"r"(d), "r"(p), "l"(v), "r"(idesc), "r"(acc)
        : "memory");
}

// The block's barrier where its warps are in different code, and its form that ORs a value.
__device__ __forceinline__ void meet() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ bool meet_any(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(uint32_t(v)), "n"(kThreads) : "memory");
    return r != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

struct Ctx {
    Args a;
    uint32_t tt;        // tokens of a tile
    int item_shift;     // log2(2 tt), -1 if that is no power of two
    float *part_o;      // [slot][D / 4][2 * kM][4]: a warp's rows side by side
    float2 *part_ml;    // [slot][2 * kM]
    Rec *rec;           // [kMaxCtas]
    unsigned long long wait_ns;
    int extra_need;
    bool whole;         // items are not cut
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ CUtensorMap map_q,
                                                            const __grid_constant__ CUtensorMap map_k,
                                                            const __grid_constant__ CUtensorMap map_v,
                                                            const __grid_constant__ Ctx c) {
    using C = Cfg<D>;
    constexpr int kSlabs = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *ctrl = smem + (2 + C::kStages) * C::kTile;
    uint64_t *kv_full = reinterpret_cast<uint64_t *>(ctrl);  // [kStages]
    uint64_t *kv_empty = kv_full + C::kStages;               // [kStages]
    uint64_t *q_full = kv_empty + C::kStages, *q_empty = q_full + 1;
    uint64_t *s_full = q_empty + 1, *s_empty = s_full + 2, *p_full = s_empty + 2, *o_full = p_full + 2, *o_empty = o_full + 2;  // [2] each
    uint64_t *v_zero = o_empty + 2, *drain = v_zero + C::kStages;  // [kStages], [2]
    Seg *segs = reinterpret_cast<Seg *>(drain + 2);  // [kMaxSegs]
    uint32_t *scan = reinterpret_cast<uint32_t *>(segs + kMaxSegs);  // [16]
    int *nseg = reinterpret_cast<int *>(scan + 16);
    volatile int *abort = nseg + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(nseg + 2);
    uint32_t *cursor = tmem_slot + 1;  // [4]: sequence, its first step, its steps per head, step within the line
    Seq *cur_seq = reinterpret_cast<Seq *>(cursor + 4);

    const Args &a = c.a;
    const Waits wt{a.err, abort, c.wait_ns, smem_u32(const_cast<int *>(abort))};
    // the warp's number from one lane: the compiler then knows it to be the same in all of them, and the
    // MMA warp's addresses and descriptors stay in the uniform registers that its instructions take
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t tt = c.tt, tt2 = 2 * tt, G = a.group, Hkv = a.n_kv_heads;
    const Item it{tt2, c.item_shift};
    if (tid == kLoadWarp * 32) {
        for (const CUtensorMap *p : {&map_q, &map_k, &map_v})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(p)) : "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&kv_full[i]), 1);
            mbar_init(smem_u32(&kv_empty[i]), C::kMmaWarps);
            mbar_init(smem_u32(&v_zero[i]), 1);
        }
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(q_empty), C::kMmaWarps);
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&s_full[t]), 1);
            mbar_init(smem_u32(&s_empty[t]), kM);
            mbar_init(smem_u32(&p_full[t]), kM + c.extra_need);
            mbar_init(smem_u32(&o_full[t]), 1);
            mbar_init(smem_u32(&o_empty[t]), kM);
        }
        mbar_init(smem_u32(&drain[0]), 1);
        mbar_init(smem_u32(&drain[1]), 1);
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
    griddep_wait();
    griddep_launch_dependents();

    // ---------------------------------------------------------------- the CTA's share
    // Steps of all heads of the sequences, scanned over the block in chunks of kThreads.
    auto scan_block = [&](uint32_t n, uint32_t *sum) {
        uint32_t incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        uint32_t before = 0, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            before += w < warp ? scan[w] : 0;
            total += scan[w];
        }
        *sum = total;
        return before + incl - n;
    };
    auto seq_places = [&](const Seq &s) { return places_before(s, items_of(s, it), it, c.whole); };
    uint32_t total = 0, n0 = 0, before0 = 0;
    bool rows_ok = true;
    Seq s0{};
    const bool few = a.n_seqs <= 32;  // every warp scans by itself, without barriers
    if (few) {
        if (lane < a.n_seqs) {
            s0 = load_seq(a, lane);
            n0 = seq_places(s0) * Hkv;
            rows_ok = s0.rows_ok;
        }
        uint32_t incl = n0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        before0 = incl - n0;
        total = __shfl_sync(0xffffffffu, incl, 31);
        rows_ok = __all_sync(0xffffffffu, rows_ok);
    } else {
        for (int b0 = 0; b0 < a.n_seqs; b0 += kThreads) {
            uint32_t n = 0, sum;
            Seq s{};
            if (b0 + tid < a.n_seqs) {
                s = load_seq(a, b0 + tid);
                n = seq_places(s) * Hkv;
                rows_ok = rows_ok && s.rows_ok;
            }
            const uint32_t before = scan_block(n, &sum);
            if (b0 == 0) {
                n0 = n;
                before0 = before;
                s0 = s;
            }
            total += sum;
        }
        rows_ok = !__syncthreads_or(!rows_ok);
    }
    // chunks that overlap could make a line longer than 32 bits count: such a call does nothing (the
    // error is recorded)
    if (!rows_ok) total = 0;
    const uint32_t cta = blockIdx.x, ctas = max(1u, min(gridDim.x, c.whole ? total : total / (kSetup + 2)));
    const Shares sh{total / ctas, total % ctas};
    const uint32_t u_begin = cta < ctas ? sh.begin(cta) : 0, u_end = cta < ctas ? sh.begin(cta + 1) : 0;
    if (tid == 0 && !c.whole) c.rec[cta].n = 0;
    if (u_begin < u_end) {
        auto found = [&](int b, uint32_t before, uint32_t n, const Seq &s) {
            if (u_begin >= before && u_begin - before < n) {
                cursor[0] = b;
                cursor[1] = before;
                cursor[2] = n / Hkv;
                *cur_seq = s;
            }
        };
        if (!few || warp == 0) found(few ? lane : tid, before0, n0, s0);
        uint32_t base = 0;
        for (int b0 = 0; a.n_seqs > kThreads && b0 < a.n_seqs; b0 += kThreads) {
            uint32_t n = 0, sum;
            Seq s{};
            if (b0 + tid < a.n_seqs) {
                s = load_seq(a, b0 + tid);
                n = seq_places(s) * Hkv;
            }
            const uint32_t before = base + scan_block(n, &sum);
            found(b0 + tid, before, n, s);
            base += sum;
            if (u_begin < base) break;
        }
        if (tid == 0) cursor[3] = u_begin;
    }
    __syncthreads();

    // ---------------------------------------------------------------- roles
    // the next segments, up to kMaxSegs, by one warp
    auto list = [&]() {
        int b = int(cursor[0]);
        uint32_t first = cursor[1], per_head = cursor[2], w = cursor[3];
        Seq s = *cur_seq;
        int k = 0;
        uint32_t h = 0, i = 0, item0 = 0;
        bool located = false;
        while (w < u_end && k < kMaxSegs) {
            if (!located) {
                while (w - first >= per_head * Hkv) {  // the next sequence with a chunk
                    first += per_head * Hkv;
                    if (++b >= a.n_seqs) break;  // not seen: the line ends with the last sequence
                    s = load_seq(a, b);
                    per_head = seq_places(s);
                }
                if (b >= a.n_seqs) {
                    w = u_end;
                    break;
                }
                h = (w - first) / per_head;
                const uint32_t rem = w - first - h * per_head;
                // the last item that begins at or before rem: 32 candidates a round
                uint32_t lo = 0, n = items_of(s, it), at_lo = 0;
                while (n > 1) {
                    const uint32_t each = (n + 31) / 32, cand = lo + lane * each;
                    const uint32_t before = lane * each < n ? places_before(s, cand, it, c.whole) : ~0u;
                    const uint32_t last = 31 - __clz(__ballot_sync(0xffffffffu, before <= rem));
                    at_lo = __shfl_sync(0xffffffffu, before, last);
                    lo += last * each;
                    n = min(each, n - last * each);
                }
                i = lo;
                item0 = first + h * per_head + at_lo;
                located = true;
            }
            const uint32_t steps = item_steps(s, i, it), setup = c.whole ? 0 : kSetup;
            const uint32_t places = c.whole ? 1 : steps + kSetup, end = min(item0 + places, u_end);
            // steps begin after the item's setup; a share that ends within it leaves the item to the next
            const uint32_t from = max(w, item0 + setup);
            const bool starts = from == item0 + setup, whole = starts && end == item0 + places;
            if (from < end) {
                if (lane == 0) {
                    Seg g;
                    g.b = b;
                    g.h = int(h);
                    g.tok0 = int(i * tt2);
                    g.q0 = s.q0;
                    g.q_len = s.q_len;
                    g.kv_len = s.kv_len;
                    g.step0 = int(from - item0 - setup);
                    g.step1 = c.whole ? int(steps) : int(end - item0 - setup);
                    g.slot = whole ? -1 : int(cta * 2 + (starts ? 1 : 0));
                    g.tiles = s.q_len - g.tok0 > int(tt) ? 2 : 1;
                    segs[k] = g;
                    if (!whole && starts) {
                        const int last = int(sh.owner(item0 + places - 1));
                        c.rec[cta] = Rec{last - int(cta) + 1, g.h, g.tok0, g.q0, g.q_len};
                    }
                }
                ++k;
            }
            w = end;
            if (end == item0 + places) {
                item0 += places;
                if (++i == items_of(s, it)) {
                    i = 0;
                    ++h;
                    if (h == Hkv) located = false;  // the next sequence
                }
            }
        }
        if (lane == 0) {
            *nseg = k;
            cursor[0] = b;
            cursor[1] = first;
            cursor[2] = per_head;
            cursor[3] = w;
            *cur_seq = s;
        }
    };
    bool ok = true;
    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        int stage = 0;                      // ring position
        uint32_t phase = 0, q_phase = 0;
        uint32_t p_phase = 0, oe_phase = 3, se_phase = 0;  // bit t: tile t
        uint32_t z_phase = 0;               // bit i: stage i
        uint32_t ring_waited = 0;           // load warp: stages whose fill was issued (for the drain)
        for (uint32_t u = u_begin; u < u_end && ok;) {
            if (warp == kListWarp) list();
            meet();
            const int ns = *nseg;
            u = cursor[3];
            if (warp == kLoadWarp) {
                // ------------------------------------------------ loads
                const int ps = a.page_size, box = min(ps, kKeys);
                for (int k = 0; k < ns && ok; ++k) {
                    const Seg g = segs[k];
                    const int keys = int(min((int64_t)g.kv_len - g.q_len + g.tok0 + tt2, (int64_t)g.kv_len));
                    const int boxes_max = kKeys / box;
                    auto page_of = [&](int step) {  // lane i: the page of box i of the step
                        const int p = step * kKeys + lane * box;
                        return lane < boxes_max && p < keys ? load_page(a, g.b, p / ps) : -1;
                    };
                    int page = page_of(g.step0);
                    ok = mbar_wait(smem_u32(q_empty), q_phase ^ 1, wt);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        const int rows = int(G * tt);
                        mbar_arrive_expect_tx(smem_u32(q_full), uint32_t(g.tiles * rows * D * 2));
                        for (int t = 0; t < g.tiles; ++t)
                            for (int d = 0; d < kSlabs; ++d)
                                tma_load_3d(smem_u32(smem + t * C::kTile + d * kM * 128), &map_q, d * 64, int(g.h * G),
                                            g.q0 + g.tok0 + t * int(tt), smem_u32(q_full));
                    }
                    q_phase ^= 1;
                    __syncwarp();
                    for (int step = g.step0; step < g.step1 && ok; ++step) {
                        const int next = step + 1 < g.step1 ? page_of(step + 1) : -1;
                        const int have = __popc(__ballot_sync(0xffffffffu, page >= 0));
                        for (int kv = 0; kv < 2; ++kv) {
                            ok = mbar_wait(smem_u32(&kv_empty[stage]), phase ^ 1, wt);
                            if (!__all_sync(0xffffffffu, ok)) {
                                ok = false;
                                break;
                            }
                            const uint32_t full = smem_u32(&kv_full[stage]);
                            if (lane == 0) mbar_arrive_expect_tx(full, uint32_t(have * box * D * 2));
                            __syncwarp();
                            if (page >= 0) {
                                const uint32_t dst = smem_u32(smem + (2 + stage) * C::kTile + lane * box * 128);
                                const int tok = ps > kKeys ? step * kKeys % ps : 0;
                                for (int d = 0; d < kSlabs; ++d)
                                    tma_load_4d(dst + d * kKeys * 128, kv ? &map_v : &map_k, d * 64, tok, g.h, page, full);
                            }
                            ring_waited |= 1u << stage;
                            if (++stage == C::kStages) {
                                stage = 0;
                                phase ^= 1;
                            }
                        }
                        page = next;
                    }
                }
            } else if (warp == kMmaWarp || (C::kMmaWarps == 2 && warp == kMma1Warp)) {
                // ------------------------------------------------ MMAs of tiles t0 .. t1 - 1
                const int t0 = warp == kMmaWarp ? 0 : 1, t_end = C::kMmaWarps == 2 ? t0 + 1 : 2;
                const uint32_t id_s = instr_desc(kM, kKeys), id_o = instr_desc(kM, D) | (1u << 16);
                auto wait = [&](uint64_t *bar, uint32_t par) {
                    const bool r = mbar_wait(smem_u32(bar), par, wt);
                    ok = __all_sync(0xffffffffu, r);
                    return ok;
                };
                auto advance = [&](int &st, uint32_t &ph) {
                    if (++st == C::kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                };
                auto issue_s = [&](int t, int st) {
                    const uint64_t qa = smem_desc(smem_u32(smem + t * C::kTile)), kb = smem_desc(smem_u32(smem + (2 + st) * C::kTile));
                    mma_s<D>(tmem + t * kKeys, qa, kb, id_s, smem_u32(&s_full[t]));
                };
                for (int k = 0; k < ns && ok; ++k) {
                    const Seg g = segs[k];
                    const int keys = int(min((int64_t)g.kv_len - g.q_len + g.tok0 + tt2, (int64_t)g.kv_len));
                    const int t1 = min(t_end, g.tiles);  // none: the warp only keeps step with the ring
                    if (!wait(q_full, q_phase)) break;
                    q_phase ^= 1;
                    if (!wait(&kv_full[stage], phase)) break;
                    tc_fence_after();
                    for (int t = t0; t < t1; ++t) issue_s(t, stage);
                    mma_commit_warp(smem_u32(&kv_empty[stage]));
                    advance(stage, phase);
                    if (g.step1 - g.step0 == 1) mma_commit_warp(smem_u32(q_empty));
                    for (int step = g.step0; step < g.step1 && ok; ++step) {
                        const bool more = step + 1 < g.step1;
                        const int v_stage = stage;
                        const uint32_t v_phase = phase;
                        advance(stage, phase);
                        auto release_k = [&]() {
                            mma_commit_warp(smem_u32(&kv_empty[stage]));
                            advance(stage, phase);
                            if (step + 2 == g.step1) mma_commit_warp(smem_u32(q_empty));
                        };
                        if (C::kEarly && more) {  // the next scores, once the softmax has these
                            if (!wait(&kv_full[stage], phase)) break;
                            for (int t = t0; t < t1 && ok; ++t) {
                                if (!wait(&s_empty[t], (se_phase >> t) & 1)) break;
                                se_phase ^= 1u << t;
                                tc_fence_after();
                                issue_s(t, stage);
                            }
                            if (!ok) break;
                            release_k();
                        }
                        if (!wait(&kv_full[v_stage], v_phase)) break;
                        // keys past the last that the item sees: their slots may hold anything (or were not
                        // loaded), and 0 * NaN is NaN: the first warp zeroes the rows
                        const int live = keys - step * kKeys;
                        if (live < kKeys && t0 == 0) {
                            const int from = max(live, 0);
                            const uint32_t vb = smem_u32(smem + (2 + v_stage) * C::kTile);
                            for (int i = from * 8 + lane; i < kKeys * 8; i += 32)
#pragma unroll
                                for (int d = 0; d < kSlabs; ++d)
                                    sts_v4(vb + d * kKeys * 128 + i * 16, make_uint4(0, 0, 0, 0));
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (C::kMmaWarps == 2 && lane == 0) mbar_arrive(smem_u32(&v_zero[v_stage]));
                        } else if (live < kKeys) {
                            if (!wait(&v_zero[v_stage], z_phase >> v_stage & 1)) break;
                            z_phase ^= 1u << v_stage;
                        }
                        for (int t = t0; t < t1 && ok; ++t) {
                            if (step == g.step0) {  // O was read out by the previous segment's epilogue
                                if (!wait(&o_empty[t], (oe_phase >> t) & 1)) break;
                                oe_phase ^= 1u << t;
                            }
                            if (!wait(&p_full[t], (p_phase >> t) & 1)) break;
                            p_phase ^= 1u << t;
                            tc_fence_after();
                            const uint64_t vb = v_desc(smem_u32(smem + (2 + v_stage) * C::kTile));
                            mma_o(tmem + C::col_o(t), tmem + C::col_p(t), vb, id_o, step > g.step0);
                            if (C::kEarly || !more) mma_commit_warp(smem_u32(&o_full[t]));
                            if (C::kEarly && !more) se_phase ^= 1u << t;  // the segment's last scores: past, with its P
                            if (!C::kEarly && more) {
                                if (t == 0 && !wait(&kv_full[stage], phase)) break;
                                issue_s(t, stage);
                            }
                        }
                        if (!ok) break;
                        mma_commit_warp(smem_u32(&kv_empty[v_stage]));
                        if (!C::kEarly && more) release_k();
                    }
                }
            }
            // the segment list is free; a role that gave up ends the CTA
            ok = !meet_any(!ok);
        }
        // an aborting CTA waits for its own copies and MMAs before it gives up its memory
        if (warp == kLoadWarp && !ok) {
            for (int i = 0; i < C::kStages; ++i) {
                // the last fill of stage i was in the current phase if i < stage, else in the one before
                const uint32_t par = i < stage ? phase : phase ^ 1;
                if (ring_waited >> i & 1) mbar_wait_drain(smem_u32(&kv_full[i]), par, wt);
            }
            mbar_wait_drain(smem_u32(q_full), q_phase ^ 1, wt);
        }
        if (warp == kMmaWarp || warp == kMma1Warp) {  // every MMA and every arrival of its commits is over before the CTA ends
            const uint32_t bar = smem_u32(&drain[warp == kMmaWarp ? 0 : 1]);
            mma_commit_warp(bar);
            mbar_wait_drain(bar, 0, wt);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        uint32_t s_phase = 0, o_phase = 0;
        for (uint32_t u = u_begin; u < u_end && ok;) {
            meet();
            const int ns = *nseg;
            u = cursor[3];
            // ------------------------------------------------ softmax and epilogue, one row a thread
            const int t = warp >> 2, r = tid & (kM - 1);
            const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's TMEM lanes
            const uint32_t ts = tmem + lanes + t * kKeys, tp = tmem + lanes + C::col_p(t), to = tmem + lanes + C::col_o(t);
            const bool neg = a.scale < 0.f;
            // a zero scale would make -inf * 0 of masked scores: the smallest normal factor moves no score by more
            // than 4, and only scores past 10^37 by more than 0.1
            const float sl2 = fmaxf(fabsf(a.scale) * kLog2e, 1.17549435e-38f);
            for (int k = 0; k < ns && ok; ++k) {
                const Seg g = segs[k];
                if (t >= g.tiles) continue;
                const int j = g.tok0 + t * int(tt) + r / int(G);  // this row's token in the chunk
                const bool live = r < int(G * tt) && j < g.q_len;
                const int past = g.kv_len - g.q_len;
                const int seen = live ? max(past + j + 1, 0) : 0;
                const int seen_all = past + g.tok0 + t * int(tt) + 1;  // keys that every row of the tile sees
                float m = kNegInf, l = 0.f;
                for (int step = g.step0; step < g.step1; ++step) {
                    ok = mbar_wait(smem_u32(&s_full[t]), s_phase, wt);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    s_phase ^= 1;
                    tc_fence_after();
                    uint32_t x[128];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld32_issue(ts + i * 32, x + i * 32);
                    tmem_ld_done(x);
                    if (C::kEarly) {
                        tc_fence_before();
                        mbar_arrive(smem_u32(&s_empty[t]));
                    }
                    if (neg) {
#pragma unroll
                        for (int i = 0; i < 128; ++i) x[i] ^= 0x80000000u;
                    }
                    const int k0 = step * kKeys;
                    if (k0 > seen_all - kKeys) {
#pragma unroll
                        for (int i = 0; i < 128; ++i)
                            if (k0 + i >= seen) x[i] = 0xff800000u;
                    }
                    float mx[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 4]));
#pragma unroll
                    for (int i = 8; i < 128; i += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx[e] = max3(mx[e], __uint_as_float(x[i + e]), __uint_as_float(x[i + e + 4]));
                    const float mn = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), m);
                    if (C::kEarly && step > g.step0) {  // the step before is added to O, its P is free
                        ok = mbar_wait(smem_u32(&o_full[t]), o_phase, wt);
                        if (!__all_sync(0xffffffffu, ok)) {
                            ok = false;
                            break;
                        }
                        o_phase ^= 1;
                        tc_fence_after();
                    }
                    if (step == g.step0) {
                        m = mn;
                    } else if (__any_sync(0xffffffffu, live && (mn - m) * sl2 > kLag)) {
                        // -inf - -inf is NaN and compares false: a row that has seen nothing stays.  Rows past the
                        // tile's hold what lay in shared memory, and decide nothing: results keep their bits.
                        const float f = mn == kNegInf ? 1.f : ex2((m - mn) * sl2);
                        m = mn;
                        l *= f;
#pragma unroll
                        for (int i = 0; i < D; i += 16) {
                            float o[16];
                            uint32_t w[16];
                            tmem_ld16(to + i, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
                            tmem_st16(to + i, w);
                        }
                    }
                    const float z = m == kNegInf ? 0.f : m * sl2;
                    const uint64_t sl2p = pair(sl2, sl2), zp = pair(-z, -z);
                    // probabilities in bf16 for the product (up to 2^-8 of each; error of the 2048-token chunk against 64 bits
                    // 0.0023 of the outputs' size, with fp32 probabilities 0.0017); their sum stays in fp32
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < 128; i += 2) {
                        float p0, p1;
                        unpair(fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), sl2p, zp), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pair(p0, p1));
                        x[i / 2] = pack_bf16(p0, p1);
                        if (i == 62) tmem_st32(tp, x);
                    }
                    tmem_st32(tp + 32, x + 32);
                    float s0, s1;
                    unpair(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(smem_u32(&p_full[t]));
                }
                if (!ok) break;
                ok = mbar_wait(smem_u32(&o_full[t]), o_phase, wt);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                o_phase ^= 1;
                tc_fence_after();
                const int64_t tok = g.q0 + j;
                const int head = g.h * int(G) + r % int(G);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const size_t prow = (size_t)max(g.slot, 0) * 2 * kM + t * kM + r;
                uint16_t *dst = static_cast<uint16_t *>(a.out) + tok * a.out_stride + (int64_t)head * D;
#pragma unroll
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    tmem_ld32(to + i, o);
                    if (g.slot >= 0) {
                        if (live) {
                            uint4 *to = reinterpret_cast<uint4 *>(c.part_o) + ((size_t)g.slot * (D / 4) + i / 4) * 2 * kM + t * kM + r;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                to[e * 2 * kM] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float v[8];
#pragma unroll
                            for (int q = 0; q < 8; ++q) v[q] = __uint_as_float(o[e + q]) * inv;
                            store8(dst + i + e, v);
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(smem_u32(&o_empty[t]));
                if (live) {
                    if (g.slot >= 0)
                        c.part_ml[prow] = make_float2(m == kNegInf ? kNegInf : m * sl2, l);
                    else if (a.lse)
                        a.lse[tok * a.n_heads + head] = l == 0.f ? kNegInf : (m * sl2 + log2f(l)) * kLn2;
                }
            }
            ok = !meet_any(!ok);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// Joins the parts of the items that were cut.  Block (cta, y): the item that starts in the share of
// `cta` and goes on, rows [16 y, 16 y + 16) of its 256; 16 threads a row.  Four parts are requested
// together, their maxima and sums with their outputs (one warp a row, part by part, took 19 us
// for a mixed batch's 150 cut items).
constexpr int kJoinThreads = kJoinRows * 16;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const __grid_constant__ Ctx c) {
    griddep_wait();
    griddep_launch_dependents();
    const Args &a = c.a;
    const int *rp = reinterpret_cast<const int *>(c.rec + blockIdx.x);
    const int n = ldp(rp), h = ldp(rp + 1), tok0 = ldp(rp + 2), q0 = ldp(rp + 3), q_len = ldp(rp + 4);
    if (n == 0) return;
    const int G = a.group, row = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows, t = row / kM, r = row % kM;
    const int rt = r / G, j = tok0 + t * int(c.tt) + rt;
    if (r >= G * int(c.tt) || j >= q_len) return;
    constexpr int kFly = 4, E = D / 64;  // float4 pieces of a thread: neighbours
    const int d0 = threadIdx.x / kJoinRows * (4 * E);
    float m = kNegInf, l = 0.f;
    float4 acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < n; p0 += kFly) {
        float pm[kFly], pl[kFly];
        float4 v[kFly][E];
#pragma unroll
        for (int p = 0; p < kFly; ++p) {
            const int i = min(p0 + p, n - 1);
            const size_t slot = (size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0);
            asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(pm[p]), "=f"(pl[p]) : "l"(c.part_ml + slot * 2 * kM + row));
#pragma unroll
            for (int e = 0; e < E; ++e)
                v[p][e] = ldp16f(c.part_o + ((slot * (D / 4) + d0 / 4 + e) * 2 * kM + row) * 4);
        }
        float mn = m;
#pragma unroll
        for (int p = 0; p < kFly; ++p) mn = fmaxf(mn, pm[p]);
        const float f0 = m == kNegInf ? 0.f : ex2(m - mn);
        m = mn;
        l *= f0;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = make_float4(acc[e].x * f0, acc[e].y * f0, acc[e].z * f0, acc[e].w * f0);
#pragma unroll
        for (int p = 0; p < kFly; ++p) {
            if (p0 + p >= n || pl[p] == 0.f) continue;  // read again past the last, or no key seen; a NaN sum stays
            const float f = ex2(pm[p] - mn);
            l = fmaf(f, pl[p], l);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                acc[e].x = fmaf(f, v[p][e].x, acc[e].x);
                acc[e].y = fmaf(f, v[p][e].y, acc[e].y);
                acc[e].z = fmaf(f, v[p][e].z, acc[e].z);
                acc[e].w = fmaf(f, v[p][e].w, acc[e].w);
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t tok = q0 + j;
    const int head = h * G + (r - rt * G);
    uint16_t *dst = static_cast<uint16_t *>(a.out) + tok * a.out_stride + (int64_t)head * D + d0;
#pragma unroll
    for (int e = 0; e < E; ++e)
        *reinterpret_cast<uint2 *>(dst + e * 4) =
            make_uint2(pack_bf16(acc[e].x * inv, acc[e].y * inv), pack_bf16(acc[e].z * inv, acc[e].w * inv));
    if (a.lse && d0 == 0) a.lse[tok * a.n_heads + head] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
}

int64_t max_items(const moe_attn_shape &s) {
    const int64_t tt2 = 2 * (kM / (s.n_heads / s.n_kv_heads));
    return ((s.n_tokens + tt2 - 1) / tt2 + s.n_seqs) * s.n_kv_heads;
}
// The longest that the line of all steps can be.
double max_places(const moe_attn_shape &s) {
    return double(max_items(s)) * ((double)s.max_pages * s.page_size / kKeys + 1 + kSetup);
}
bool not_cut(const moe_attn_shape &s) { return (int64_t)s.max_pages * s.page_size <= kWholeKeys; }
int max_ctas(const moe_attn_shape &s) {
    const double n = not_cut(s) ? double(max_items(s)) : max_places(s) / (kSetup + 2);
    return n < 1 ? 1 : n < kMaxCtas ? int(n) : kMaxCtas;
}
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <int D>
bool set_smem_attr() {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        if (cudaFuncSetAttribute(chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem) != cudaSuccess)
            return false;
        // the softmax's registers come from the launch's: fewer, and the kernel would wait for them for ever
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, chunk_kernel<D>) != cudaSuccess || fa.numRegs < kLaunchRegs) return false;
        attr_set[dev] = true;
    }
    return true;
}

template <int D>
cudaError_t launch_typed(const Ctx &c, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, int grid,
                         cudaStream_t st) {
    if (!set_smem_attr<D>()) return cudaErrorInvalidValue;
    const cudaError_t e = launch_pdl(chunk_kernel<D>, dim3(grid), dim3(kThreads), Cfg<D>::kSmem, st, mq, mk, mv, c);
    if (e != cudaSuccess || c.whole) return e;
    return launch_pdl(chunk_join_kernel<D>, dim3(grid, 2 * kM / kJoinRows), dim3(kJoinThreads), 0, st, c);
}

}  // namespace

// bf16, head sizes 64 and 128, a group that fits a tile, pages that fill key steps (or that key
// steps fill), and a line of steps that 32 bits count.
bool chunk_supported(const moe_attn_shape &s) {
    const int G = s.n_heads / s.n_kv_heads;
    const bool pages = s.page_size >= 8 && (kKeys % s.page_size == 0 || s.page_size % kKeys == 0);
    return s.dtype == MOE_DT_BF16 && (s.head_dim == 64 || s.head_dim == 128) && G <= kM && pages &&
           max_places(s) < 2147483648.0;
}

size_t chunk_ws_bytes(const moe_attn_shape &s) {
    const size_t slots = 2 * (size_t)max_ctas(s);
    return round256(kMaxCtas * sizeof(Rec)) + round256(slots * 2 * kM * sizeof(float2)) + slots * 2 * kM * s.head_dim * 4;
}

cudaError_t launch_chunk(const Args &a, const moe_attn_shape &s, char *ws, int sms, cudaStream_t st) {
    Ctx c{};
    c.a = a;
    c.tt = uint32_t(kM / a.group);
    c.item_shift = -1;
    if ((c.tt & (c.tt - 1)) == 0)
        for (c.item_shift = 0; (1u << c.item_shift) < 2 * c.tt;) ++c.item_shift;
    const int cap = max_ctas(s), grid = sms < cap ? sms : cap;
    c.rec = reinterpret_cast<Rec *>(ws);
    c.part_ml = reinterpret_cast<float2 *>(ws + round256(kMaxCtas * sizeof(Rec)));
    c.part_o = reinterpret_cast<float *>(reinterpret_cast<char *>(c.part_ml) + round256((size_t)2 * cap * 2 * kM * sizeof(float2)));
    c.wait_ns = wait_limit_ns();
    c.extra_need = debug_extra_need();
    c.whole = not_cut(s);
    const uint64_t D = s.head_dim;
    CUtensorMap mq, mk, mv;
    const uint64_t qd[3] = {D, (uint64_t)s.n_heads, (uint64_t)s.n_tokens}, qs[2] = {D * 2, (uint64_t)a.q_stride * 2};
    const uint32_t qb[3] = {64, (uint32_t)a.group, c.tt};
    // a dimension of one element is never stepped over: any legal stride stands in for its own
    const uint64_t row = D * 2;
    const uint64_t kd[4] = {D, (uint64_t)s.page_size, (uint64_t)s.n_kv_heads, (uint64_t)s.n_pages};
    const uint64_t ks[3] = {(uint64_t)a.token_stride * 2, s.n_kv_heads > 1 ? (uint64_t)a.head_stride * 2 : row,
                            s.n_pages > 1 ? (uint64_t)a.page_stride * 2 : row};
    const uint32_t kb[4] = {64, (uint32_t)(s.page_size < kKeys ? s.page_size : kKeys), 1, 1};
    if (!make_map_nd(&mq, a.q, 3, qd, qs, qb) || !make_map_nd(&mk, a.k, 4, kd, ks, kb) || !make_map_nd(&mv, a.v, 4, kd, ks, kb))
        return cudaErrorInvalidValue;
    return D == 128 ? launch_typed<128>(c, mq, mk, mv, grid, st) : launch_typed<64>(c, mq, mk, mv, grid, st);
}

}  // namespace attn
}  // namespace moe
