// q4_linear.cu -- out = x . W^T (+ residual) with 4-bit weights (codes, one bf16 scale per
// q_block inputs, a 16-entry codebook), for batches of few rows.
#include "attn.cuh"

namespace moe {
namespace {

struct Q4Args {
    const uint16_t *x;
    const uint8_t *codes;
    const uint16_t *scales;
    const uint16_t *res;
    void *out;
    int64_t x_stride, res_stride, out_stride;
    int T, K, N, q_block;
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

}  // namespace

cudaError_t launch_q4_linear(const moe_q4_linear_shape &s, const void *x, int64_t x_stride, const moe_q4_weight &w,
                             const void *res, int64_t res_stride, void *out, int64_t out_stride, cudaStream_t st) {
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
    for (int i = 0; i < 16; ++i) a.codebook[i] = w.codebook[i];
    return launch_any(a, s.out_dtype, st);
}

}  // namespace moe
