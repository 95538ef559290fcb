// attn_api.cu -- the extern "C" entry points of the attention half of a decoder layer:
// host-side validation, workspace sizes and the choice of kernel.
#include "attn.cuh"
#include "q4_linear.cuh"
#include "tc_common.cuh"

#include <cmath>

using namespace moe;

namespace {

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
int launch_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

int validate(const moe_attn_shape *s) {
    if (!s) return MOE_ERR_NULLPTR;
    if (s->n_tokens < 0 || s->n_tokens > (1 << 20) || s->n_seqs < 0 || s->n_seqs > (1 << 16)) return MOE_ERR_SHAPE;
    if (s->n_tokens > 0 && s->n_seqs == 0) return MOE_ERR_SHAPE;
    if (s->n_heads <= 0 || s->n_heads > 1024 || s->n_kv_heads <= 0 || s->n_heads % s->n_kv_heads) return MOE_ERR_SHAPE;
    if (s->head_dim <= 0 || s->head_dim > 256 || s->head_dim % 8) return MOE_ERR_SHAPE;
    if (s->page_size <= 0 || s->n_pages <= 0 || s->max_pages <= 0) return MOE_ERR_SHAPE;
    if ((int64_t)s->max_pages * s->page_size > INT32_MAX) return MOE_ERR_SHAPE;
    if (s->max_q < 0 || s->max_q > s->n_tokens) return MOE_ERR_SHAPE;
    if (s->dtype != MOE_DT_F32 && s->dtype != MOE_DT_BF16) return MOE_ERR_DTYPE;
    return MOE_OK;
}

int64_t elem_bytes(const moe_attn_shape &s) { return s.dtype == MOE_DT_F32 ? 4 : 2; }

// A row stride in elements: a multiple of 16 bytes that does not overlap rows.
int check_stride(const moe_attn_shape &s, int64_t stride, int heads) {
    if (stride < (int64_t)heads * s.head_dim || stride > INT32_MAX) return MOE_ERR_SHAPE;
    return (stride * elem_bytes(s)) % 16 ? MOE_ERR_ALIGN : MOE_OK;
}

int check_cache(const moe_attn_shape &s, const moe_kv_cache *c) {
    if (!c || !c->k || !c->v) return MOE_ERR_NULLPTR;
    const int64_t st[3] = {c->page_stride, c->head_stride, c->token_stride};
    for (int64_t x : st)
        if (x < 0 || x > (int64_t(1) << 40)) return MOE_ERR_SHAPE;
    // two slots or two heads of a page must not share elements (a size-1 dimension's stride is free)
    if ((s.page_size > 1 && c->token_stride < s.head_dim) || (s.n_kv_heads > 1 && c->head_stride < s.head_dim))
        return MOE_ERR_SHAPE;
    for (int64_t x : st)
        if ((x * elem_bytes(s)) % 16) return MOE_ERR_ALIGN;
    return misaligned(c->k) || misaligned(c->v) ? MOE_ERR_ALIGN : MOE_OK;
}

int check_batch(const moe_attn_batch *b) {
    if (!b || !b->cu_q || !b->kv_len || !b->block_table) return MOE_ERR_NULLPTR;
    return misaligned4(b->cu_q) || misaligned4(b->kv_len) || misaligned4(b->block_table) ? MOE_ERR_ALIGN : MOE_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need) {
    if (!ws || bytes < need) return MOE_ERR_WORKSPACE;
    return (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) ? MOE_ERR_ALIGN : MOE_OK;
}

attn::Args make_args(const moe_attn_shape &s, const moe_kv_cache &c, const moe_attn_batch &b, const void *q,
                     int64_t q_stride, void *out, int64_t out_stride, void *ws) {
    attn::Args a{};
    a.cu_q = b.cu_q;
    a.kv_len = b.kv_len;
    a.table = b.block_table;
    a.k = c.k;
    a.v = c.v;
    a.page_stride = c.page_stride;
    a.head_stride = c.head_stride;
    a.token_stride = c.token_stride;
    a.n_tokens = s.n_tokens;
    a.n_seqs = s.n_seqs;
    a.n_heads = s.n_heads;
    a.n_kv_heads = s.n_kv_heads;
    a.head_dim = s.head_dim;
    a.group = s.n_heads / s.n_kv_heads;
    a.page_size = s.page_size;
    a.n_pages = s.n_pages;
    a.max_pages = s.max_pages;
    a.max_q = s.max_q;
    a.page_shift = -1;
    if ((s.page_size & (s.page_size - 1)) == 0)
        for (a.page_shift = 0; (1 << a.page_shift) < s.page_size;) ++a.page_shift;
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.err = static_cast<int32_t *>(ws);
    return a;
}

}  // namespace

#define MOE_TRY(expr)                  \
    do {                               \
        const int _rc = (expr);        \
        if (_rc != MOE_OK) return _rc; \
    } while (0)

extern "C" {

int moe_attn_workspace_size(const moe_attn_shape *shape, size_t *bytes) {
    if (!bytes) return MOE_ERR_NULLPTR;
    MOE_TRY(validate(shape));
    *bytes = kHdrBytes + (attn::decode_supported(*shape)  ? attn::decode_ws_bytes(*shape)
                          : attn::chunk_supported(*shape) ? attn::chunk_ws_bytes(*shape)
                                                          : attn::generic_ws_bytes(*shape));
    return MOE_OK;
}

int moe_rope_turns(int32_t rot_dim, int32_t scaling, double base, double factor, int32_t trained_len, uint64_t *turns,
                   float *mscale) {
    if (!turns || !mscale) return MOE_ERR_NULLPTR;
    if (rot_dim <= 0 || rot_dim > 256 || rot_dim % 16) return MOE_ERR_SHAPE;
    if (scaling < MOE_ROPE_NONE || scaling > MOE_ROPE_YARN) return MOE_ERR_SHAPE;
    if (!(base > 1.0) || !(base < 1e30)) return MOE_ERR_SHAPE;
    if (scaling != MOE_ROPE_NONE && (!(factor >= 1.0) || !(factor < 1e9))) return MOE_ERR_SHAPE;
    if (scaling == MOE_ROPE_YARN && trained_len <= 0) return MOE_ERR_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    const double r = rot_dim;
    if (scaling == MOE_ROPE_NTK) base *= std::pow(factor, r / (r - 2.0));
    double low = 0.0, high = 0.0;
    *mscale = 1.0f;
    if (scaling == MOE_ROPE_YARN) {
        // the (fractional) pair whose rate makes n turns within trained_len positions
        auto pair_of = [&](double n) { return r * std::log(trained_len / (n * two_pi)) / (2.0 * std::log(base)); };
        low = std::fmax(std::floor(pair_of(32.0)), 0.0);
        high = std::fmin(std::ceil(pair_of(1.0)), r - 1.0);
        *mscale = float(0.1 * std::log(factor) + 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / r);
        if (scaling == MOE_ROPE_LINEAR) f /= factor;
        if (scaling == MOE_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        turns[i] = uint64_t(f / two_pi * 18446744073709551616.0 + 0.5);  // f <= 1: below 2^62
    }
    return MOE_OK;
}

int moe_rope_append(const moe_attn_shape *shape, const moe_rope *rope, const void *q, int64_t q_stride, const void *k,
                    int64_t k_stride, const void *v, int64_t v_stride, const moe_kv_cache *cache,
                    const moe_attn_batch *batch, const int32_t *positions, void *q_out, int64_t q_out_stride,
                    void *workspace, size_t workspace_bytes, moe_stream_t stream) {
    MOE_TRY(validate(shape));
    const moe_attn_shape &s = *shape;
    if (!rope) return MOE_ERR_NULLPTR;
    if (rope->rot_dim <= 0 || rope->rot_dim > s.head_dim || rope->rot_dim % 16) return MOE_ERR_SHAPE;
    if (!std::isfinite(rope->mscale)) return MOE_ERR_SHAPE;
    if ((rope->q_gamma || rope->k_gamma) && (!(rope->eps >= 0.f) || !std::isfinite(rope->eps))) return MOE_ERR_SHAPE;
    if (s.n_tokens == 0) return MOE_OK;
    if (!rope->turns || !q || !k || !v || !q_out) return MOE_ERR_NULLPTR;
    MOE_TRY(check_cache(s, cache));
    MOE_TRY(check_batch(batch));
    MOE_TRY(check_stride(s, q_stride, s.n_heads));
    MOE_TRY(check_stride(s, q_out_stride, s.n_heads));
    MOE_TRY(check_stride(s, k_stride, s.n_kv_heads));
    MOE_TRY(check_stride(s, v_stride, s.n_kv_heads));
    MOE_TRY(check_workspace(workspace, workspace_bytes, kHdrBytes));
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(q_out) || misaligned(rope->turns) ||
        misaligned(rope->q_gamma) || misaligned(rope->k_gamma) || misaligned4(positions))
        return MOE_ERR_ALIGN;
    const attn::Args a = make_args(s, *cache, *batch, q, q_stride, q_out, q_out_stride, workspace);
    return launch_rc(launch_rope(s, *rope, a, k, k_stride, v, v_stride, positions,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

int moe_paged_attention(const moe_attn_shape *shape, const void *q, int64_t q_stride, const moe_kv_cache *cache,
                        const moe_attn_batch *batch, float scale, void *out, int64_t out_stride, float *lse,
                        void *workspace, size_t workspace_bytes, moe_stream_t stream) {
    MOE_TRY(validate(shape));
    const moe_attn_shape &s = *shape;
    if (!std::isfinite(scale)) return MOE_ERR_SHAPE;
    if (s.n_tokens == 0) return MOE_OK;
    if (!q || !out) return MOE_ERR_NULLPTR;
    MOE_TRY(check_cache(s, cache));
    MOE_TRY(check_batch(batch));
    MOE_TRY(check_stride(s, q_stride, s.n_heads));
    MOE_TRY(check_stride(s, out_stride, s.n_heads));
    size_t need = 0;
    MOE_TRY(moe_attn_workspace_size(shape, &need));
    MOE_TRY(check_workspace(workspace, workspace_bytes, need));
    if (misaligned(q) || misaligned(out) || misaligned4(lse)) return MOE_ERR_ALIGN;
    attn::Args a = make_args(s, *cache, *batch, q, q_stride, out, out_stride, workspace);
    a.lse = lse;
    a.scale = scale;
    char *hdr = static_cast<char *>(workspace), *ws = hdr + kHdrBytes;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (attn::decode_supported(s)) return launch_rc(attn::launch_decode(a, s, hdr, ws, tc::sm_count(), st));
    if (attn::chunk_supported(s)) return launch_rc(attn::launch_chunk(a, s, ws, tc::sm_count(), st));
    return launch_rc(attn::launch_generic(a, s.dtype, s, ws, st));
}

int moe_q4_linear(const moe_q4_linear_shape *shape, const void *x, int64_t x_stride, const moe_q4_weight *weight,
                  const void *residual, int64_t residual_stride, void *out, int64_t out_stride, moe_stream_t stream) {
    if (!shape) return MOE_ERR_NULLPTR;
    const moe_q4_linear_shape &s = *shape;
    if (s.T < 0 || s.T > (1 << 18) || s.K <= 0 || s.K % 8 || s.K > (1 << 22) || s.N <= 0 || s.N > (1 << 22))
        return MOE_ERR_SHAPE;
    if (s.q_block <= 0 || s.q_block % 2 || s.K % s.q_block) return MOE_ERR_SHAPE;
    if (s.out_dtype != MOE_DT_BF16 && s.out_dtype != MOE_DT_F32) return MOE_ERR_DTYPE;
    if (s.T == 0) return MOE_OK;
    if (!x || !out || !weight || !weight->codes || !weight->scales) return MOE_ERR_NULLPTR;
    if (x_stride < s.K || out_stride < s.N || (residual && residual_stride < s.N)) return MOE_ERR_SHAPE;
    if (x_stride % 8 || misaligned(x) || misaligned(out) || misaligned(weight->codes) || misaligned(weight->scales) ||
        misaligned(residual))
        return MOE_ERR_ALIGN;
    return launch_rc(launch_q4_linear(s, x, x_stride, *weight, residual, residual_stride, out, out_stride, tc::sm_count(),
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int moe_q4_linear_read_error(int32_t *code, moe_stream_t stream) {
    if (!code) return MOE_ERR_NULLPTR;
    return launch_rc(q4::read_error(code, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
