// attn_decode.cu -- attention of a few new tokens a sequence over all keys of a bf16 cache, what the
// decode kernels support, and their workspace.
#include "attn_decode.cuh"

namespace moe {
namespace attn {

// bf16, head sizes 64 and 128, at most 16 query rows a key head, and a line of steps that
// 32 bits count even if every sequence fills its row of the block table.
bool decode_supported(const moe_attn_shape &s) {
    const double steps = double(s.n_seqs) * s.n_kv_heads * ((double)s.max_pages * s.page_size / kStep + 1);
    return s.dtype == MOE_DT_BF16 && (s.head_dim == 64 || s.head_dim == 128) &&
           (int64_t)s.max_q * (s.n_heads / s.n_kv_heads) <= kRows && steps < 2147483648.0;
}
// Over an 8-bit cache a step also lies within a page and within a block of one scale.
bool decode_q8_supported(const moe_attn_shape &s, int block) { return decode_supported(s) && block % kStep == 0; }

size_t decode_ws_bytes(const moe_attn_shape &s) { return (size_t)kMaxGrid * 2 * kRows * (s.head_dim + 2) * 4; }

cudaError_t launch_decode(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int sms, Mode mode, cudaStream_t st) {
    if (mode == kAll) return launch<kAll>(a, s, hdr, ws, sms, st);
    return mode == kWindow ? launch_decode_window(a, s, hdr, ws, sms, st) : launch_decode_q8(a, s, hdr, ws, sms, st);
}

}  // namespace attn
}  // namespace moe
