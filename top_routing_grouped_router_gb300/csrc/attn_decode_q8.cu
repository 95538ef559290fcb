// attn_decode_q8.cu -- attention of a few new tokens a sequence over an 8-bit cache.
#include "attn_decode.cuh"

namespace moe {
namespace attn {

cudaError_t launch_decode_q8(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int sms, cudaStream_t st) {
    if ((int64_t)s.max_q * a.group <= 8) return launch_decode_q8_half(a, s, hdr, ws, sms, st);
    return launch<kQ8>(a, s, hdr, ws, sms, st);
}

}  // namespace attn
}  // namespace moe
