// attn_decode_q8_half.cu -- the same of up to 8 query rows a key head.
#include "attn_decode.cuh"

namespace moe {
namespace attn {

cudaError_t launch_decode_q8_half(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int sms, cudaStream_t st) {
    return launch<kQ8, true>(a, s, hdr, ws, sms, st);
}

}  // namespace attn
}  // namespace moe
