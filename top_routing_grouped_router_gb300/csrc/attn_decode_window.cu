// attn_decode_window.cu -- attention of a few new tokens a sequence with a window over a bf16 cache.
#include "attn_decode.cuh"

namespace moe {
namespace attn {

cudaError_t launch_decode_window(const Args &a, const moe_attn_shape &s, char *hdr, char *ws, int sms, cudaStream_t st) {
    return launch<kWindow>(a, s, hdr, ws, sms, st);
}

}  // namespace attn
}  // namespace moe
