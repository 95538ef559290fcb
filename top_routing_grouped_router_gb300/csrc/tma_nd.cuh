// tma_nd.cuh -- tensor maps and loads of up to four dimensions, for tensors with strides of
// their own (the paged cache, slices of a projection's output).
#pragma once

#include "tc_common.cuh"

namespace moe {
namespace tc {

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// bf16 map of rank 2 to 4 with any strides (bytes, multiples of 16, of dimensions 1 ..), 128-byte
// swizzle: box[0] is 64 elements.
bool make_map_nd(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                 const uint32_t *box);
// The same of bytes, not swizzled: box[0] is a multiple of 16.
bool make_map_bytes(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                    const uint32_t *box);

}  // namespace tc
}  // namespace moe
