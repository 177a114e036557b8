// tma_warp.cuh -- a 4-D TMA tile load (of whole rows of the other dimensions) and the announcement of its bytes, issued by one
// lane of a converged warp: the operands are the same in every lane, and as the compiler sees that, they go straight to
// the uniform registers that the instruction takes.
#pragma once

#include "tcgen05.cuh"

namespace sffn {
namespace tc {

SFFN_DEV void tma_load_rows_warp(uint32_t dst, const CUtensorMap *map, int u, uint32_t bar, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %2, %2, %3}], [%4], %5;\n\t}\n" ::"r"(dst),
        "l"(map), "r"(0), "r"(u), "r"(bar), "l"(policy)
        : "memory");
}
SFFN_DEV void mbar_expect_tx_warp(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}\n" ::"r"(bar),
        "r"(bytes)
        : "memory");
}

}  // namespace tc
}  // namespace sffn
