// Tensor copies into shared memory and what they are counted with, issued by a
// converged warp (the attention kernels').
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace kda {
namespace attn {

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// Tensor copies issued by a converged warp, of which the lane with `lead` set takes
// part: its operands stay in uniform registers (a copy issued by a lane of its own
// choice cost 100 cycles, which at 16-row pages bounded the loads).
__device__ __forceinline__ void tma_2d(uint32_t lead, uint32_t dst, const CUtensorMap *m, int c0, int c1, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n"
        " @q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
        "l"(m), "r"(c0), "r"(c1), "r"(bar), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t lead, uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %6, 0;\n"
        " @q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
        "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t lead, uint32_t bar, uint32_t bytes) {
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}\n" ::"r"(bar),
                 "r"(bytes), "r"(lead)
                 : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(m) : "memory");
}

}  // namespace attn
}  // namespace kda
