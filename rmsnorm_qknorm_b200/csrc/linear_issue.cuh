// TMA loads, MMAs and commits of the fused linear layer, issued by a whole
// warp of which one elected lane acts.
//
// Descriptors, coordinates and barrier addresses of these instructions live in
// uniform registers.  In a loop that a single lane runs the compiler has to
// move each of them there for every instruction; run by the whole warp, with
// the election inside the instruction, the loop stays uniform and they are
// there already.  (One token, 512 x 16384, K over eight CTAs: a block of 64 k
// took 0.29 us in a one-lane loop whatever the tile's size.)  elect.sync
// chooses the same lane every time, so commits follow the MMAs they track.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "qkn_sync.cuh"

namespace qkn {
namespace lin {

__device__ __forceinline__ void elect_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .pred e;\n\t.reg .b64 st;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}"
                 ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void elect_tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];\n\t}"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}

// The CTA-pair form: into this CTA's shared memory, completing on the barrier at the
// shared::cluster address `bar` (the even CTA's).
__device__ __forceinline__ void elect_tma_load_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];\n\t}"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}

// One MMA of CTA group GROUP (1, or 2 for a pair) with the instruction descriptor DESC.
template <int GROUP, uint32_t DESC>
__device__ __forceinline__ void elect_umma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
    if constexpr (GROUP == 1)
        asm volatile("{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(DESC), "r"(accumulate));
    else
        asm volatile("{\n\t.reg .pred e, p;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(DESC), "r"(accumulate));
}

// Arrives on the barrier (shared::cluster address) once the MMAs issued so far have completed.
template <int GROUP> __device__ __forceinline__ void elect_commit(uint32_t bar) {
    if constexpr (GROUP == 1)
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                     ::"r"(bar) : "memory");
    else
        asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                     "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                     ::"r"(bar) : "memory");
}

// mbar_wait by a whole warp: the same answer on every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int *err, uint64_t timeout_ns = kWaitTimeoutNs) {
    return __all_sync(0xffffffffu, mbar_wait_fast(bar, parity, err, timeout_ns));
}

// The limit of a wait for a whole product of k_blocks blocks of 64 k (at most 0.5 us each; 2^31 k
// alone pass the usual limit).
__device__ __forceinline__ uint64_t product_timeout(int k_blocks) { return kWaitTimeoutNs + 4000ull * (uint64_t)k_blocks; }

}  // namespace lin
}  // namespace qkn
