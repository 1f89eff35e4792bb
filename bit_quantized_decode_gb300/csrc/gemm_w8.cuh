// Waits, copies and conversions shared by the tensor-core products of INT8
// weights (gemm_w8.cu, gemm_w8_pair.cu).
#pragma once
#include <cuda_fp16.h>

#include "operators.h"
#include "ptx.cuh"
#include "typed_io.cuh"

namespace w4k {

constexpr uint64_t kG8WaitNs = 250ull * 1000ull * 1000ull;

// Wait of a whole warp: a test first, as the phase is usually complete.  The
// lanes vote on every try and leave together: what follows are .aligned
// tensor-memory instructions, which a warp whose lanes come one after another
// (each out of a loop of its own) must not reach.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity)
{
    bool ok = __all_sync(0xffffffffu, mbar_test_wait(bar, parity));
    if (!ok) {
        uint64_t t0 = 0;
#pragma unroll 1
        for (uint32_t i = 1; !ok; ++i) {
            ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
            if (!ok && (i & 31u) == 0u) {          // the timer is slow to read
                const uint64_t now = globaltimer_ns();
                if (i == 32u) t0 = now;
                else if (__any_sync(0xffffffffu, now - t0 > kG8WaitNs)) break;
            }
        }
    }
    __syncwarp();
    return ok;
}

// Box of a 2-D tensor map -> shared memory.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
        "%3}], [%4], %5;" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar), "l"(pol)
        : "memory");
}

// L2 policy for the activation codes, which every row group reads again.
__device__ __forceinline__ uint64_t l2_policy_evict_last()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// 32 int8 weights of a row as 16 words of fp16 pairs.
__device__ __forceinline__ void unit_f16(const uint4& lo, const uint4& hi, uint32_t (&h)[16])
{
    i8_to_f16(lo.x, h[0], h[1]);
    i8_to_f16(lo.y, h[2], h[3]);
    i8_to_f16(lo.z, h[4], h[5]);
    i8_to_f16(lo.w, h[6], h[7]);
    i8_to_f16(hi.x, h[8], h[9]);
    i8_to_f16(hi.y, h[10], h[11]);
    i8_to_f16(hi.z, h[12], h[13]);
    i8_to_f16(hi.w, h[14], h[15]);
}

}  // namespace w4k
