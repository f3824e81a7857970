// Beside common.cuh, for the kernels of cross attention, whose warps have roles of
// their own: waits that keep a warp together, the end of a CTA with work in
// flight, 3-D TMA, either 16-bit type.
#pragma once

#include "common.cuh"
#include "ring.h"

namespace mbert {

// limit of a wait for what a CTA still has in flight when it ends (100 ms or more)
constexpr long long kDrainClocks = 250000000;

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v)
{
    asm volatile("st.volatile.shared.u32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}

// mbar_wait for the roles of a CTA that share the shared-memory word at
// `gave_up` (0 at first): a wait that gives up sets it, and ends the others'
// early.  A lane must not leave its warp alone before an instruction of the
// whole warp, and to compare the lanes' results at each wait costs 8 % (209 us
// against 194, 8192 x 8192 cross attention, 12 heads of 64); so such roles go on
// as if the wait had passed, on whatever their tiles hold then, and look at the
// word (all lanes together, any_gave_up) before they use anything as an address
// or write to global memory.
__device__ __forceinline__ bool mbar_wait_mark(uint32_t bar, uint32_t parity, int *err, uint32_t gave_up)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const unsigned long long t0 = globaltimer_ns();
    const long long c0 = clock64();
    constexpr long long climit = static_cast<long long>(kWaitLimitNs) * 5 / 2;
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, 20000u))
            return true;
        if (lds32(gave_up))
            return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs || clock64() - c0 > climit)
            break;
    }
    sts32(gave_up, 1u);
    atomicOr(err, kErrTimeout);
    return false;
}

// Has a wait of this CTA given up?  One answer for the warp; no means that
// every wait of its lanes so far has passed.
__device__ __forceinline__ bool any_gave_up(uint32_t gave_up)
{
    return __any_sync(0xffffffffu, lds32(gave_up) != 0u);
}

// A CTA must not end, nor give its shared memory or TMEM to the next one, before
// what it has issued is done, even where a wait has given up.  These waits take
// at most kDrainClocks each and report nothing: where something is late, the
// wait that needed it has.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity)
{
    const long long c0 = clock64();
    while (!mbar_try_wait_sleep(bar, parity, 1000000u) && clock64() - c0 < kDrainClocks)
        ;
}
// The `issued` loads of a ring whose barriers lie from bar0 on.
__device__ __forceinline__ void ring_drain(uint32_t bar0, uint32_t issued, uint32_t stages)
{
#pragma unroll 1
    for (uint32_t t = ring_pending(issued, stages); t < issued; ++t)
        drain_wait(bar0 + 8u * ring_slot(t, stages), ring_parity(t, stages));
}

// 3-D tiled load of the box at (x, y, z); otherwise as tma_load_2d.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int x, int y, int z,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// Two numbers as a pair of fp16 or bf16.
template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (kHalf)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace mbert
