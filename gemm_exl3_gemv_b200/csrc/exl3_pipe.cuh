// exl3_pipe.cuh -- what the warp-specialised kernels of the cache's attention
// and of the 4-bit products share: places in rings and waits that give up.
#pragma once
#include "exl3_common.cuh"

namespace exl3 {

// Place and phase in a ring.
template <int SIZE>
struct Turn {
    int at = 0;
    uint32_t phase = 0;
    template <int BY = 1>                                    // a divisor of SIZE
    __device__ __forceinline__ void next()
    {
        at += BY;
        if (at >= SIZE) {
            at -= SIZE;
            phase ^= 1;
        }
    }
};

// Waits of a warp that give up after 2 s: after the first that runs out the
// others return at once.  The warp tries once; if that fails, its first lane
// waits, suspended in hardware: in a CTA of 27 warps those that poll took the
// issue slots of the others (a 4-bit product of 32 rows: 28.5 us, 24.5 so).
struct Patience {
    uint32_t* status;
    bool alive;
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity)
    {
        if (!alive || __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
        int there = 1;
        if ((threadIdx.x & 31) == 0) {
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait_sleep(bar, parity, 1000))
                if (global_ns() - t0 > 2000000000ull) {
                    there = 0;
                    atomicOr(status, kStatusTimeout);
                    break;
                }
        }
        alive = __shfl_sync(0xffffffffu, there, 0) != 0;
    }
};

// Waits, with the same limit, for the last of `issued` copies that a warp sent
// round a ring, copy i to place i % SIZE, whose barrier's phase they complete:
// none is on its way to a CTA's shared memory when the CTA ends, whichever
// waits ran out.
template <int SIZE>
__device__ __forceinline__ void copies_landed(uint64_t* bars, int issued, uint32_t* status)
{
    Patience p = {status, true};
    for (int i = max(0, issued - SIZE); i < issued; ++i) p.wait(bars + i % SIZE, (uint32_t)(i / SIZE) & 1u);
}

// A named barrier over `threads` threads that tells each of them whether any of
// them said yes: the same answer for all, with nothing in shared memory that a
// faster warp could write over.
__device__ __forceinline__ bool named_bar_any(int id, int threads, bool yes)
{
    int any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(id), "r"(threads), "r"(yes ? 1 : 0)
        : "memory");
    return any != 0;
}

}  // namespace exl3
