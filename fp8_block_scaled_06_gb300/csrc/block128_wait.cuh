// The mbarrier wait of the block-128 product kernels.
#pragma once
#include "block128.h"
#include "kernel_common.cuh"

namespace fp8g {

// Bounded wait of a whole warp, for a phase that orders no memory of this proxy by
// itself (tcgen05.commit, TMA, the relaxed arrivals): every lane asks, which is
// quicker than one lane's answer handed round; a wait that runs long goes on in
// wait_bar_warp.
__device__ __forceinline__ bool b128_wait_all(uint32_t bar, uint32_t parity, volatile int *abort_flag, const B128Params &p,
                                              unsigned detail) {
    return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)) ||
           wait_bar_warp(bar, parity, abort_flag, p, detail);
}

}  // namespace fp8g
