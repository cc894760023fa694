// tcg_pipe.cuh -- the bounded barrier waits of the pipelined kernels.  Ctl is a kernel's
// control block in shared memory (abort_flag), Args its arguments (err, wait_limit_ns).
#pragma once

#include "tcg_ptx.cuh"

namespace tcg {

// Raise the abort flag in this CTA and, for a pair, in the peer CTA.
template <int CG, typename Ctl, typename Args>
__device__ __forceinline__ void raise_abort(Ctl *ctl, const Args &p, uint32_t err_bit)
{
    ctl->abort_flag = 1;
    if constexpr (CG == 2)
        st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int *>(&ctl->abort_flag)),
                                          cluster_ctarank() ^ 1u),
                              1u);
    atomicOr(p.err, err_bit);
}

// Bounded wait on an mbarrier phase.  Returns false if the kernel was aborted or the
// limit ran out (then the error bit is recorded and the abort flag raised).
template <int CG, typename Ctl, typename Args>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, Ctl *ctl,
                                             const Args &p, uint32_t err_bit,
                                             bool honour_abort = true)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (honour_abort && ctl->abort_flag)
            return false;
        if (globaltimer_ns() - t0 > p.wait_limit_ns) {
            raise_abort<CG>(ctl, p, err_bit);
            return false;
        }
    }
}

}  // namespace tcg
