// vp_pair.cuh -- how the kernels on CTA pairs (clusters of two CTAs) end when a
// bounded wait has run out. Their barriers (Bars) have, beside the ring's full[] and
// empty[]:
//   uint64_t done;      // the leader's: every MMA is done
//   uint32_t fills;     // stages that this CTA has filled, stored before it ends
//   uint32_t gave_up;   // 0 at first
#pragma once

#include <stdint.h>

#include "vp_gemm_host.cuh"
#include "vp_tma.cuh"
#include "vp_waits.h"

namespace vp {

// Arrive once on a barrier of this CTA when the pair MMAs issued so far by this thread have completed.
__device__ __forceinline__ void umma_commit_pair_here(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// A bounded wait ran out: flagged for the host and, before they leave, for both CTAs.
template <class Bars>
__device__ __forceinline__ void pair_gives_up(Bars &bars, uint32_t bit) {
    atomicOr(&g_linear_fault, bit);
    st_cluster_u32(cluster_addr(&bars.gave_up, 0), 1u);
    st_cluster_u32(cluster_addr(&bars.gave_up, 1), 1u);
}

// At a producer's end: every stage it filled is used, so its copies have landed and the
// arrivals that say so as well. False where that did not come to pass.
template <int kStages, class Bars>
__device__ __forceinline__ bool pair_ring_used(Bars &bars, uint32_t fills) {
    for (uint32_t i = 0; i < (uint32_t)kStages; ++i) {
        const LateStage l = late_stage(i, fills, fills, kStages);
        if (l.owed != kOwedNothing && !mbar_wait_cluster(&bars.empty[i], l.parity)) return false;
    }
    return true;
}

// The last thing that all threads of both CTAs do before the tensor memory is given
// back: no arrival or copy targets either CTA behind it. Where a wait ran out, the
// leader waits (again with a limit) for the copies of both that are still under way;
// kStageBytes: a CTA's half of a stage.
template <int kStages, uint32_t kStageBytes, class Bars>
__device__ __forceinline__ void pair_ends(Bars &bars, uint32_t rank) {
    cluster_sync();
    if (!bars.gave_up) return;                            // the same in both
    if (rank == 0 && threadIdx.x == 0) {
        const uint32_t peer = ld_cluster_u32(cluster_addr(&bars.fills, 1));
        for (uint32_t i = 0; i < (uint32_t)kStages; ++i) {
            const LateStage l = late_stage(i, bars.fills, peer, kStages);
            if (l.owed == kOwedNothing) continue;
            if (l.owed == kOwedNoPeer) mbar_complete_tx(&bars.full[i], kStageBytes);
            if (l.owed == kOwedNoLeader) mbar_arrive_expect_tx(&bars.full[i], kStageBytes);
            if (!mbar_wait_cluster(&bars.full[i], l.parity)) break;
        }
    }
    __syncthreads();
    cluster_sync();
}

}  // namespace vp
