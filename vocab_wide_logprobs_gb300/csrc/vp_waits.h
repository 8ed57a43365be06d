// vp_waits.h -- which copies a kernel still has to wait for when it ends, however
// it ends: bulk copies write to shared memory and arrive on barriers there, so a
// CTA may not leave before they have landed. Plain C++, also compiled for the host
// by the tests.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define VP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define VP_HOST_DEVICE inline
#endif

namespace vp {

// A ring of n stages, filled in turn by two CTAs (each its half of a stage, both
// counted on the leader's barrier, which the leader arms for both) that have begun
// `leader` and `peer` fills. A stage is filled again only after both halves of its
// last fill were used, so at most a stage's last fill is under way, and the two
// counts of it differ by at most one. For a ring of one CTA the counts are the same.
enum Owed : uint32_t {
    kOwedNothing,   // never filled
    kOwedAll,       // wait for the phase
    kOwedNoPeer,    // the peer's half never comes: take its bytes off first
    kOwedNoLeader   // only the peer's half comes: arm the phase for it first
};
struct LateStage {
    Owed owed;
    uint32_t parity;   // of the stage's last phase
};
VP_HOST_DEVICE LateStage late_stage(uint32_t stage, uint32_t leader, uint32_t peer, uint32_t n) {
    // fills of this stage by each: those of the numbers stage, stage + n, ...
    const uint32_t a = (leader + n - 1 - stage) / n, b = (peer + n - 1 - stage) / n, last = a > b ? a : b;
    if (last == 0) return LateStage{kOwedNothing, 0u};
    return LateStage{a == b ? kOwedAll : a > b ? kOwedNoPeer : kOwedNoLeader, (last - 1) & 1u};
}

// Two buffers that bulk copies fill in turn, each with a barrier of its own: bit b of
// `parity` is that of the phase which the next wait for buffer b is for, and flips with
// every wait, whether it ended or ran out. After one that ran out its phase is still
// open and the arrival on it spent, so no copy may be begun on that barrier again.
VP_HOST_DEVICE uint32_t next_phase(uint32_t parity, uint32_t b) { return parity >> b & 1u; }

// The fault word that a caller reads (vp_fault_status in include/vp.h), of the words of
// the forward scans, of the matrix products and of the rules' kernels: bits of their
// own, so that it says whose outputs are void.
VP_HOST_DEVICE uint32_t fault_word(uint32_t scans, uint32_t products, uint32_t rules) {
    return scans | products << 2 | (rules ? 32u : 0u);
}

}  // namespace vp
