// vp_gemm_host.cuh -- what the translation units with tensor-core kernels and the
// rules' share: the fault word of their bounded waits, and on the host the driver's
// tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace vp {

// Set when a bounded wait of this translation unit's kernels gave up.
static __device__ uint32_t g_linear_fault;   // one per translation unit

// Reads (and optionally clears) this translation unit's fault word.
static cudaError_t read_tu_fault(uint32_t *value, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_linear_fault, sizeof(uint32_t));
    if (e == cudaSuccess && clear && *value) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_linear_fault, &zero, sizeof(uint32_t));
    }
    return e;
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load();
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

}  // namespace vp
