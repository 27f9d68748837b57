// win_bwd64_sm103.cu -- dK and dV of the windowed backward for d = 64.
#include "bwd_main64.cuh"
#include "win_bwd.cuh"

namespace fa {

cudaError_t launch_bwd_window_main64(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                                     const CUtensorMap& dk, const CUtensorMap& dv, const WinBwdArgs& a, int grid,
                                     cudaStream_t s) {
    static std::atomic<uint64_t> smem_done;
    const cudaError_t e = allow_smem(bwd64_kernel<BwdArgs>, kSmemAlloc, smem_done);
    if (e != cudaSuccess) return e;
    // set up while win_bwd_prep runs: 0.8% of a step (the d = 128 kernel lost as much that way)
    return launch_pdl(bwd64_kernel<BwdArgs>, dim3(grid), dim3(kThreads), kSmemAlloc, s, q, k, v, dO, dk, dv, a);
}

}  // namespace fa
