// cross_bwd64_sm103.cu -- dK and dV of the backward of attention to another sequence's keys for d = 64.
#include "bwd_main64.cuh"
#include "cross_bwd.cuh"

namespace fa {

cudaError_t launch_bwd_cross_main64(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                                    const CUtensorMap& dk, const CUtensorMap& dv, const CrossBwdArgs& a, int grid,
                                    cudaStream_t s) {
    static std::atomic<uint64_t> smem_done;
    const cudaError_t e = allow_smem(bwd64_kernel<CrossBwdArgs>, kSmemAlloc, smem_done);
    if (e != cudaSuccess) return e;
    return launch_pdl(bwd64_kernel<CrossBwdArgs>, dim3(grid), dim3(kThreads), kSmemAlloc, s, q, k, v, dO, dk, dv, a);
}

}  // namespace fa
