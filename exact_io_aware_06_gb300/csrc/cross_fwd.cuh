// cross_fwd.cuh -- attention to another sequence's keys: what the kernels of the forward share.
#pragma once

#include "cross_deal.cuh"
#include "fwd_tile.cuh"
#include "layer_ops.h"
#include "ptx.cuh"

namespace fa {

// Attention of up to four rows a K/V head and batch (all of share R), on 2^cluster CTAs each.
cudaError_t launch_cross_few(const CrossArgs& a, int d, const void* q, const void* k, const void* v, cudaStream_t s);

namespace {

__device__ __forceinline__ void cluster_sync() {  // what any thread of the cluster wrote before is visible after
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
constexpr int kPartTile = kBM;  // rows of a part's second tile start here

// A row's end from its state (reference maximum m in log2 units, sum l): the factor of O, and lse.
__device__ __forceinline__ float row_factor(float l) { return l == 0.f ? 0.f : __frcp_rn(l); }
__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// Floats of one part: O of its rows, then m and l.
__host__ __device__ inline size_t part_floats(int D, int part_rows) {
    return static_cast<size_t>(part_rows) * (D + 2);
}

}  // namespace
}  // namespace fa
