// win_fwd.cuh -- what the two windowed forward kernels share: their arguments, the plan of key
// blocks that a pair of query tiles visits, and per-thread pieces.
#pragma once

#include <cmath>

#include "fwd_tile.cuh"
#include "layer_ops.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kShort = 32;     // keys of a short sink block
constexpr int kThreads = 384;  // 12 warps

struct WinArgs {
    float* lse;
    int N, n_pairs, BH, n_items;
    int window, sinks;
    float c_log2;  // scale * log2(e), not 0
    int H, H_kv;
    DevCtl ctl;
};

// Which key blocks a pair of query tiles visits.  List index n: blocks 0 .. n_sink - 1, then
// lo .. ; the first is a short one if `shorty`.  Tile 0 leaves out the last entry when tile 1
// has a diagonal block of its own, tile 1 leaves out entry skip1 (-1: none).
struct Plan {
    int n;          // entries
    int n_sink, lo;
    int skip1;
    bool shorty, two;
    __device__ __forceinline__ int block(int i) const { return i < n_sink ? i : lo + i - n_sink; }
    __device__ __forceinline__ bool active(int t, int i) const {
        return t ? (two && i != skip1) : (!two || i != n - 1);
    }
};
__device__ __forceinline__ Plan plan_of(const WinArgs& a, int r0) {
    Plan p;
    p.two = r0 + kBM < a.N;
    p.lo = max(0, static_cast<int>(static_cast<long long>(r0) - a.window + 1)) / kBN;
    const int lo1 = max(0, static_cast<int>(static_cast<long long>(r0) + kBM - a.window + 1)) / kBN;
    const int last = r0 / kBN + (p.two ? 1 : 0);
    p.shorty = a.sinks > 0 && a.sinks <= kShort && p.lo > 0;
    p.n_sink = min(p.lo, a.sinks / kBN + (a.sinks % kBN ? 1 : 0));
    p.n = p.n_sink + last - p.lo + 1;
    // tile 1 sees nothing of block lo if its window starts behind it and no sink lies in it
    p.skip1 = (p.two && lo1 > p.lo && static_cast<long long>(p.lo) * kBN >= a.sinks) ? p.n_sink : -1;
    return p;
}

// What a launch of either kernel needs besides its tensor maps.
inline WinArgs win_args(float* lse, int B, int H, int H_kv, int N, float c_log2, int window, int sinks, DevCtl ctl) {
    WinArgs a;
    a.lse = lse;
    a.N = N;
    a.n_pairs = (N + 2 * kBM - 1) / (2 * kBM);
    a.BH = B * H;
    a.n_items = a.n_pairs * a.BH;
    a.window = window;
    a.sinks = sinks < N ? sinks : N;
    // a scale of 0 makes all scores 0; the mask multiplies -inf by c, which has to stay -inf
    a.c_log2 = c_log2 == 0.f ? 1e-30f : c_log2;
    a.H = H;
    a.H_kv = H_kv;
    a.ctl = ctl;
    return a;
}
// The tensor maps of q, k, v (128-row boxes) and o (a warp's 32 rows).
inline int win_maps(CUtensorMap (&m)[4], const void* q, const void* k, const void* v, const void* o, int B, int H, int H_kv,
                    int N, int d) {
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = make_map_3d(&m[0], q, dt, 2, d, N, B * H, 64, kBM);
    if (rc == 0) rc = make_map_3d(&m[1], k, dt, 2, d, N, B * H_kv, 64, kBN);
    if (rc == 0) rc = make_map_3d(&m[2], v, dt, 2, d, N, B * H_kv, 64, kBN);
    if (rc == 0) rc = make_map_3d(&m[3], o, dt, 2, d, N, B * H, 64, 32);
    return rc;
}

}  // namespace
}  // namespace fa
