// win_bwd.cuh -- what the windowed backward's kernels share.
#pragma once

#include <cmath>

#include "bwd_tile.cuh"

namespace fa {

struct WinBwdArgs {
    const float* ws_delta;  // [BH][Np], negated: -delta_i
    const float* ws_lse2;   // [BH][Np], negated: -lse_i * log2(e)
    void* dk;
    void* dv;
    int N, Np, n_kv, BH;    // BH: K/V heads (B * H_kv), the grid's head count
    int H, H_kv;            // query heads and K/V heads per batch; H_kv divides H
    WinSplit split;         // sink blocks' pieces
    float* part;            // their dV, dK: [BH][n_part][pieces + 1][2][d / 4][128][4] float32
    float c_log2;           // scale * log2(e), not 0
    float scale;
    DevCtl ctl;
};

using BwdArgs = WinBwdArgs;

// An item: one K/V head's 128-key block kvb with the query blocks of its window, or a piece of a
// sink block's later query blocks.  Pieces come first, then the key blocks in order: all but a
// head's last ones meet equally many.
static __device__ __forceinline__ int far_items(const BwdArgs& a) { return a.split.n_part * a.split.pieces * a.BH; }
static __device__ __forceinline__ Item item_at(const BwdArgs& a, int x) {
    const int n_far = far_items(a), n_q = a.n_kv, reach = a.split.reach;
    Item I;
    I.bh = x % a.BH;
    const int y = x / a.BH;
    if (x < n_far) {
        I.kvb = y % a.split.n_part;
        const int piece = y / a.split.n_part;
        I.i0 = I.kvb + reach + 1 + piece * a.split.per;
        I.n_loc = max(0, min(a.split.per, n_q - I.i0));
        I.slot = 1 + piece;
    } else {
        I.kvb = y - a.split.n_part * a.split.pieces;
        I.i0 = I.kvb;
        I.n_loc = min(n_q - 1, I.kvb + reach) - I.kvb + 1;
        I.slot = I.kvb < a.split.n_part ? 0 : -1;
    }
    // with grouped-query attention, that range for each of the query heads that share this K/V
    // head (dK, dV sum over all of them)
    I.n_it = a.H / a.H_kv * I.n_loc;
    return I;
}
// The query blocks of an item one after the other, without a division a step.
struct WinWalk {
    int head, blk, end, i0;
    __device__ __forceinline__ WinWalk(const BwdArgs& a, const Item& I)
        : head((I.bh / a.H_kv) * a.H + (I.bh % a.H_kv) * (a.H / a.H_kv)), blk(I.i0), end(I.i0 + I.n_loc), i0(I.i0) {}
    __device__ __forceinline__ void next() {
        if (++blk == end) {
            blk = i0;
            ++head;
        }
    }
};
static __device__ __forceinline__ int item_count(const BwdArgs& a) { return far_items(a) + a.n_kv * a.BH; }
static __device__ __forceinline__ WinWalk walk_of(const BwdArgs& a, const Item& I) { return WinWalk(a, I); }
static __device__ __forceinline__ int key_rows(const BwdArgs& a) { return a.N; }
static __device__ __forceinline__ size_t part_of(const BwdArgs& a, const Item& I) {
    return (static_cast<size_t>(I.bh) * a.split.n_part + I.kvb) * (a.split.pieces + 1) + I.slot;
}
static __device__ __forceinline__ constexpr bool hides(const BwdArgs&) { return false; }
// A key's queries counted from query q0: from the key on, a window's worth, or all for a sink.
static __device__ __forceinline__ void query_range(const BwdArgs& a, const Item&, int key, int q0, int& q_first, int& q_end) {
    const WinSplit& sp = a.split;
    q_first = key - q0;
    const long long end = static_cast<long long>(q_first) + sp.window;
    q_end = key < sp.sinks ? kBlk : static_cast<int>(min(static_cast<long long>(kBlk), end));
}

// dV and dK of the blocks that were dealt in parts: the parts added in order, dK times scale,
// rounded once.  Thread t of n (whole warps), eight neighbouring values of a row at a time: a warp
// takes 8 rows x 32 columns, whole lines of the parts and 64-byte runs of the result.
template <int D>
static __device__ __forceinline__ void join_parts(const BwdArgs& a, int t, int n) {
    constexpr int kCols = D / 32, kTiles = kCols * (kBlk / 8);  // such tiles of a block's dV or dK
    const WinSplit& sp = a.split;
    const size_t work = static_cast<size_t>(a.BH) * sp.n_part * 2 * kTiles * 32;
    for (size_t x = t; x < work; x += n) {
        const int lane = static_cast<int>(x % 32), tile = static_cast<int>(x / 32 % kTiles);
        const int row = tile / kCols * 8 + lane % 8, vec = tile % kCols * 4 + lane / 8;
        const int which = static_cast<int>(x / (32 * kTiles) % 2);
        const size_t blk = x / (2 * 32 * kTiles);  // bh * n_part + kvb
        const int kvb = static_cast<int>(blk % sp.n_part);
        const size_t bh = blk / sp.n_part;
        const int key = kvb * kBlk + row;
        if (key >= a.N) continue;
        const int slots = 1 + (a.n_kv - 1 - sp.reach - kvb + sp.per - 1) / sp.per;
        const float4* src =
            reinterpret_cast<const float4*>(a.part) + (blk * (sp.pieces + 1) * 2 + which) * (kBlk * D / 4) + 2 * vec * kBlk + row;
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
#pragma unroll 4
        for (int i = 0; i < slots; ++i) {
            const float4 y = src[0], z = src[kBlk];
            u.x += y.x, u.y += y.y, u.z += y.z, u.w += y.w;
            w.x += z.x, w.y += z.y, w.z += z.z, w.w += z.w;
            src += 2 * (kBlk * D / 4);
        }
        const float f = which ? a.scale : 1.f;
        static_cast<uint4*>(which ? a.dk : a.dv)[(bh * a.N + key) * (D / 8) + vec] =
            make_uint4(pack_bf16x2(u.x * f, u.y * f), pack_bf16x2(u.z * f, u.w * f), pack_bf16x2(w.x * f, w.y * f),
                       pack_bf16x2(w.z * f, w.w * f));
    }
}

// dK and dV of the windowed backward for d = 64; grid: CTAs.
cudaError_t launch_bwd_window_main64(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                                     const CUtensorMap& dk, const CUtensorMap& dv, const WinBwdArgs& a, int grid,
                                     cudaStream_t s);
// dQ, and the join of the parts that the dK/dV kernel has left.
int launch_bwd_window_dq(const void* q, const void* k, const void* v, const void* dO, void* dq, const WinBwdArgs& a, int d,
                         cudaStream_t s);

}  // namespace fa
