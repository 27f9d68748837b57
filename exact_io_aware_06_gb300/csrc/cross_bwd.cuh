// cross_bwd.cuh -- the backward of attention to another sequence's keys: its arguments, and which blocks
// its kernels take (the overloads that bwd_tile.cuh and bwd_dq.cuh name).
//
// As in the forward the G N_q rows of the query heads that share a K/V head in one batch are the R rows of
// one longer head.  A key block meets all of their 128-row blocks, those of every batch that shares
// the keys one after the other; where there are fewer key blocks than SMs these are dealt in pieces,
// whose float32 dK and dV are added in order afterwards.  So are the key blocks of a query block for dQ.
#pragma once

#include "bwd_tile.cuh"

namespace fa {

struct CrossBwdArgs {
    const float* ws_delta;  // [B][H_kv][Np], negated: -delta_i
    const float* ws_lse2;   // [B][H_kv][Np], negated: -lse_i * log2(e)
    void* dk;
    void* dv;
    float* part;            // with pieces > 1: dV, dK [BH_kv][n_k][pieces][2][d / 4][128][4] float32
    const int* lengths;     // [B_kv] or null
    int N, Np;              // R and that in whole blocks
    int N_kv, n_q, n_k;     // keys; blocks of queries and of keys
    float* part_q;          // with pieces_q > 1: dQ [B H_kv][n_q][pieces_q][d / 4][128][4] float32
    int share, H_kv, BH_kv;
    int per, pieces;        // query blocks of a piece, over the batches that share
    int per_q, pieces_q;    // key blocks of a piece of dQ
    float c_log2;           // scale * log2(e), not 0
    float scale;
    DevCtl ctl;
};
struct CrossPieceArgs : CrossBwdArgs {};  // for dQ in pieces
struct CrossShortArgs : CrossBwdArgs {};  // for dQ of up to 32 keys

static __device__ __forceinline__ int key_count(const CrossBwdArgs& a, int kv_batch) {
    return a.lengths ? min(max(__ldg(a.lengths + kv_batch), 0), a.N_kv) : a.N_kv;
}

// A sequence without keys has one block, all of it hidden: its queries' gradients are zeros from it.
static __device__ __forceinline__ int key_blocks(int len) { return max(1, (len + kBlk - 1) / kBlk); }

struct CrossItem {
    int bh, kvb, i0, n_it;
    int slot;  // -1: dK and dV are final; else the part that this item leaves
    int len;
};
static __device__ __forceinline__ int item_count(const CrossBwdArgs& a) { return a.BH_kv * a.n_k * a.pieces; }
static __device__ __forceinline__ CrossItem item_at(const CrossBwdArgs& a, int x) {
    CrossItem I;
    I.bh = x % a.BH_kv;
    const int y = x / a.BH_kv, piece = y / a.n_k;
    I.kvb = y - piece * a.n_k;
    I.len = key_count(a, I.bh / a.H_kv);
    I.i0 = piece * a.per;
    I.n_it = I.kvb * kBlk < I.len ? min(a.per, a.share * a.n_q - I.i0) : 0;
    I.slot = a.pieces > 1 ? piece : -1;
    return I;
}
struct CrossWalk {
    int head, blk, n_q, step;
    __device__ __forceinline__ void next() {
        if (++blk == n_q) {
            blk = 0;
            head += step;
        }
    }
};
static __device__ __forceinline__ CrossWalk walk_of(const CrossBwdArgs& a, const CrossItem& I) {
    const int b = I.bh / a.H_kv, over = I.i0 / a.n_q;
    return {(b * a.share + over) * a.H_kv + I.bh - b * a.H_kv, I.i0 - over * a.n_q, a.n_q, a.H_kv};
}
static __device__ __forceinline__ void query_range(const CrossBwdArgs&, const CrossItem& I, int key, int, int& q_first,
                                                   int& q_end) {
    q_first = 0;
    q_end = key < I.len ? kBlk : 0;
}
static __device__ __forceinline__ int key_rows(const CrossBwdArgs& a) { return a.N_kv; }
static __device__ __forceinline__ size_t part_of(const CrossBwdArgs& a, const CrossItem& I) {
    return (static_cast<size_t>(I.bh) * a.n_k + I.kvb) * a.pieces + I.slot;
}
static __device__ __forceinline__ constexpr bool hides(const CrossBwdArgs&) { return true; }

// dK and dV for d = 64; grid: CTAs.
cudaError_t launch_bwd_cross_main64(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                                    const CUtensorMap& dk, const CUtensorMap& dv, const CrossBwdArgs& a, int grid,
                                    cudaStream_t s);
// dQ of all B * H_kv heads of R rows, on `sms` SMs, after (or beside) dK and dV.
cudaError_t launch_bwd_cross_dq(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                                void* dq, const CrossBwdArgs& a, int d, int sms, cudaStream_t s);

}  // namespace fa
