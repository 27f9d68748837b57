// cross_bwd_dq_sm103.cu -- dQ of the backward of attention to another sequence's keys.
#include "bwd_dq.cuh"
#include "cross_bwd.cuh"

namespace fa {

// A head's query blocks one after the other (those of a piece of its keys), so that neighbouring CTAs read the
// same K and V.
struct CrossQItem {
    int bh, bh_kv, qb, n_kv, len;
    static constexpr bool shorty = false, kParts = false;
    __device__ __forceinline__ int block(int j) const { return j; }
};
static __device__ __forceinline__ CrossQItem q_item_at(const CrossBwdArgs& a, int x) {
    CrossQItem I;
    I.bh = x / a.n_q;
    I.qb = x - I.bh * a.n_q;
    const int b = I.bh / a.H_kv, kv_batch = b / a.share;
    I.bh_kv = kv_batch * a.H_kv + I.bh - b * a.H_kv;
    I.len = a.lengths ? min(max(__ldcg(a.lengths + kv_batch), 0), a.N_kv) : a.N_kv;  // (from L2, as the rows' values)
    I.n_kv = key_blocks(I.len);
    return I;
}
// Apart, as the pieces' arithmetic would cost every item of the others some hundred cycles (a step of 8 x 512
// queries on 100 to 512 keys 76 -> 79 us).
struct CrossQPiece : CrossQItem {
    int first, part;
    static constexpr bool kParts = true;
    __device__ __forceinline__ int block(int j) const { return first + j; }
};
static __device__ __forceinline__ CrossQPiece q_item_at(const CrossPieceArgs& a, int x) {
    const int run = x / a.n_q, head = run / a.pieces_q, piece = run - head * a.pieces_q;  // run: of a head and a piece
    CrossQPiece I = {q_item_at(static_cast<const CrossBwdArgs&>(a), x - (run - head) * a.n_q), piece * a.per_q, -1};
    if (I.n_kv > a.per_q) I.part = (I.bh * a.n_q + I.qb) * a.pieces_q + piece;
    I.n_kv = min(a.per_q, max(0, I.n_kv - I.first));
    return I;
}
// Sequences of up to 32 keys (6 x 2629 queries of 16 heads on 4 keys 94 -> 88 us with the rest of the step).  As a
// property of each item it would cost the others 2 to 4%.
struct CrossQShort : CrossQItem {
    static constexpr bool shorty = true;
};
static __device__ __forceinline__ CrossQShort q_item_at(const CrossShortArgs& a, int x) {
    return {q_item_at(static_cast<const CrossBwdArgs&>(a), x)};
}
// From L2: where this kernel starts beside the one before it, it has waited for none, and its SM's L1 may hold an
// earlier call's.
static __device__ __forceinline__ float row_value(const CrossBwdArgs&, const float* p) { return __ldcg(p); }
static __device__ __forceinline__ void key_range(const CrossBwdArgs&, const CrossQItem& I, int, int key0, int& first,
                                                 int& last, int& sink) {
    first = -1;
    last = I.len - 1 - key0;
    sink = 0;
}
static __device__ __forceinline__ bool hidden_rows(const CrossBwdArgs& a, const CrossQItem& I, int block, int& r0, int& r1) {
    r0 = max(0, I.len - block * kBlk);
    r1 = min(kBlk, a.N_kv - block * kBlk);
    return r0 < r1;
}
// This kernel may start when every CTA of the dK/dV kernel has waited for the rows' values (and all that came
// before them); it needs nothing of that kernel, but what comes after it may.
template <int D>
static __device__ __forceinline__ void idle_warp(const CrossBwdArgs&, std::integral_constant<int, D>, int, int) {
    griddep_wait();
}

namespace {

// Up to two items an SM have a CTA each, launched programmatically, which takes over an SM as soon as the dK/dV kernel
// leaves it or at once (a step of 2 x 900 queries on 2000 keys 90 -> 83 us, 12 x 82 on 272-2179 112 -> 105, 8 x 8 on 16
// 23 -> 19).  With several items a CTA the order in which SMs get free undoes the deal, which costs up to 10%; with
// three CTAs an SM their starts do (1681 on 21 41.7 -> 45.3).
template <int D, class Args>
cudaError_t launch_impl(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO, void* dq,
                        const Args& a, int sms, cudaStream_t s) {
    static std::atomic<uint64_t> smem_done;
    const cudaError_t e = allow_smem(bwd_dq_kernel<D, Args>, Cfg<D>::kSmemAlloc, smem_done);
    if (e != cudaSuccess) return e;
    const int n_items = a.BH_kv * a.share * a.n_q * a.pieces_q, grid = n_items <= 2 * sms ? n_items : sms;
    if (n_items <= 2 * sms)
        return launch_pdl(bwd_dq_kernel<D, Args>, dim3(grid), dim3(kThreads), Cfg<D>::kSmemAlloc, s, q, k, v, dO, a, dq, n_items);
    bwd_dq_kernel<D, Args><<<grid, kThreads, Cfg<D>::kSmemAlloc, s>>>(q, k, v, dO, a, dq, n_items);
    return cudaGetLastError();
}
template <class Args>
cudaError_t launch_d(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO, void* dq,
                     const Args& a, int d, int sms, cudaStream_t s) {
    return d == 64 ? launch_impl<64>(q, k, v, dO, dq, a, sms, s) : launch_impl<128>(q, k, v, dO, dq, a, sms, s);
}

}  // namespace

cudaError_t launch_bwd_cross_dq(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                                void* dq, const CrossBwdArgs& a, int d, int sms, cudaStream_t s) {
    if (a.N_kv <= 32) return launch_d(q, k, v, dO, dq, CrossShortArgs{a}, d, sms, s);
    if (a.pieces_q == 1) return launch_d(q, k, v, dO, dq, a, d, sms, s);
    return launch_d(q, k, v, dO, dq, CrossPieceArgs{a}, d, sms, s);
}

}  // namespace fa
