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
    I.len = key_count(a, kv_batch);
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
// This kernel starts when every CTA of the dK/dV kernel has seen the rows' values ready; it needs nothing of that
// kernel, but what comes after it may.
template <int D>
static __device__ __forceinline__ void idle_warp(const CrossBwdArgs&, std::integral_constant<int, D>, int, int) {
    griddep_wait();
}

namespace {

template <int D, class Args>
int launch_impl(const void* q, const void* k, const void* v, const void* dO, void* dq, const Args& a, int main_ctas,
                cudaStream_t s) {
    const int heads = a.BH_kv * a.share, n_items = heads * a.n_q * a.pieces_q;
    CUtensorMap tq, tk, tv, tdo;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = make_map_3d(&tq, q, dt, 2, D, a.N, heads, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, D, a.N_kv, a.BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, D, a.N_kv, a.BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tdo, dO, dt, 2, D, a.N, heads, 64, kBlk);
    if (rc != 0) return rc;
    static std::atomic<uint64_t> smem_done;
    cudaError_t e = allow_smem(bwd_dq_kernel<D, Args>, Cfg<D>::kSmemAlloc, smem_done);
    int dev = 0, sms = 152;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    const int grid = n_items < sms ? n_items : sms;
    if (n_items <= sms || main_ctas + grid <= sms)
        return static_cast<int>(launch_pdl(bwd_dq_kernel<D, Args>, dim3(grid), dim3(kThreads), Cfg<D>::kSmemAlloc, s,
                                           tq, tk, tv, tdo, a, dq, n_items));
    bwd_dq_kernel<D, Args><<<grid, kThreads, Cfg<D>::kSmemAlloc, s>>>(tq, tk, tv, tdo, a, dq, n_items);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_bwd_cross_dq(const void* q, const void* k, const void* v, const void* dO, void* dq, const CrossBwdArgs& a, int d,
                        int main_ctas, cudaStream_t s) {
    if (a.pieces_q > 1) {
        const CrossPieceArgs p = {a};
        return d == 64 ? launch_impl<64>(q, k, v, dO, dq, p, main_ctas, s) : launch_impl<128>(q, k, v, dO, dq, p, main_ctas, s);
    }
    return d == 64 ? launch_impl<64>(q, k, v, dO, dq, a, main_ctas, s) : launch_impl<128>(q, k, v, dO, dq, a, main_ctas, s);
}

}  // namespace fa
