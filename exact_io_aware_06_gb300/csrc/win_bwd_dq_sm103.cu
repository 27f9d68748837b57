// win_bwd_dq_sm103.cu -- dQ of the windowed backward, and the join of the parts that its dK/dV kernel has
// left.
#include "bwd_dq.cuh"
#include "win_bwd.cuh"

namespace fa {

struct WinQItem {
    static constexpr bool kParts = false;
    int bh, bh_kv, qb, lo, n_sink, n_kv;
    bool shorty;  // the first block is that of up to 32 sinks, in front of the window
    __device__ __forceinline__ int block(int j) const { return j < n_sink ? j : lo + j - n_sink; }
};
static __device__ __forceinline__ WinQItem q_item_at(const WinBwdArgs& args, int x) {
    const int q_heads = args.BH / args.H_kv * args.H;
    WinQItem I;
    I.bh = x % q_heads;
    I.qb = args.n_kv - 1 - x / q_heads;
    // grouped-query attention: query head bh reads K/V head bh_kv of its group
    I.bh_kv = (I.bh / args.H) * args.H_kv + (I.bh % args.H) / (args.H / args.H_kv);
    // key blocks: the sinks' in front of the window, then lo .. qb
    I.lo = max(0, static_cast<int>(static_cast<long long>(I.qb) * kBlk - args.split.window + 1)) / kBlk;
    I.n_sink = min(I.lo, (args.split.sinks + kBlk - 1) / kBlk);
    I.n_kv = I.n_sink + I.qb - I.lo + 1;
    I.shorty = I.n_sink > 0 && args.split.sinks <= 32;
    return I;
}
static __device__ __forceinline__ float row_value(const WinBwdArgs&, const float* p) { return *p; }
static __device__ __forceinline__ void key_range(const WinBwdArgs& args, const WinQItem&, int row, int key0, int& first, int& last,
                                          int& sink) {
    last = row - key0;
    sink = args.split.sinks - key0;
    first = static_cast<int>(max(-1ll, static_cast<long long>(last) - args.split.window + 1));
}
// The sinks' parts of dK and dV that the kernel before has left.
template <int D>
static __device__ __forceinline__ void idle_warp(const WinBwdArgs& args, std::integral_constant<int, D>, int t, int n) {
    if (args.split.n_part > 0) join_parts<D>(args, t, n);
}

namespace {

template <int D>
int launch_impl(const void* q, const void* k, const void* v, const void* dO, void* dq, const WinBwdArgs& a, cudaStream_t s) {
    const int BH_kv = a.BH, BH = BH_kv / a.H_kv * a.H, N = a.N, n_items = a.n_kv * BH;
    CUtensorMap tq, tk, tv, tdo;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = make_map_3d(&tq, q, dt, 2, D, N, BH, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, D, N, BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, D, N, BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tdo, dO, dt, 2, D, N, BH, 64, kBlk);
    if (rc != 0) return rc;
    static std::atomic<uint64_t> smem_done;
    cudaError_t e = allow_smem(bwd_dq_kernel<D, WinBwdArgs>, Cfg<D>::kSmemAlloc, smem_done);
    int dev = 0, sms = 152;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    // An ordinary launch.  Launched with programmatic serialization, its CTAs taking over the SMs as
    // those of the dK/dV kernel finish (of which dQ needs nothing), a step took 2-3% longer.
    bwd_dq_kernel<D, WinBwdArgs>
        <<<n_items < sms ? n_items : sms, kThreads, Cfg<D>::kSmemAlloc, s>>>(tq, tk, tv, tdo, a, dq, n_items);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_bwd_window_dq(const void* q, const void* k, const void* v, const void* dO, void* dq, const WinBwdArgs& a, int d,
                         cudaStream_t s) {
    return d == 64 ? launch_impl<64>(q, k, v, dO, dq, a, s) : launch_impl<128>(q, k, v, dO, dq, a, s);
}

}  // namespace fa
