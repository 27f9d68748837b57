// win_bwd_sm103.cu -- backward of attention under a causal sliding window with sinks, by
// recomputation on the sm_103a tensor core.
//
// The mathematics are the plain backward's (bwd_sm103.cu), over the pairs (i, j) that the
// forward saw, j <= i and (j > i - W or j < S):
//     P_ij = exp(S_ij - lse_i),  dV = P^T dO,  dP = dO V^T,  delta_i = dO_i . O_i,
//     dS = P o (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q.
//
// Kernels on one stream: win_bwd_prep (delta and padded -lse log2 e), the main kernel (dK and dV in
// TMEM per 128-key block: bwd_main128.cuh and bwd_main64.cuh), and a query-parallel
// kernel for dQ (win_bwd_dq_sm103.cu), which also joins the sinks' parts.  Nothing is summed by
// atomics: the same bits every time.  (For d = 64 the plain backward's scheme, dQ partials added to a
// float32 accumulator by TMA reductions, was also measured: the main kernel took 79 us of a B4 H16
// N2048 W512 step, zeroing and converting the accumulator 13 more; dK/dV and dQ take 52 and 42.)
//
// What the window changes:
//   * A key block j meets the query blocks j .. j + (W + 126) / 128 only.
//   * A block that holds sinks meets all later query blocks too: N / 128 of them where the
//     others meet W / 128, so that one CTA would still be at it long after the rest are done.
//     Its later query blocks are dealt in pieces, as items of their own, first of all; the
//     pieces of a block leave float32 dK and dV in the workspace, and an idle warp of the dQ
//     kernel adds them in order and rounds once.
//   * The visible queries of a key row are a range; blocks that hold its ends take them as
//     bit words made by shifts.
//   * dS is taken from P before its rounding to bf16: with P rounded first, dQ and dK carried two
//     bf16 roundings before their own.
#include "bwd_main128.cuh"
#include "win_bwd.cuh"

namespace fa {
namespace {

// ---------------------------------------------------------------- pre / post passes
// -delta_i and -lse_i * log2(e) (rows past N: 0 and -inf, so that recomputed P is exactly 0 there).
// Both are stored negated so the main kernels add them with packed FMA/FADD.  D / 8 threads per row.
//
// delta_i = dO_i . O_i takes the O that the forward rounded to bf16, which is off by up to 2^-8 |O| |dO|
// beside dP's spread: little against dS's own rounding where many keys average out in O, as much as
// it at four keys.  A head's first kFirst rows, which see kFirst keys at most and have the largest
// gradients, take delta_i = sum_j P_ij dP_ij instead, in `extra` CTAs beside the others, a warp a row
// (dQ's error relative to 64 bits, N1024 W512 d64: 2.54e-3 -> 2.46e-3 for 1% of a step).  So do all rows
// of sequences of up to kShort, and under a window and sinks of up to kNarrow keys in all, in a kernel
// of their own.
constexpr int kFirst = 16, kNarrow = 24, kShort = 128;

struct PrepArgs {
    const uint4 *o, *dO, *q, *k, *v;
    const float* lse;
    float *ws_delta, *ws_lse2;
    int BH, H, H_kv, N, Np;
    int window, sinks;
    float c_log2;
    int extra;
};

// sum_j P_ij dP_ij of row i < min(N, kFirst) of query head bh, by one warp: D / 8 lanes a key, two
// such rounds of keys at a time.
template <int D>
__device__ __forceinline__ float delta_of_first(const PrepArgs& a, int bh, int i) {
    constexpr int kT = D / 8, kSlots = 32 / kT;
    const int lane = threadIdx.x % 32, part = lane % kT;
    const int lo = max(0, static_cast<int>(max(-1ll, static_cast<long long>(i) - a.window + 1)));
    const int front = min(a.sinks, lo), n = front + i - lo + 1;  // sinks in front of the window; keys
    const size_t row = static_cast<size_t>(bh) * a.N + i;
    const size_t kv = static_cast<size_t>((bh / a.H) * a.H_kv + (bh % a.H) / (a.H / a.H_kv)) * a.N;
    const uint4 q = a.q[row * kT + part], d = a.dO[row * kT + part], zero = make_uint4(0, 0, 0, 0);
    const float nl = -a.lse[row] * kLog2e;
    float delta = 0.f;
    for (int t = lane / kT; t - lane / kT < n; t += 2 * kSlots) {
        uint4 k[2], v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int x = t + u * kSlots;
            const size_t at = (kv + (x < front ? x : lo + x - front)) * kT + part;
            k[u] = x < n ? a.k[at] : zero;
            v[u] = x < n ? a.v[at] : zero;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float p = ex2_approx(fmaf(lanes_sum<1, kT>(dot8(q, k[u])), a.c_log2, nl));
            const float dp = lanes_sum<1, kT>(dot8(d, v[u]));
            if (t + u * kSlots < n) delta = fmaf(p, dp, delta);
        }
    }
    return lanes_sum<kT, 32>(delta);
}

template <int D>
__global__ void __launch_bounds__(256, 8) win_bwd_prep_kernel(const PrepArgs a) {
    griddep_wait();               // O, dO may come from the kernel before this one
    griddep_launch_dependents();  // the main kernel may launch and set up meanwhile
    constexpr int kT = D / 8;     // threads per row (8 or 16): the shuffles stay inside a warp
    const int N = a.N, Np = a.Np, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (static_cast<int>(blockIdx.x) < a.extra) {
        const long long rows = static_cast<long long>(a.BH) * kFirst, step = a.extra * 8;
        for (long long r = blockIdx.x * 8 + warp; r < rows; r += step) {
            const int bh = static_cast<int>(r / kFirst), i = static_cast<int>(r % kFirst);
            if (i >= N) continue;
            const float delta = delta_of_first<D>(a, bh, i);
            if (lane == 0) a.ws_delta[static_cast<size_t>(bh) * Np + i] = -delta;
        }
        return;
    }
    const int part = lane % kT;
    const size_t tid = static_cast<size_t>(blockIdx.x - a.extra) * blockDim.x + threadIdx.x;
    const size_t nthreads = static_cast<size_t>(gridDim.x - a.extra) * blockDim.x;
    const size_t rows = static_cast<size_t>(a.BH) * Np;
    for (size_t base = tid; base < rows * kT; base += nthreads) {
        const size_t r = base / kT;
        const int bh = static_cast<int>(r / Np), i = static_cast<int>(r % Np);
        float sum = 0.f;
        if (i < N) {
            const size_t src = (static_cast<size_t>(bh) * N + i) * kT + part;
            sum = dot8(a.o[src], a.dO[src]);
        }
        sum = lanes_sum<1, kT>(sum);
        if (part == 0) {
            if (i >= N || i >= kFirst) a.ws_delta[r] = -sum;
            a.ws_lse2[r] = (i < N) ? -a.lse[static_cast<size_t>(bh) * N + i] * kLog2e : -INFINITY;
        }
    }
}

// The same rows of the workspace for few keys: delta_i = sum_j P_ij dP_ij.  A warp takes 16
// query rows with the keys that any of them sees, eight at a time: S and dP as m16n8k16 products of
// the same layout, multiplied element by element.  Against dO . o, a step of B4 H16 N2048 d64: W2 83 ->
// 92 us and dQ's error 3.8e-3 -> 2.35e-3, W16 84 -> 95 and 2.5e-3 -> 2.34e-3 (W32 84 -> 100 and 2.48e-3 ->
// 2.36e-3, hence kNarrow).  The order of d in a product is free, so that a lane
// (row or key g, t) loads its operands as 16 neighbouring bytes: values 32 c + 8 t .. + 7, of which the
// first four serve one product and the rest the next.  Bound by memory: q, k, v and dO are read here
// (and by the kernels after this one, from L2) where the other kernel reads o and dO.
template <int D>
__global__ void __launch_bounds__(256) win_bwd_narrow_prep_kernel(const PrepArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kC = D / 32, kT = D / 8;  // 16-byte loads of a lane and of a row
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int N = a.N, Np = a.Np, tiles_head = Np / 16;
    const long long tiles = static_cast<long long>(a.BH) * tiles_head;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (long long x = static_cast<long long>(blockIdx.x) * 8 + warp; x < tiles; x += static_cast<long long>(gridDim.x) * 8) {
        const int bh = static_cast<int>(x / tiles_head), i0 = static_cast<int>(x % tiles_head) * 16;
        const size_t q_row = static_cast<size_t>(bh) * N;
        const size_t k_row = static_cast<size_t>((bh / a.H) * a.H_kv + (bh % a.H) / (a.H / a.H_kv)) * N;
        uint4 q[2][kC], d[2][kC];  // rows i0 + g, i0 + g + 8
        float nl[2], delta[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = i0 + g + 8 * r;
            const size_t at = (q_row + i) * kT + t;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                q[r][c] = i < N ? a.q[at + 4 * c] : zero;
                d[r][c] = i < N ? a.dO[at + 4 * c] : zero;
            }
            nl[r] = i < N ? -a.lse[q_row + i] * kLog2e : -INFINITY;
        }
        const int start = max(0, i0 - a.window + 1) & ~7, end = min(i0 + 16, N);  // the window's keys
        const int front = min(a.sinks, start);                                    // sinks before them
        for (int kt = front > 0 ? 0 : start; kt < end; kt = kt < front && kt + 8 >= front ? start : kt + 8) {
            const bool of_front = kt < front;
            const int key = kt + g;  // this lane's
            const bool there = key < N;
            const size_t at = (k_row + key) * kT + t;
            float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const uint4 k = there ? a.k[at + 4 * c] : zero, v = there ? a.v[at + 4 * c] : zero;
                mma_bf16(s, q[0][c].x, q[1][c].x, q[0][c].y, q[1][c].y, k.x, k.y);
                mma_bf16(s, q[0][c].z, q[1][c].z, q[0][c].w, q[1][c].w, k.z, k.w);
                mma_bf16(dp, d[0][c].x, d[1][c].x, d[0][c].y, d[1][c].y, v.x, v.y);
                mma_bf16(dp, d[0][c].z, d[1][c].z, d[0][c].w, d[1][c].w, v.z, v.w);
            }
            // rows g, g + 8 and keys 2 t, 2 t + 1
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + g + 8 * (e / 2), j = kt + 2 * t + e % 2;
                const bool seen = of_front ? j < front : j <= i && (j > i - a.window || j < a.sinks);
                if (seen) delta[e / 2] = fmaf(ex2_approx(fmaf(s[e], a.c_log2, nl[e / 2])), dp[e], delta[e / 2]);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float sum = lanes_sum<1, 4>(delta[r]);
            if (t == 0) {
                const size_t at = static_cast<size_t>(bh) * Np + i0 + g + 8 * r;
                a.ws_delta[at] = -sum;
                a.ws_lse2[at] = nl[r];
            }
        }
    }
}

}  // namespace

namespace {

// delta and lse rows in bytes; the parts follow
size_t rows_bytes(int BH, int N) {
    return 2 * static_cast<size_t>(BH) * static_cast<size_t>(round_up(N, kBlk)) * sizeof(float);
}

}  // namespace

// How a sink block's later query blocks are dealt: pieces no shorter than a window's run of
// blocks, at most 64 a block, and together about two per SM, which keeps any one of them
// below the mean load of a CTA (B1 H_kv1 N131072 W1024: 1024 later blocks in 64 pieces of 16
// against 60 blocks a CTA).  Two per SM of 152, whatever the current device: the workspace's size and
// the order of the sums follow from the sizes alone.
WinSplit win_split(int B, int H_kv, int N, int window, int sinks) {
    const int n_q = (N + kBlk - 1) / kBlk;
    WinSplit sp;
    sp.window = window;
    sp.sinks = sinks < N ? sinks : N;
    const long long reach = (static_cast<long long>(window) + kBlk - 2) / kBlk;
    sp.reach = static_cast<int>(reach < n_q - 1 ? reach : n_q - 1);
    const int later = n_q - 1 - sp.reach;  // of block 0; one fewer for each block after it
    const int n_sink = (sp.sinks + kBlk - 1) / kBlk;
    sp.n_part = n_sink < later ? n_sink : later;
    sp.per = 1;
    sp.pieces = 0;
    if (sp.n_part > 0) {
        const long long blocks = static_cast<long long>(B) * H_kv * sp.n_part;
        long long most = (304 + blocks - 1) / blocks;
        if (most > 64) most = 64;
        sp.per = static_cast<int>((later + most - 1) / most);
        if (sp.per < sp.reach + 1) sp.per = sp.reach + 1;
        sp.pieces = (later + sp.per - 1) / sp.per;
    }
    return sp;
}

size_t bwd_window_workspace_bytes(int B, int H, int H_kv, int N, int d, int window, int sinks) {
    const WinSplit sp = win_split(B, H_kv, N, window, sinks);
    return rows_bytes(B * H, N) +
           static_cast<size_t>(B) * H_kv * sp.n_part * (sp.pieces + 1) * 2 * kBlk * d * sizeof(float);
}

int launch_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                      void* dq, void* dk, void* dv, void* workspace, int B, int H, int H_kv, int N, int d, float scale,
                      int window, int sinks, DevCtl ctl, cudaStream_t s) {
    const WinSplit sp = win_split(B, H_kv, N, window, sinks);
    const int BH = B * H, BH_kv = B * H_kv;  // query heads; K/V heads
    const int Np = round_up(N, kBlk);
    float* ws_delta = static_cast<float*>(workspace);
    float* ws_lse2 = ws_delta + static_cast<size_t>(BH) * Np;

    int sms = 152, dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    PrepArgs pa;
    pa.o = static_cast<const uint4*>(o);
    pa.dO = static_cast<const uint4*>(dO);
    pa.q = static_cast<const uint4*>(q);
    pa.k = static_cast<const uint4*>(k);
    pa.v = static_cast<const uint4*>(v);
    pa.lse = lse;
    pa.ws_delta = ws_delta;
    pa.ws_lse2 = ws_lse2;
    pa.BH = BH;
    pa.H = H;
    pa.H_kv = H_kv;
    pa.N = N;
    pa.Np = Np;
    pa.window = window;
    pa.sinks = sp.sinks;
    pa.c_log2 = scale == 0.f ? 1e-30f : scale * kLog2e;
    if (N <= kShort || static_cast<long long>(window) + sp.sinks <= kNarrow) {
        pa.extra = 0;
        e = launch_pdl(d == 64 ? win_bwd_narrow_prep_kernel<64> : win_bwd_narrow_prep_kernel<128>,
                       dim3(grid_for(static_cast<size_t>(BH) * Np / 16, 8, sms * 4)), dim3(256), 0, s, pa);
    } else {
        pa.extra = grid_for(static_cast<size_t>(BH) * kFirst, 8, 2 * sms);
        const int others = grid_for(static_cast<size_t>(BH) * Np * (d / 8), 256, sms * 8 - pa.extra);
        e = launch_pdl(d == 64 ? win_bwd_prep_kernel<64> : win_bwd_prep_kernel<128>, dim3(others + pa.extra), dim3(256), 0,
                       s, pa);
    }
    if (e != cudaSuccess) return static_cast<int>(e);

    CUtensorMap tq, tk, tv, tdo, tdk, tdv;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = make_map_3d(&tq, q, dt, 2, d, N, BH, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, d, N, BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, d, N, BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tdo, dO, dt, 2, d, N, BH, 64, kBlk);
    // d = 64: dK, dV written in boxes of a warp's 32 rows
    if (rc == 0 && d == 64) rc = make_map_3d(&tdk, dk, dt, 2, d, N, BH_kv, 64, 32);
    if (rc == 0 && d == 64) rc = make_map_3d(&tdv, dv, dt, 2, d, N, BH_kv, 64, 32);
    if (rc != 0) return rc;
    BwdArgs a;
    a.ws_delta = ws_delta;
    a.ws_lse2 = ws_lse2;
    a.dk = dk;
    a.dv = dv;
    a.N = N;
    a.Np = Np;
    a.n_kv = Np / kBlk;
    a.BH = BH_kv;
    a.H = H;
    a.H_kv = H_kv;
    a.split = sp;
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + rows_bytes(BH, N));
    a.c_log2 = scale == 0.f ? 1e-30f : scale * kLog2e;  // not 0: the mask multiplies -inf by it
    a.scale = scale;
    a.ctl = ctl;
    // persistent: one CTA per SM (fewer if there are fewer items), each looping over items.  An
    // ordinary launch, as of the causal plain backward: the deal takes it that every CTA
    // starts together.
    const int n_items = (a.n_kv + sp.n_part * sp.pieces) * BH_kv;
    const int grid = n_items < sms ? n_items : sms;
    if (d == 64) {
        e = launch_bwd_window_main64(tq, tk, tv, tdo, tdk, tdv, a, grid, s);
    } else {
        static std::atomic<uint64_t> smem_done;
        e = allow_smem(bwd_main_kernel<BwdArgs>, kSmemAlloc, smem_done);
        if (e != cudaSuccess) return static_cast<int>(e);
        bwd_main_kernel<BwdArgs><<<grid, kThreads, kSmemAlloc, s>>>(tq, tk, tv, tdo, a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return static_cast<int>(e);
    return launch_bwd_window_dq(q, k, v, dO, dq, a, d, s);
}

}  // namespace fa
