// cross_bwd_sm103.cu -- backward of attention to another sequence's keys, by recomputation on the sm_103a
// tensor core.
//
// The mathematics are the plain backward's (bwd_sm103.cu) over the keys j < len_b:
//     P_ij = exp(S_ij - lse_i),  dV = P^T dO,  dP = dO V^T,  delta_i = dO_i . O_i,
//     dS = P o (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,
// dK and dV summed over the query heads and the batches that share a K/V head.  Kernels on one stream:
// prep (delta, padded -lse log2 e; zeros for dK and dV of key blocks without keys), dK/dV per 128-key block
// (bwd_main128.cuh, bwd_main64.cuh), dQ (bwd_dq.cuh), the join of their pieces where there are any.  Nothing is
// summed by atomics: the same bits every time.
//
// Measured: 4 x 2048 queries of 16 heads on 300-1000 keys, d = 64: prep 9 us, dK/dV 57, dQ 43 (the tensor pipe 34% and
// 33% busy: the exponentials' warps and their hand-overs, as in bwd_main64.cuh); 1021 queries of 16 / 4 heads on
// 8191 keys, d = 128: prep 5, dK/dV 97, dQ 73 on 128 of the 152 SMs (58%, inside an item 81%).
#include "bwd_main128.cuh"
#include "cross_bwd.cuh"

namespace fa {
namespace {

// Sequences of up to kNarrow keys take delta_i = sum_j P_ij dP_ij: dO . o carries the rounding of o to bf16,
// as much as dS's own where few keys average out in o (the windowed backward's measurements).
constexpr int kNarrow = 24;

struct PrepArgs {
    const uint4 *o, *dO, *q, *k, *v;
    const float* lse;
    float *ws_delta, *ws_lse2;
    CrossBwdArgs b;
};

// -delta_i and -lse_i log2(e) (rows past R: 0 and -inf, so that recomputed P is exactly 0 there; so too
// for a sequence without keys, whose lse is -inf).  Both are stored negated so that the other kernels add
// them with packed FMA/FADD.  A warp takes 16 rows; a lane (g, t) values 32 c + 8 t .. + 7 of rows g
// and g + 8.  With few keys S and dP are m16n8k16 products of the same layout, eight keys at a time,
// multiplied element by element; the order of d in a product is free, so that operands are a lane's 16
// neighbouring bytes, of which the first four values serve one product and the rest the next.
template <int D>
__global__ void __launch_bounds__(256) cross_bwd_prep_kernel(const PrepArgs a) {
    griddep_wait();               // O, dO may come from the kernel before this one
    griddep_launch_dependents();  // the main kernel may launch and set up meanwhile
    constexpr int kC = D / 32, kT = D / 8;  // 16-byte loads of a lane and of a row
    const CrossBwdArgs& b = a.b;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int N = b.N, Np = b.Np, tiles_head = Np / 16;
    const long long tiles = static_cast<long long>(b.BH_kv) * b.share * tiles_head;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (long long x = static_cast<long long>(blockIdx.x) * 8 + warp; x < tiles; x += static_cast<long long>(gridDim.x) * 8) {
        const int bh = static_cast<int>(x / tiles_head), i0 = static_cast<int>(x % tiles_head) * 16;
        const int batch = bh / b.H_kv, kv_batch = batch / b.share;
        const int len = key_count(b, kv_batch);
        const size_t q_row = static_cast<size_t>(bh) * N;
        uint4 d[2][kC], y[2][kC];  // rows i0 + g, i0 + g + 8 of dO and of o or q
        const uint4* other = len <= kNarrow ? a.q : a.o;
        float nl[2], delta[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = i0 + g + 8 * r;
            const size_t at = (q_row + i) * kT + t;
            const bool there = i < N && len > 0;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                d[r][c] = there ? a.dO[at + 4 * c] : zero;
                y[r][c] = there ? other[at + 4 * c] : zero;
            }
            nl[r] = there ? -a.lse[q_row + i] * kLog2e : -INFINITY;
        }
        if (len > kNarrow) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int c = 0; c < kC; ++c) delta[r] += dot8(d[r][c], y[r][c]);
        } else {
            const size_t k_row = static_cast<size_t>(kv_batch * b.H_kv + bh % b.H_kv) * b.N_kv;
            for (int kt = 0; kt < len; kt += 8) {
                const bool there = kt + g < len;  // this lane's key
                const size_t at = (k_row + kt + g) * kT + t;
                float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const uint4 k = there ? a.k[at + 4 * c] : zero, v = there ? a.v[at + 4 * c] : zero;
                    mma_bf16(s, y[0][c].x, y[1][c].x, y[0][c].y, y[1][c].y, k.x, k.y);
                    mma_bf16(s, y[0][c].z, y[1][c].z, y[0][c].w, y[1][c].w, k.z, k.w);
                    mma_bf16(dp, d[0][c].x, d[1][c].x, d[0][c].y, d[1][c].y, v.x, v.y);
                    mma_bf16(dp, d[0][c].z, d[1][c].z, d[0][c].w, d[1][c].w, v.z, v.w);
                }
                // rows g, g + 8 and keys kt + 2 t, kt + 2 t + 1
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (kt + 2 * t + e % 2 < len)
                        delta[e / 2] = fmaf(ex2_approx(fmaf(s[e], b.c_log2, nl[e / 2])), dp[e], delta[e / 2]);
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
    if (b.lengths == nullptr) return;
    // dK and dV of key blocks that the main kernel passes over
    const int blocks = b.BH_kv * b.n_k;
    for (int x = blockIdx.x; x < blocks; x += gridDim.x) {
        const int bh = x / b.n_k, row0 = (x - bh * b.n_k) * kBlk;
        if (row0 < key_count(b, bh / b.H_kv)) continue;
        const size_t first = (static_cast<size_t>(bh) * b.N_kv + row0) * kT;
        const int n = min(kBlk, b.N_kv - row0) * kT;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            static_cast<uint4*>(b.dk)[first + i] = zero;
            static_cast<uint4*>(b.dv)[first + i] = zero;
        }
    }
}

// What was dealt in pieces: the float32 parts added in order, times a factor, rounded once.  blockIdx.x: dV and dK
// of every key block, then dQ of every query block.  A warp takes 8 rows x 32 columns, whole lines of the parts
// and 64-byte runs of the result, of every WARPS-th part; the warps' sums meet in shared memory.  Few blocks of
// many parts need more than a warp a tile: 2 blocks of 53 33 -> 7 us, 6 of 25 at d = 128 31 -> 8.
template <int D, int WARPS>
__global__ void __launch_bounds__(256) cross_bwd_join_kernel(const CrossBwdArgs a, void* const dq, const int key_places) {
    constexpr int kCols = D / 32, kTiles = kCols * (kBlk / 8);
    __shared__ float4 sums[WARPS > 1 ? 8 : 1][2][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, first = warp % WARPS;
    griddep_wait();
    const float4* src;
    uint4* out;  // of the block's first row
    int rows, n;
    float f = a.scale;
    if (static_cast<int>(blockIdx.x) < key_places) {
        const int place = static_cast<int>(blockIdx.x) / 2, which = blockIdx.x % 2;
        const int bh = place / a.n_k, row0 = (place - bh * a.n_k) * kBlk;
        if (row0 >= key_count(a, bh / a.H_kv)) return;  // zeros already
        src = reinterpret_cast<const float4*>(a.part) + (static_cast<size_t>(place) * a.pieces * 2 + which) * (kBlk * D / 4);
        out = static_cast<uint4*>(which ? a.dk : a.dv) + (static_cast<size_t>(bh) * a.N_kv + row0) * (D / 8);
        rows = a.N_kv - row0;
        n = a.pieces;
        if (which == 0) f = 1.f;
    } else {
        const int place = static_cast<int>(blockIdx.x) - key_places, bh = place / a.n_q, row0 = (place - bh * a.n_q) * kBlk;
        const int blocks = key_blocks(key_count(a, bh / a.H_kv / a.share));
        if (blocks <= a.per_q) return;  // one piece, which wrote the result
        src = reinterpret_cast<const float4*>(a.part_q) + static_cast<size_t>(place) * a.pieces_q * (kBlk * D / 4);
        out = static_cast<uint4*>(dq) + (static_cast<size_t>(bh) * a.N + row0) * (D / 8);
        rows = a.N - row0;
        n = (blocks + a.per_q - 1) / a.per_q;
    }
    const int step = (static_cast<int>(blockIdx.x) < key_places ? 2 : 1) * (kBlk * D / 4);
    const int tile = blockIdx.y * (8 / WARPS) + warp / WARPS;
    const int row = tile / kCols * 8 + lane % 8, vec = tile % kCols * 4 + lane / 8;
    static_assert(kTiles % (8 / WARPS) == 0, "whole CTAs");
    const float4* p = src + 2 * vec * kBlk + row + static_cast<size_t>(first) * step;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
    if (row < rows) {
#pragma unroll 4
        for (int i = first; i < n; i += WARPS) {
            const float4 y = p[0], z = p[kBlk];
            u.x += y.x, u.y += y.y, u.z += y.z, u.w += y.w;
            w.x += z.x, w.y += z.y, w.z += z.z, w.w += z.w;
            p += static_cast<size_t>(WARPS) * step;
        }
    }
    if constexpr (WARPS > 1) {
        sums[warp][0][lane] = u;
        sums[warp][1][lane] = w;
        __syncthreads();
        if (first > 0) return;
#pragma unroll
        for (int i = 1; i < WARPS; ++i) {
            const float4 y = sums[warp + i][0][lane], z = sums[warp + i][1][lane];
            u.x += y.x, u.y += y.y, u.z += y.z, u.w += y.w;
            w.x += z.x, w.y += z.y, w.z += z.z, w.w += z.w;
        }
    }
    if (row < rows)
        out[row * (D / 8) + vec] = make_uint4(pack_bf16x2(u.x * f, u.y * f), pack_bf16x2(u.z * f, u.w * f),
                                              pack_bf16x2(w.x * f, w.y * f), pack_bf16x2(w.z * f, w.w * f));
}
template <int D>
cudaError_t join(const CrossBwdArgs& a, void* dq, int key_places, int places, cudaStream_t s) {
    constexpr int kTiles = D / 32 * (kBlk / 8);
    const int most = a.pieces > a.pieces_q ? a.pieces : a.pieces_q;
    if (most >= 8) return launch_pdl(cross_bwd_join_kernel<D, 8>, dim3(places, kTiles), dim3(256), 0, s, a, dq, key_places);
    return launch_pdl(cross_bwd_join_kernel<D, 1>, dim3(places, kTiles / 8), dim3(256), 0, s, a, dq, key_places);
}

// delta and lse rows in bytes; the parts follow
size_t rows_bytes(const CrossBwdArgs& a) { return 2 * static_cast<size_t>(a.BH_kv) * a.share * a.Np * sizeof(float); }
size_t part_bytes(const CrossBwdArgs& a, int d) {
    return a.pieces > 1 ? static_cast<size_t>(a.BH_kv) * a.n_k * a.pieces * 2 * kBlk * d * sizeof(float) : 0;
}
size_t part_q_bytes(const CrossBwdArgs& a, int d) {
    return a.pieces_q > 1 ? static_cast<size_t>(a.BH_kv) * a.share * a.n_q * a.pieces_q * kBlk * d * sizeof(float) : 0;
}

// `blocks` blocks that meet `all` others each: in how many pieces these are dealt.  The number that gives the
// busiest of 152 CTAs the least to do, counted in pairs of blocks, with `edge` more an item for its start and end,
// `part` a part for its way to memory and back, and `join` for the launch of the join.
// 152 SMs, whatever the current device: the workspace's size and the order of the sums follow from the sizes
// alone.
void pieces_of(long long blocks, long long all, double edge, double part, double join, int* per_piece, int* pieces) {
    double least = 0;
    for (int p = 1; p <= 64 && p <= all && (p == 1 || blocks < 304); ++p) {
        const long long per = (all + p - 1) / p, n = (all + per - 1) / per;
        const double cost = static_cast<double>((blocks * n + 151) / 152) * (per + edge) +
                            (n > 1 ? join + part * blocks * n : 0);
        if (p == 1 || cost < least) {
            least = cost;
            *per_piece = static_cast<int>(per);
            *pieces = static_cast<int>(n);
        }
    }
}
// Sizes and pieces.  At d = 128 a pair of blocks takes 1.3 us for dK and dV, whose parts of 128 KB take about 0.06 us
// of all SMs, less at d = 64 and where a block has fewer keys than rows; for dQ 0.9 us, and a part half of that;
// the join 4 us unless there is one already.
CrossBwdArgs deal(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    CrossBwdArgs a = {};
    a.N = H / H_kv * N_q;
    a.Np = round_up(a.N, kBlk);
    a.N_kv = N_kv;
    a.n_q = a.Np / kBlk;
    a.n_k = (N_kv + kBlk - 1) / kBlk;
    a.share = B / B_kv;
    a.H_kv = H_kv;
    a.BH_kv = B_kv * H_kv;
    auto filled = [&](int rows) { return (rows < kBlk ? rows : kBlk) * d / (128.0 * kBlk); };  // of a part of 64 KB
    pieces_of(static_cast<long long>(a.BH_kv) * a.n_k, static_cast<long long>(a.share) * a.n_q, 1.5, 0.045 * filled(N_kv),
              3, &a.per, &a.pieces);
    pieces_of(static_cast<long long>(a.BH_kv) * a.share * a.n_q, a.n_k, 2, 0.03 * filled(a.N), a.pieces > 1 ? 0 : 5,
              &a.per_q, &a.pieces_q);
    return a;
}

}  // namespace

size_t bwd_cross_workspace_bytes(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    const CrossBwdArgs a = deal(B, B_kv, H, H_kv, N_q, N_kv, d);
    return rows_bytes(a) + part_bytes(a, d) + part_q_bytes(a, d);
}

int launch_bwd_cross(const void* q, const void* k, const void* v, const int* lengths, const void* o, const float* lse,
                     const void* dO, void* dq, void* dk, void* dv, void* workspace, int B, int B_kv, int H, int H_kv,
                     int N_q, int N_kv, int d, float scale, DevCtl ctl, cudaStream_t s) {
    PrepArgs pa;
    CrossBwdArgs& a = pa.b;
    a = deal(B, B_kv, H, H_kv, N_q, N_kv, d);
    const int heads = a.BH_kv * a.share;
    pa.ws_delta = static_cast<float*>(workspace);
    pa.ws_lse2 = pa.ws_delta + static_cast<size_t>(heads) * a.Np;
    a.ws_delta = pa.ws_delta;
    a.ws_lse2 = pa.ws_lse2;
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + rows_bytes(a));
    a.part_q = a.part + part_bytes(a, d) / sizeof(float);
    a.dk = dk;
    a.dv = dv;
    a.lengths = lengths;
    a.c_log2 = scale == 0.f ? 1e-30f : scale * kLog2e;  // not 0: the mask multiplies -inf by it
    a.scale = scale;
    a.ctl = ctl;
    pa.o = static_cast<const uint4*>(o);
    pa.dO = static_cast<const uint4*>(dO);
    pa.q = static_cast<const uint4*>(q);
    pa.k = static_cast<const uint4*>(k);
    pa.v = static_cast<const uint4*>(v);
    pa.lse = lse;

    int sms = 152, dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    CUtensorMap tq, tk, tv, tdo, tdk, tdv;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = make_map_3d(&tq, q, dt, 2, d, a.N, heads, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, d, N_kv, a.BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, d, N_kv, a.BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tdo, dO, dt, 2, d, a.N, heads, 64, kBlk);
    // d = 64: dK, dV written in boxes of a warp's 32 rows
    if (rc == 0 && d == 64) rc = make_map_3d(&tdk, dk, dt, 2, d, N_kv, a.BH_kv, 64, 32);
    if (rc == 0 && d == 64) rc = make_map_3d(&tdv, dv, dt, 2, d, N_kv, a.BH_kv, 64, 32);
    if (rc != 0) return rc;
    // CTAs for the rows, or for the key blocks that may have to be zeroed (few rows on long ragged sequences)
    const int for_rows = grid_for(static_cast<size_t>(heads) * (a.Np / 16), 8, sms * 8);
    const int for_keys = lengths ? grid_for(static_cast<size_t>(a.BH_kv) * a.n_k, 1, sms * 4) : 0;
    e = launch_pdl(d == 64 ? cross_bwd_prep_kernel<64> : cross_bwd_prep_kernel<128>,
                   dim3(for_rows > for_keys ? for_rows : for_keys), dim3(256), 0, s, pa);
    if (e != cudaSuccess) return static_cast<int>(e);
    const int n_items = a.BH_kv * a.n_k * a.pieces;
    const int grid = n_items < sms ? n_items : sms;
    if (d == 64) {
        e = launch_bwd_cross_main64(tq, tk, tv, tdo, tdk, tdv, a, grid, s);
    } else {
        static std::atomic<uint64_t> smem_done;
        e = allow_smem(bwd_main_kernel<CrossBwdArgs>, kSmemAlloc, smem_done);
        if (e != cudaSuccess) return static_cast<int>(e);
        e = launch_pdl(bwd_main_kernel<CrossBwdArgs>, dim3(grid), dim3(kThreads), kSmemAlloc, s, tq, tk, tv, tdo, a);
    }
    if (e == cudaSuccess) e = launch_bwd_cross_dq(tq, tk, tv, tdo, dq, a, d, sms, s);
    const int key_places = a.pieces > 1 ? 2 * a.BH_kv * a.n_k : 0;
    const int places = key_places + (a.pieces_q > 1 ? heads * a.n_q : 0);
    if (e != cudaSuccess || places == 0) return static_cast<int>(e);
    return static_cast<int>(d == 64 ? join<64>(a, dq, key_places, places, s) : join<128>(a, dq, key_places, places, s));
}

}  // namespace fa
