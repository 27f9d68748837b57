// cross_few_sm103.cu -- attention of a few rows of queries (single tokens) to another sequence's keys.
//
// With up to four rows to a K/V head in a batch a tile of 128 is nearly empty, and what a call costs is a tile's way
// through the tensor core: 2.9 us for every two blocks of keys, where their bytes take 1.  Here the keys stream through
// registers: D / 8 lanes hold a key's 16 bytes each, multiply them with each row's part of q, and add up p V in the
// same places; a lane group keeps a running maximum and sum of its own.  The states of a warp's groups, of a CTA's
// eight warps and of the up to eight CTAs of a cluster that share a K/V head are joined in a fixed order.  Everything
// is float32 up to the result.
//
// Bound by HBM on long sequences, as long as a warp's next 16 keys are in flight while it works on these (64 x 16
// heads on 1500-4096 keys, d = 64: 112 us, 6.5 TB/s; without 130; by tiles 129), by the loads' latency on short ones,
// where more CTAs an SM and nothing ahead are better (64 x 16 heads on 100 keys 7.6 us; with loads ahead 11.1; by tiles
// 23).  One token of 16 heads on 1500 keys 4.7 us (by tiles 8.2).  CTAs an SM: three of 80 registers where there are
// many (128 x 16 heads on 700-1500 keys 89 -> 83 us), two of 110 where there are few (8 heads on 2900 keys 7.5 -> 6.1).
#include "cross_fwd.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;
constexpr int kTogether = 4;  // keys of a lane group in flight

// A state over some of the keys, of one row and some columns: reference maximum (log2 units) and sum.
__device__ __forceinline__ float state_weight(float m, float l, float top) {
    // of a part whose keys' scores are all -inf nothing; a NaN in l stays
    return m == -INFINITY && l == 0.f ? 0.f : ex2_approx(m == top ? 0.f : m - top);
}
__device__ __forceinline__ float shared_of(uint32_t addr, int rank) {  // of a CTA of the cluster
    float x;
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(there) : "memory");
    return x;
}

template <int D, int R, bool AHEAD, int CTAS>
__global__ void __launch_bounds__(32 * kWarps, CTAS) cross_few_kernel(const CrossArgs a, const uint4* q, const uint4* k, const uint4* v) {
    constexpr int kLanes = D / 8, kKeys = 32 / kLanes, kRow = D + 2;  // a state: D columns, m, l
    __shared__ float states[kWarps][R][kRow], joined[R][kRow], own_lse[R];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, grp = lane / kLanes, j = lane % kLanes;
    const int rank = static_cast<int>(blockIdx.x) & ((1 << a.cluster) - 1), item = static_cast<int>(blockIdx.x) >> a.cluster;
    const int batch = item / a.H_kv, h = item - batch * a.H_kv;
    const TileRows T = tile_rows(a, batch, 0);
    griddep_wait();
    griddep_launch_dependents();
    const int len = cross_length(a, batch);
    const int lo = static_cast<int>(static_cast<long long>(len) * rank >> a.cluster);
    const int hi = static_cast<int>(static_cast<long long>(len) * (rank + 1) >> a.cluster);
    float2 qf[R][4], acc[R][4];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint4 x = r < T.rows ? q[global_row(a, T, h, r) * kLanes + j] : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            qf[r][e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
            acc[r][e] = make_float2(0.f, 0.f);
        }
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    const size_t first = static_cast<size_t>(item) * a.N_kv * kLanes + j;
    constexpr int kStep = kWarps * kKeys * kTogether;
    struct Keys {
        uint4 k[kTogether], v[kTogether];
    };
    auto load = [&](int key0) {
        Keys x;
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            const int key = key0 + u * kKeys;
            const size_t at = first + static_cast<size_t>(key) * kLanes;
            x.k[u] = key < hi ? __ldcs(k + at) : make_uint4(0, 0, 0, 0);
            x.v[u] = key < hi ? __ldcs(v + at) : make_uint4(0, 0, 0, 0);
        }
        return x;
    };
    int key0 = lo + warp * (kKeys * kTogether) + grp;
    Keys now, ahead;
    if (AHEAD) now = load(key0);
    for (; key0 - grp < hi; key0 += kStep) {
        if (AHEAD)
            ahead = load(key0 + kStep);
        else
            now = load(key0);
        const uint4(&kr)[kTogether] = now.k;
        const uint4(&vr)[kTogether] = now.v;
        float s[R][kTogether];
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            const uint32_t w[4] = {kr[u].x, kr[u].y, kr[u].z, kr[u].w};
            float2 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 t = __ffma2_rn(qf[r][3], x[3], __ffma2_rn(qf[r][2], x[2], __ffma2_rn(qf[r][1], x[1], __fmul2_rn(qf[r][0], x[0]))));
                s[r][u] = t.x + t.y;
            }
        }
#pragma unroll
        for (int off = 1; off < kLanes; off <<= 1)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < kTogether; ++u) s[r][u] += __shfl_xor_sync(0xffffffffu, s[r][u], off);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = m[r];
#pragma unroll
            for (int u = 0; u < kTogether; ++u) {
                s[r][u] = key0 + u * kKeys < hi ? s[r][u] * a.c_log2 : -INFINITY;
                top = fmaxf(top, s[r][u]);
            }
            const float ref = top == -INFINITY ? 0.f : top, keep = ex2_approx(m[r] - ref);
            m[r] = top;
            l[r] *= keep;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][e] = __fmul2_rn(acc[r][e], make_float2(keep, keep));
#pragma unroll
            for (int u = 0; u < kTogether; ++u) {
                s[r][u] = ex2_approx(s[r][u] - ref);
                l[r] += s[r][u];
            }
        }
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            const uint32_t w[4] = {vr[u].x, vr[u].y, vr[u].z, vr[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r][e] = __ffma2_rn(make_float2(s[r][u], s[r][u]), x, acc[r][e]);
            }
        }
        if (AHEAD) now = ahead;
    }
    // the warp's groups
#pragma unroll
    for (int off = kLanes; off < 32; off <<= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float m1 = __shfl_xor_sync(0xffffffffu, m[r], off), l1 = __shfl_xor_sync(0xffffffffu, l[r], off);
            const float top = fmaxf(m[r], m1), w0 = state_weight(m[r], l[r], top), w1 = state_weight(m1, l1, top);
            // (the same order in both groups)
            const bool low = (lane & off) == 0;
            m[r] = top;
            l[r] = low ? fmaf(w1, l1, w0 * l[r]) : fmaf(w0, l[r], w1 * l1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = __shfl_xor_sync(0xffffffffu, acc[r][e].x, off), y = __shfl_xor_sync(0xffffffffu, acc[r][e].y, off);
                acc[r][e].x = low ? fmaf(w1, x, w0 * acc[r][e].x) : fmaf(w0, acc[r][e].x, w1 * x);
                acc[r][e].y = low ? fmaf(w1, y, w0 * acc[r][e].y) : fmaf(w0, acc[r][e].y, w1 * y);
            }
        }
    if (grp == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(&states[warp][r][8 * j + 2 * e]) = acc[r][e];
            if (j == 0) {
                states[warp][r][D] = m[r];
                states[warp][r][D + 1] = l[r];
            }
        }
    }
    // (lse may be written to where this is read)
    if (a.o_own != nullptr && threadIdx.x < T.rows) own_lse[threadIdx.x] = a.lse_own[global_row(a, T, h, threadIdx.x)];
    __syncthreads();
    // A column of a row over `n` states, and their maximum and sum.
    auto join = [&](int n, int r, int col, auto state, float& top, float& sum) {
        top = -INFINITY;
        for (int i = 0; i < n; ++i) top = fmaxf(top, state(i, r, D));
        float x = 0.f;
        sum = 0.f;
        for (int i = 0; i < n; ++i) {
            const float w = state_weight(state(i, r, D), state(i, r, D + 1), top);
            x = fmaf(w, state(i, r, col), x);
            sum = fmaf(w, state(i, r, D + 1), sum);
        }
        return x;
    };
    auto finish = [&](int r, int col, float top, float sum, float x) {
        if (r >= T.rows) return;
        const size_t row = global_row(a, T, h, r);
        if (a.o_own != nullptr) {
            const float own = own_lse[r] * 1.4426950408889634f, l_own = own == -INFINITY ? 0.f : 1.f;
            const float all = fmaxf(top, own), w = state_weight(top, sum, all), w_own = state_weight(own, l_own, all);
            const uint16_t bits = static_cast<const uint16_t*>(a.o_own)[row * D + col];
            x = w * x + (l_own == 0.f ? 0.f : w_own * __uint_as_float(static_cast<uint32_t>(bits) << 16));
            sum = fmaf(w_own, l_own, w * sum);
            top = all;
        }
        const float y = x * row_factor(sum);
        static_cast<uint16_t*>(a.o)[row * D + col] = static_cast<uint16_t>(pack_bf16x2(y, 0.f));
        if (col == 0 && a.lse != nullptr) a.lse[row] = row_lse(top, sum);
    };
    auto of_warp = [&](int i, int r, int c) { return states[i][r][c]; };
    for (int x = threadIdx.x; x < R * D; x += 32 * kWarps) {
        const int r = x / D, col = x % D;
        float top, sum;
        const float y = join(kWarps, r, col, of_warp, top, sum);
        if (a.cluster == 0) {
            finish(r, col, top, sum, y);
        } else {
            joined[r][col] = y;
            if (col == 0) joined[r][D] = top, joined[r][D + 1] = sum;
        }
    }
    if (a.cluster == 0) return;
    cluster_sync();
    if (rank == 0) {
        const uint32_t base = smem_u32(&joined[0][0]);
        auto of_cta = [&](int i, int r, int c) { return shared_of(base + (r * kRow + c) * 4, i); };
        for (int x = threadIdx.x; x < R * D; x += 32 * kWarps) {
            const int r = x / D, col = x % D;
            float top, sum;
            const float y = join(1 << a.cluster, r, col, of_cta, top, sum);
            finish(r, col, top, sum, y);
        }
    }
    cluster_sync();  // rank 0 has read the others' shared memory
}

template <int D, int R, bool AHEAD, int CTAS>
cudaError_t launch(const CrossArgs& a, const void* q, const void* k, const void* v, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B_kv * a.H_kv) << a.cluster);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {1u << a.cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, cross_few_kernel<D, R, AHEAD, CTAS>, a, static_cast<const uint4*>(q), static_cast<const uint4*>(k),
                              static_cast<const uint4*>(v));
}

}  // namespace

cudaError_t launch_cross_few(const CrossArgs& a, int d, const void* q, const void* k, const void* v, cudaStream_t s) {
    const int rows = a.R * a.share;
    if (a.N_kv > kFewShort) {
        const bool many = (static_cast<long long>(a.B_kv * a.H_kv) << a.cluster) > 2 * 152;
        if (rows == 2) return launch<64, 2, true, 2>(a, q, k, v, s);
        if (d == 64) return many ? launch<64, 1, true, 3>(a, q, k, v, s) : launch<64, 1, true, 2>(a, q, k, v, s);
        return many ? launch<128, 1, true, 3>(a, q, k, v, s) : launch<128, 1, true, 2>(a, q, k, v, s);
    }
    if (rows > 2) return d == 64 ? launch<64, 4, false, 2>(a, q, k, v, s) : launch<128, 4, false, 2>(a, q, k, v, s);
    if (rows == 2) return d == 64 ? launch<64, 2, false, 3>(a, q, k, v, s) : launch<128, 2, false, 3>(a, q, k, v, s);
    return d == 64 ? launch<64, 1, false, 4>(a, q, k, v, s) : launch<128, 1, false, 4>(a, q, k, v, s);
}

}  // namespace fa
