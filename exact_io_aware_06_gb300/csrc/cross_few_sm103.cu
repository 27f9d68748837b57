// cross_few_sm103.cu -- attention of a few rows of queries (single tokens) to another sequence's keys.
//
// With up to four rows to a K/V head in a batch a tile of 128 is nearly empty, and what a call costs is a tile's way
// through the tensor core: 2.9 us for every two blocks of keys, where their bytes take 1.  Here the keys stream through
// registers: D / 8 lanes hold a key's 16 bytes of V each and add up p V for every row.  Up to two rows take their
// scores in the same way, from K's 16 bytes, and a lane group keeps a running maximum and sum of its own; more take
// the scores of 16 keys from small matrix products (64 x 32 / 8 heads on 100 keys at d = 128 14.2 -> 11.1 us).  The
// states of a warp's groups, of a CTA's eight warps and of the up to eight CTAs of a cluster that share a K/V head are
// joined in a fixed order.  Sums, statistics, P and O are float32 up to the result.
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
constexpr int kShort = 128;   // keys, up to which there are no loads ahead

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

__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
    float2 acc[R][4];
    float m[R], l[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][e] = make_float2(0.f, 0.f);
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    const size_t first = static_cast<size_t>(item) * a.N_kv * kLanes;
    if constexpr (R <= 2) {
        float2 qf[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint4 x = r < T.rows ? q[global_row(a, T, h, r) * kLanes + j] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) qf[r][e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
        }
        constexpr int kStep = kWarps * kKeys * kTogether;
        struct Keys {
            uint4 k[kTogether], v[kTogether];
        };
        auto load = [&](int key0) {
            Keys x;
#pragma unroll
            for (int u = 0; u < kTogether; ++u) {
                const int key = key0 + u * kKeys;
                const size_t at = first + static_cast<size_t>(key) * kLanes + j;
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
    } else {
        // Scores of 16 keys and eight rows by matrix fragments straight from memory: the order of d in a product is
        // free, so that a lane's 16 neighbouring bytes serve two products.  Lane (g, t) has the scores of keys g and
        // g + 8 with rows 2 t and 2 t + 1; the lanes that hold V's columns fetch their key's from there.
        constexpr int kC = D / 32, kLoads = 16 / kKeys, kStep = 16 * kWarps;
        const int g = lane / 4, t = lane % 4;
        uint4 qb[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c)
            qb[c] = g < T.rows ? q[global_row(a, T, h, g) * kLanes + 4 * c + t] : make_uint4(0, 0, 0, 0);
        float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};  // of rows 2 t, 2 t + 1
        for (int key0 = lo + 16 * warp; key0 < hi; key0 += kStep) {
            uint4 kr[2][kC], vr[kLoads];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const int key = key0 + g + 8 * i;
                    kr[i][c] = key < hi ? __ldcs(k + first + static_cast<size_t>(key) * kLanes + 4 * c + t) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const int key = key0 + u * kKeys + grp;
                vr[u] = key < hi ? __ldcs(v + first + static_cast<size_t>(key) * kLanes + j) : make_uint4(0, 0, 0, 0);
            }
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                mma_16x8(s, kr[0][c].x, kr[1][c].x, kr[0][c].y, kr[1][c].y, qb[c].x, qb[c].y);
                mma_16x8(s, kr[0][c].z, kr[1][c].z, kr[0][c].w, kr[1][c].w, qb[c].z, qb[c].w);
            }
            float keep[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s[i] = key0 + g < hi ? s[i] * a.c_log2 : -INFINITY;
                s[2 + i] = key0 + g + 8 < hi ? s[2 + i] * a.c_log2 : -INFINITY;
                float mx = fmaxf(s[i], s[2 + i]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                mx = fmaxf(mx, top[i]);
                const float ref = mx == -INFINITY ? 0.f : mx;
                keep[i] = ex2_approx(top[i] - ref);
                top[i] = mx;
                s[i] = ex2_approx(s[i] - ref);
                s[2 + i] = ex2_approx(s[2 + i] - ref);
                sum[i] = fmaf(sum[i], keep[i], s[i] + s[2 + i]);
            }
            if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = __shfl_sync(0xffffffffu, keep[r % 2], r / 2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][e] = __fmul2_rn(acc[r][e], make_float2(f, f));
                }
            }
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const uint32_t w[4] = {vr[u].x, vr[u].y, vr[u].z, vr[u].w};
                float2 x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
                const int from = (u * kKeys + grp) % 8 * 4;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float p = __shfl_sync(0xffffffffu, s[u * kKeys / 8 * 2 + r % 2], from + r / 2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][e] = __ffma2_rn(make_float2(p, p), x[e], acc[r][e]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
#pragma unroll
        for (int r = 0; r < R; ++r) {  // the warp's sum once, in its first group
            m[r] = __shfl_sync(0xffffffffu, top[r % 2], r / 2);
            const float x = __shfl_sync(0xffffffffu, sum[r % 2], r / 2);
            l[r] = grp == 0 ? x : 0.f;
        }
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
    // A column of a row over `n` states, and their maximum and sum.  (Every thread works out the weights; a stage
    // of its own for them made one token 4.7 -> 5.4 us.)
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
    if (rows > 2 || rows * d > 128) return d == 64 ? launch<64, 4, false, 2>(a, q, k, v, s) : launch<128, 4, false, 2>(a, q, k, v, s);
    if (a.N_kv > kShort) {
        const bool many = (static_cast<long long>(a.B_kv * a.H_kv) << a.cluster) > 2 * 152;
        if (rows == 2) return launch<64, 2, true, 2>(a, q, k, v, s);
        if (d == 64) return many ? launch<64, 1, true, 3>(a, q, k, v, s) : launch<64, 1, true, 2>(a, q, k, v, s);
        return many ? launch<128, 1, true, 3>(a, q, k, v, s) : launch<128, 1, true, 2>(a, q, k, v, s);
    }
    if (rows == 2) return launch<64, 2, false, 3>(a, q, k, v, s);
    return d == 64 ? launch<64, 1, false, 4>(a, q, k, v, s) : launch<128, 1, false, 4>(a, q, k, v, s);
}

}  // namespace fa
