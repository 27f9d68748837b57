// qk_norm_rope.cu -- from a layer's projections to the attention call's operands, in one
// pass: the norm of every query and key head, its rotation by position, and the change of
// layout from [B][N][H + 2 H_kv][d] (as a projection writes) to [B][H][N][d] (as the
// attention kernels read).  And the gradient of all three.
//
// For a head row x, weights w, pair frequencies f_p and position t:
//     r = (mean(x^2) + eps)^(-1/2),   y = r x w,
//     (a, b)_p -> (a cos t f_p - b sin t f_p,  b cos t f_p + a sin t f_p).
// Backward, with g the incoming gradient turned back by the same angles:
//     dw = sum over rows of g r x,    dx = r (w g - r^2 x mean(w g x)).
// Nothing is kept from the forward: the backward reads x for dw and dx anyway, and r
// follows from it.
//
// Bound by memory: every element is read once and written once.  A row is held by d / 8
// lanes (16 bytes of bf16 each), so a warp works through 32 / (d / 8) heads of one token at
// a time with 512-byte loads, and the sums of a row are shuffles.  The token's angles are
// computed once per warp and serve all of its heads.
//
// Angles: t f_p / (2 pi) turns.  A float product would lose the fraction at far positions
// (t = 10^6: errors of 0.06 rad); a table would be read again by every token.  f_p / (2 pi)
// is held as a 64-bit fraction instead, and t times it modulo 2^64 is an integer product
// that drops whole turns exactly: the error is t 2^-65 turns, plus one float rounding.
#include <atomic>

#include "layer_ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBwdMaxBlocks = 1024;  // partial weight gradients in the workspace

// Eight neighbouring elements of a row, as loaded: 16 bytes of bf16 or 32 of float.
template <bool F32>
struct Raw {
    uint4 u[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw<F32> load8(const void* base, size_t elem, bool valid) {
    Raw<F32> r;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + elem * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) r.u[i] = valid ? __ldcs(p + i) : make_uint4(0, 0, 0, 0);
    return r;
}
template <bool F32>
__device__ __forceinline__ void store8(void* base, size_t elem, const Raw<F32>& r) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + elem * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) p[i] = r.u[i];
}
template <bool F32>
__device__ __forceinline__ void unpack(const Raw<F32>& r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) {
        const uint32_t w[4] = {r.u[i].x, r.u[i].y, r.u[i].z, r.u[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (F32) {
                x[4 * i + j] = __uint_as_float(w[j]);
            } else {
                x[2 * j] = __uint_as_float(w[j] << 16);
                x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    }
}
template <bool F32>
__device__ __forceinline__ Raw<F32> pack(const float (&x)[8]) {
    Raw<F32> r;
    if (F32) {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
            r.u[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
    } else {
        r.u[0] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                            pack_bf16x2(x[6], x[7]));
    }
    return r;
}

// Sum over the LANES lanes that hold a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The rotation of this lane's eight elements: x[e] -> x[e] c[e] + partner(x[e]) s[e], the
// partner being the other element of e's pair.  Neighbouring pairs (INTER): in this lane;
// halves (e, e + rot / 2): in lane `mate`, rot / 2 being a multiple of 8.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&x)[8], const float (&c)[8], const float (&s)[8], int mate) {
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = INTER ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], mate);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], c[e], o[e] * s[e]);
}

// The factors of this lane's eight elements at position t; `tab` is the warp's own.
template <int D, bool INTER>
__device__ __forceinline__ void token_angles(const NormRopeArgs& a, int t, float2* tab, int lane, float (&c)[8],
                                             float (&s)[8], int& mate) {
    constexpr int kLanes = D / 8;
    const int half = a.rot / 2, j = lane % kLanes, e0 = 8 * j;
    __syncwarp();  // the last token's factors have been read
    for (int p = lane; p < half; p += 32) {
        // signed fraction of a turn, in half turns: [-1, 1)
        const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(t)) * a.freq.f[p];
        const float h = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
        float sn, cs;
        sincospif(h, &sn, &cs);
        tab[p] = make_float2(cs, sn);
    }
    __syncwarp();
    mate = lane;
    if (!INTER && e0 < a.rot) mate = e0 < half ? lane + half / 8 : lane - half / 8;
    const bool turned = e0 < a.rot;  // rot is a multiple of 16: all eight elements, or none
    const bool first = e0 < half;
    const float2* f = tab + (INTER ? e0 / 2 : first ? e0 : e0 - half);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 v = turned ? f[INTER ? e / 2 : e] : make_float2(1.f, 0.f);
        c[e] = v.x;
        s[e] = (INTER ? (e & 1) == 0 : first) ? -v.y : v.y;
    }
}

// A warp's work: passes [p0, p1) of a token, a pass being 32 / (D / 8) neighbouring heads of
// Q, K or V.  Items count chunks of `per` passes, all tokens of a chunk together.
struct Split {
    int first[4];     // first pass of Q, K, V, and the end
    int per;          // passes per item
    int chunks;       // items per token
    Div by_tokens, by_n;
};

// A warp's place in its work: some passes of a token, from `pa` on.
struct Place {
    uint32_t it, tk, b;
    int n, pa, p1, pos;
    bool fresh;  // the first passes of the token
};
__device__ __forceinline__ Place place_at(const NormRopeArgs& a, const Split& sp, uint32_t it, uint32_t items) {
    Place p;
    p.it = it;
    p.fresh = true;
    if (it < items) {
        const uint32_t chunk = sp.by_tokens.of(it);
        p.tk = it - chunk * a.tokens;
        p.pa = static_cast<int>(chunk) * sp.per;
        p.p1 = min(p.pa + sp.per, sp.first[3]);
        p.b = sp.by_n.of(p.tk);
        p.n = static_cast<int>(p.tk - p.b * sp.by_n.d);
        p.pos = a.pos ? __ldg(a.pos + p.tk) : p.n;
    }
    return p;
}
// Pass p: 0, 1 or 2 for Q, K or V, and this lane's head there.
struct Pass {
    int seg, h, heads, before;
};
template <int HEADS>
__device__ __forceinline__ Pass pass_at(const NormRopeArgs& a, const Split& sp, int p, int grp) {
    Pass x;
    x.seg = (p >= sp.first[1]) + (p >= sp.first[2]);
    const int first = x.seg == 0 ? 0 : x.seg == 1 ? sp.first[1] : sp.first[2];
    x.h = (p - first) * HEADS + grp;
    x.heads = x.seg == 0 ? a.heads[0] : a.heads[1];
    x.before = x.seg == 0 ? 0 : x.seg == 1 ? a.heads[0] : a.heads[0] + a.heads[1];
    return x;
}

// The loads of the next passes (of this token or the warp's next one) are in flight while
// these are worked on: a warp that waited for each batch reached 52% of the copy rate.
template <int D, bool F32, bool INTER>
__global__ void __launch_bounds__(kThreads, 2)
    qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Split sp) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    constexpr int kAhead = F32 ? 2 : 4;  // passes of a batch
    __shared__ float2 tab[kWarps][D / 2];
    __shared__ __align__(16) float w[2][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int grp = lane / kLanes, e0 = 8 * (lane % kLanes);
    const int all_heads = a.heads[0] + 2 * a.heads[1];
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t items = a.tokens * sp.chunks, step = gridDim.x * kWarps;
    auto load = [&](const Place& at, Raw<F32>(&raw)[kAhead]) {
        const size_t in0 = static_cast<size_t>(at.tk) * all_heads * D + e0;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const Pass x = pass_at<kHeads>(a, sp, at.pa + u, grp);
            raw[u] = load8<F32>(a.qkv, in0 + static_cast<size_t>(x.before + x.h) * D, at.pa + u < at.p1 && x.h < x.heads);
        }
    };
    Place at = place_at(a, sp, blockIdx.x * kWarps + warp, items);
    Raw<F32> raw[kAhead];
    if (at.it < items) load(at, raw);
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        const float* src = x < D ? a.weight[0] : a.weight[1];
        w[x / D][x % D] = src ? src[x % D] : 1.f;
    }
    __syncthreads();

    float c[8], s[8];
    int mate = lane;
    while (at.it < items) {
        Place next = at;
        next.pa += kAhead;
        next.fresh = false;
        if (next.pa >= at.p1) next = place_at(a, sp, at.it + step, items);
        Raw<F32> ahead[kAhead];
        if (next.it < items) load(next, ahead);
        if (at.fresh && at.pa < sp.first[2]) token_angles<D, INTER>(a, at.pos, tab[warp], lane, c, s, mate);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (at.pa + u >= at.p1) break;
            const Pass ps = pass_at<kHeads>(a, sp, at.pa + u, grp);
            if (ps.seg < 2) {
                float x[8];
                unpack<F32>(raw[u], x);
                float sq = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
                const float r = rsqrtf(row_sum<kLanes>(sq) * (1.f / D) + a.eps);
                const float4* w4 = reinterpret_cast<const float4*>(&w[ps.seg][e0]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 v = w4[i];
                    x[4 * i] *= r * v.x;
                    x[4 * i + 1] *= r * v.y;
                    x[4 * i + 2] *= r * v.z;
                    x[4 * i + 3] *= r * v.w;
                }
                if (a.rot) rotate<INTER>(x, c, s, mate);
                raw[u] = pack<F32>(x);
            }
            if (ps.h < ps.heads)
                store8<F32>(ps.seg == 0 ? a.out[0] : ps.seg == 1 ? a.out[1] : a.out[2],
                            ((static_cast<size_t>(at.b) * ps.heads + ps.h) * a.N + at.n) * D + e0, raw[u]);
        }
        at = next;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) raw[u] = ahead[u];
    }
}

// Gradient.  Each lane keeps its eight elements' sums of dw over all of the warp's rows; the
// block's warps are then added in order and written as one partial row per block, and
// dweight_sum_kernel adds the blocks in order: no atomics, the same bits every time.
template <int D, bool F32, bool INTER>
__global__ void __launch_bounds__(kThreads, 2)
    qk_norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Split sp) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
    constexpr int kAhead = F32 ? 1 : 2;
    __shared__ float2 tab[kWarps][D / 2];
    __shared__ __align__(16) float w[2][D];
    __shared__ float sums[kWarps][2][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int grp = lane / kLanes, e0 = 8 * (lane % kLanes);
    const int all_heads = a.heads[0] + 2 * a.heads[1];
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t items = a.tokens * sp.chunks, step = gridDim.x * kWarps;
    auto load = [&](const Place& at, Raw<F32>(&rx)[kAhead], Raw<F32>(&rg)[kAhead]) {
        const size_t in0 = static_cast<size_t>(at.tk) * all_heads * D + e0;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const Pass x = pass_at<kHeads>(a, sp, at.pa + u, grp);
            const bool valid = at.pa + u < at.p1 && x.h < x.heads;
            rx[u] = load8<F32>(a.qkv, in0 + static_cast<size_t>(x.before + x.h) * D, valid && x.seg < 2);
            rg[u] = load8<F32>(x.seg == 0 ? a.grad[0] : x.seg == 1 ? a.grad[1] : a.grad[2],
                               ((static_cast<size_t>(at.b) * x.heads + x.h) * a.N + at.n) * D + e0, valid);
        }
    };
    Place at = place_at(a, sp, blockIdx.x * kWarps + warp, items);
    Raw<F32> rx[kAhead], rg[kAhead];
    if (at.it < items) load(at, rx, rg);
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        const float* src = x < D ? a.weight[0] : a.weight[1];
        w[x / D][x % D] = src ? src[x % D] : 1.f;
    }
    __syncthreads();

    float c[8], s[8], dw[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.f;
    int mate = lane;
    while (at.it < items) {
        Place next = at;
        next.pa += kAhead;
        next.fresh = false;
        if (next.pa >= at.p1) next = place_at(a, sp, at.it + step, items);
        Raw<F32> nx[kAhead], ng[kAhead];
        if (next.it < items) load(next, nx, ng);
        if (at.fresh && at.pa < sp.first[2]) {
            // turned back: the opposite angle
            token_angles<D, INTER>(a, at.pos, tab[warp], lane, c, s, mate);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = -s[e];
        }
        const size_t in0 = static_cast<size_t>(at.tk) * all_heads * D + e0;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (at.pa + u >= at.p1) break;
            const Pass ps = pass_at<kHeads>(a, sp, at.pa + u, grp);
            if (ps.seg < 2) {
                float x[8], g[8], wg[8];
                unpack<F32>(rx[u], x);
                unpack<F32>(rg[u], g);
                if (a.rot) rotate<INTER>(g, c, s, mate);
                const float4* w4 = reinterpret_cast<const float4*>(&w[ps.seg][e0]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 v = w4[i];
                    wg[4 * i] = v.x * g[4 * i];
                    wg[4 * i + 1] = v.y * g[4 * i + 1];
                    wg[4 * i + 2] = v.z * g[4 * i + 2];
                    wg[4 * i + 3] = v.w * g[4 * i + 3];
                }
                float sq = 0.f, dot = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sq = fmaf(x[e], x[e], sq);
                    dot = fmaf(wg[e], x[e], dot);
                }
                const float r = rsqrtf(row_sum<kLanes>(sq) * (1.f / D) + a.eps);
                const float m = row_sum<kLanes>(dot) * (1.f / D) * r * r;
                // rows of heads past the end are zeros: they add nothing
                if (ps.seg == 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[0][e] = fmaf(g[e], r * x[e], dw[0][e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dw[1][e] = fmaf(g[e], r * x[e], dw[1][e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = r * fmaf(-m, x[e], wg[e]);
                rg[u] = pack<F32>(x);
            }
            if (ps.h < ps.heads) store8<F32>(a.dqkv, in0 + static_cast<size_t>(ps.before + ps.h) * D, rg[u]);
        }
        at = next;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            rx[u] = nx[u];
            rg[u] = ng[u];
        }
    }
    if (a.part == nullptr) return;
    // lanes that hold the same elements of other heads, then the block's warps
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = dw[i][e];
#pragma unroll
            for (int off = kLanes; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (grp == 0) sums[warp][i][e0 + e] = v;
        }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += sums[k][x / D][x % D];
        a.part[static_cast<size_t>(blockIdx.x) * 2 * D + x] = v;
    }
}

// Sum of `rows` partial rows of 2 D values: a block owns 8 columns, 32 threads each.
template <int D>
__global__ void __launch_bounds__(256)
    dweight_sum_kernel(const float* __restrict__ part, int rows, float* dq, float* dk) {
    __shared__ float sums[32][9];
    griddep_wait();
    const int col = threadIdx.x % 8, k = threadIdx.x / 8;
    const int x = blockIdx.x * 8 + col;
    float v = 0.f;
    for (int r = k; r < rows; r += 32) v += part[static_cast<size_t>(r) * 2 * D + x];
    sums[k][col] = v;
    __syncthreads();
    if (k == 0) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) v += sums[i][col];
        float* dst = x < D ? dq : dk;
        if (dst != nullptr) dst[x % D] = v;
    }
}

// Passes of Q, K and V, and how many a warp takes: all of a token's where there are tokens
// enough to fill the GPU (the angles are then computed once per token), fewer where there
// are not (one token of 40 heads: a warp per pass).
Split split_passes(const NormRopeArgs& a, int d, int sms) {
    const int per_pass = 256 / d;  // heads of one pass
    Split sp;
    sp.first[0] = 0;
    for (int i = 0; i < 3; ++i) sp.first[i + 1] = sp.first[i] + (a.heads[i] + per_pass - 1) / per_pass;
    const long long passes = static_cast<long long>(a.tokens) * sp.first[3];
    const long long target = static_cast<long long>(sms) * 32;
    const long long per = (passes + target - 1) / target;
    sp.per = static_cast<int>(per < sp.first[3] ? per : sp.first[3]);
    sp.chunks = (sp.first[3] + sp.per - 1) / sp.per;
    sp.by_tokens = make_div(a.tokens);
    sp.by_n = make_div(a.N);
    return sp;
}

// CTAs of a kernel that are resident together on the current device, asked once per device.
template <typename K>
cudaError_t resident_ctas(K kernel, std::atomic<int> (&known)[64], int* sms, int* ctas) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    *ctas = dev < 64 ? known[dev].load() : 0;
    if (*ctas == 0) {
        int per_sm = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, 0);
        if (e != cudaSuccess) return e;
        *ctas = *sms * (per_sm < 1 ? 1 : per_sm);
        if (dev < 64) known[dev].store(*ctas);
    }
    return cudaSuccess;
}

template <int D, bool F32, bool INTER>
cudaError_t launch_fwd(const NormRopeArgs& a, cudaStream_t s) {
    static std::atomic<int> known[64];
    int sms = 0, cap = 0;
    const cudaError_t e = resident_ctas(qk_norm_rope_kernel<D, F32, INTER>, known, &sms, &cap);
    if (e != cudaSuccess) return e;
    const Split sp = split_passes(a, D, sms);
    const long long blocks = (static_cast<long long>(a.tokens) * sp.chunks + kWarps - 1) / kWarps;
    return launch_pdl(qk_norm_rope_kernel<D, F32, INTER>, dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)),
                      dim3(kThreads), 0, s, a, sp);
}

template <int D, bool F32, bool INTER>
cudaError_t launch_bwd(NormRopeArgs a, float* const (&dweight)[2], cudaStream_t s) {
    static std::atomic<int> known[64];
    int sms = 0, cap = 0;
    const cudaError_t e = resident_ctas(qk_norm_rope_bwd_kernel<D, F32, INTER>, known, &sms, &cap);
    if (e != cudaSuccess) return e;
    const Split sp = split_passes(a, D, sms);
    const bool want = dweight[0] != nullptr || dweight[1] != nullptr;
    if (!want) a.part = nullptr;
    const long long blocks = (static_cast<long long>(a.tokens) * sp.chunks + kWarps - 1) / kWarps;
    if (cap > kBwdMaxBlocks) cap = kBwdMaxBlocks;
    const int grid = static_cast<int>(blocks < cap ? blocks : cap);
    const cudaError_t e2 = launch_pdl(qk_norm_rope_bwd_kernel<D, F32, INTER>, dim3(grid), dim3(kThreads), 0, s, a, sp);
    if (e2 != cudaSuccess || !want) return e2;
    return launch_pdl(dweight_sum_kernel<D>, dim3(2 * D / 8), dim3(256), 0, s, a.part, grid, dweight[0],
                      dweight[1]);
}

}  // namespace

size_t qk_norm_rope_bwd_workspace_bytes(int d) {
    return static_cast<size_t>(kBwdMaxBlocks) * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int d, int f32, int interleaved, cudaStream_t s) {
    if (d == 64) {
        if (f32) return interleaved ? launch_fwd<64, true, true>(a, s) : launch_fwd<64, true, false>(a, s);
        return interleaved ? launch_fwd<64, false, true>(a, s) : launch_fwd<64, false, false>(a, s);
    }
    if (f32) return interleaved ? launch_fwd<128, true, true>(a, s) : launch_fwd<128, true, false>(a, s);
    return interleaved ? launch_fwd<128, false, true>(a, s) : launch_fwd<128, false, false>(a, s);
}

cudaError_t launch_qk_norm_rope_bwd(const NormRopeArgs& a, float* const (&dweight)[2], int d, int f32,
                                    int interleaved, cudaStream_t s) {
    if (d == 64) {
        if (f32)
            return interleaved ? launch_bwd<64, true, true>(a, dweight, s)
                               : launch_bwd<64, true, false>(a, dweight, s);
        return interleaved ? launch_bwd<64, false, true>(a, dweight, s)
                           : launch_bwd<64, false, false>(a, dweight, s);
    }
    if (f32)
        return interleaved ? launch_bwd<128, true, true>(a, dweight, s)
                           : launch_bwd<128, true, false>(a, dweight, s);
    return interleaved ? launch_bwd<128, false, true>(a, dweight, s)
                       : launch_bwd<128, false, false>(a, dweight, s);
}

}  // namespace fa
