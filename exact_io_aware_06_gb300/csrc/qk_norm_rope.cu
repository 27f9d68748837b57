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
// lanes, so a warp works through 32 / (d / 8) heads of one token at a time (512 bytes of
// bf16), and the sums of a row are shuffles.  The token's angles are computed once per warp
// and serve all of its heads.  At 43 cycles of an SM per pass (read and write at the copy
// rate) the instructions count too: pairs within a lane, packed float32 arithmetic.
//
// Positions may have several axes (time, height and width of a video's tokens): pair p then turns by
// t[axis_p] f_p, and a lane keeps the axes of its pairs and fetches its own positions a batch ahead.
//
// Angles: t f_p / (2 pi) turns.  A float product would lose the fraction at far positions
// (t = 10^6: errors of 0.06 rad); a table would be read again by every token.  f_p / (2 pi)
// is held as a 64-bit fraction instead, off by under 2^-62 (rope_turns.h), and t times it modulo
// 2^64 is an integer product that drops whole turns exactly.  Of the product the upper 32 bits are
// taken and rounded to a float: at |t| = 2^31 the angle is off by 2^-31 + 2^-32 + 2^-26 turns.
#include <atomic>
#include <type_traits>

#include "layer_ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBwdMaxBlocks = 1024;  // partial weight gradients in the workspace

// A lane's eight elements of a row are two groups of four, a[0..3] and b[0..3], chosen so that
// both elements of every pair are in one lane: with halves (p, p + rot / 2), groups j and
// j + rot / 8 for the lanes below rot / 8, and neighbouring groups of the unturned rest for the
// others; with neighbours (2 p, 2 p + 1), groups 2 j and 2 j + 1.  (Sixteen neighbouring bytes
// a lane and shuffles between the halves: eight more instructions a row where 60 do the work.)
// Pair i of a lane is (a[i], b[i]) for halves, and (a0, a1), (a2, a3), (b0, b1), (b2, b3) for
// neighbours.
template <bool F32>
struct Raw {
    uint32_t u[F32 ? 8 : 4];
};

template <bool F32>
__device__ __forceinline__ Raw<F32> load8(const char* pa, const char* pb, bool valid) {
    Raw<F32> r;
    if constexpr (F32) {
        const uint4 a = valid ? __ldcs(reinterpret_cast<const uint4*>(pa)) : make_uint4(0, 0, 0, 0);
        const uint4 b = valid ? __ldcs(reinterpret_cast<const uint4*>(pb)) : make_uint4(0, 0, 0, 0);
        r.u[0] = a.x, r.u[1] = a.y, r.u[2] = a.z, r.u[3] = a.w;
        r.u[4] = b.x, r.u[5] = b.y, r.u[6] = b.z, r.u[7] = b.w;
    } else {
        const uint2 a = valid ? __ldcs(reinterpret_cast<const uint2*>(pa)) : make_uint2(0, 0);
        const uint2 b = valid ? __ldcs(reinterpret_cast<const uint2*>(pb)) : make_uint2(0, 0);
        r.u[0] = a.x, r.u[1] = a.y, r.u[2] = b.x, r.u[3] = b.y;
    }
    return r;
}
template <bool F32>
__device__ __forceinline__ void store8(char* pa, char* pb, const Raw<F32>& r) {
    if constexpr (F32) {
        *reinterpret_cast<uint4*>(pa) = make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
        *reinterpret_cast<uint4*>(pb) = make_uint4(r.u[4], r.u[5], r.u[6], r.u[7]);
    } else {
        *reinterpret_cast<uint2*>(pa) = make_uint2(r.u[0], r.u[1]);
        *reinterpret_cast<uint2*>(pb) = make_uint2(r.u[2], r.u[3]);
    }
}

// The lane's four pairs as two float2 of first and two of second elements: first[k] holds those
// of pairs 2k, 2k + 1.
struct Quad {
    float2 first[2], second[2];
};
template <bool F32>
__device__ __forceinline__ float elem(const Raw<F32>& r, int i) {
    if constexpr (F32)
        return __uint_as_float(r.u[i]);
    else
        return __uint_as_float((i & 1) ? r.u[i / 2] & 0xFFFF0000u : r.u[i / 2] << 16);
}
template <bool F32, bool INTER>
__device__ __forceinline__ Quad unpack(const Raw<F32>& r) {
    Quad q;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (INTER) {
            q.first[k] = make_float2(elem<F32>(r, 4 * k), elem<F32>(r, 4 * k + 2));
            q.second[k] = make_float2(elem<F32>(r, 4 * k + 1), elem<F32>(r, 4 * k + 3));
        } else {
            q.first[k] = make_float2(elem<F32>(r, 2 * k), elem<F32>(r, 2 * k + 1));
            q.second[k] = make_float2(elem<F32>(r, 4 + 2 * k), elem<F32>(r, 5 + 2 * k));
        }
    }
    return q;
}
template <bool F32, bool INTER>
__device__ __forceinline__ Raw<F32> pack(const Quad& q) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        x[INTER ? 4 * k : 2 * k] = q.first[k].x;
        x[INTER ? 4 * k + 2 : 2 * k + 1] = q.first[k].y;
        x[INTER ? 4 * k + 1 : 4 + 2 * k] = q.second[k].x;
        x[INTER ? 4 * k + 3 : 5 + 2 * k] = q.second[k].y;
    }
    Raw<F32> r;
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) r.u[i] = F32 ? __float_as_uint(x[i]) : pack_bf16x2(x[2 * i], x[2 * i + 1]);
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Sum over the LANES lanes that hold a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
__device__ __forceinline__ float dot(const Quad& a, const Quad& b) {
    const float2 s = fma2(a.second[1], b.second[1],
                          fma2(a.first[1], b.first[1], fma2(a.second[0], b.second[0], mul2(a.first[0], b.first[0]))));
    return s.x + s.y;
}

// First elements of the lane's two groups (see Raw).
template <int D, bool INTER>
__device__ __forceinline__ void lane_groups(int rot, int j, int& ea, int& eb) {
    const int turned = rot / 8;
    if (INTER || j >= turned) {
        ea = INTER ? 8 * j : rot + 8 * (j - turned);
        eb = ea + 4;
    } else {
        ea = 4 * j;
        eb = ea + rot / 2;
    }
}

// cos and sin of the lane's pairs at the token's position (1 and 0 past rot); `tab` is the warp's own.
template <int D, bool INTER, int AXES>
__device__ __forceinline__ void token_angles(const NormRopeArgs& a, const int (&pos)[AXES], float2* tab, int lane,
                                             float2 (&c)[2], float2 (&s)[2]) {
    constexpr int kLanes = D / 8;
    const int half = a.rot / 2, j = lane % kLanes;
    __syncwarp();  // the last token's factors have been read
    for (int p = lane; p < half; p += 32) {
        const int t = AXES == 2 && p >= 32 ? pos[AXES - 1] : pos[0];
        // signed fraction of a turn, in half turns: [-1, 1)
        const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(t)) * a.freq.f[p];
        const float h = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
        float sn, cs;
        sincospif(h, &sn, &cs);
        tab[p] = make_float2(cs, sn);
    }
    __syncwarp();
    const bool turned = j < a.rot / 8;  // four pairs a lane either way
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float2 u = turned ? tab[4 * j + 2 * k] : make_float2(1.f, 0.f);
        const float2 v = turned ? tab[4 * j + 2 * k + 1] : make_float2(1.f, 0.f);
        c[k] = make_float2(u.x, v.x);
        s[k] = make_float2(u.y, v.y);
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

// The axes of the lane's pairs, lane and lane + 32; -1 past rot.
struct LaneAxes {
    int of[2];
    __device__ __forceinline__ LaneAxes(const NormRopeArgs& a, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) of[i] = lane + 32 * i < a.rot / 2 ? a.axis[lane + 32 * i] : -1;
    }
};

// A warp's place in its work: a batch of up to AHEAD passes of one of Q, K, V of a token.  With several
// axes (AXES = 2) the positions are those of the lane's two pairs.
template <int AXES>
struct Place {
    uint32_t it, tk, b;
    int n, pos[AXES];
    int seg, p, p1;     // this batch's first pass, and the item's end
    int count;          // passes of the batch
    bool fresh;         // the item's first batch
};
template <int AHEAD, int AXES>
__device__ __forceinline__ void batch_at(const Split& sp, Place<AXES>& p) {
    p.seg = (p.p >= sp.first[1]) + (p.p >= sp.first[2]);
    const int end = p.seg == 0 ? sp.first[1] : p.seg == 1 ? sp.first[2] : sp.first[3];
    p.count = min(AHEAD, min(end, p.p1) - p.p);
}
template <int AHEAD, int AXES>
__device__ __forceinline__ Place<AXES> place_at(const NormRopeArgs& a, const Split& sp, const LaneAxes& axis,
                                                uint32_t it, uint32_t items) {
    Place<AXES> p;
    p.it = it;
    p.fresh = true;
    if (it < items) {
        const uint32_t chunk = sp.by_tokens.of(it);
        p.tk = it - chunk * a.tokens;
        p.p = static_cast<int>(chunk) * sp.per;
        p.p1 = min(p.p + sp.per, sp.first[3]);
        p.b = sp.by_n.of(p.tk);
        p.n = static_cast<int>(p.tk - p.b * sp.by_n.d);
        if constexpr (AXES == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                p.pos[i] = axis.of[i] < 0 ? 0 : __ldg(a.pos + (static_cast<size_t>(axis.of[i]) * a.tokens + p.tk));
        } else {
            p.pos[0] = a.pos ? __ldg(a.pos + p.tk) : p.n;
        }
        batch_at<AHEAD>(sp, p);
    }
    return p;
}
template <int AHEAD, int AXES>
__device__ __forceinline__ Place<AXES> place_after(const NormRopeArgs& a, const Split& sp, const LaneAxes& axis,
                                                   const Place<AXES>& at, uint32_t step, uint32_t items) {
    if (at.p + at.count >= at.p1) return place_at<AHEAD, AXES>(a, sp, axis, at.it + step, items);
    Place<AXES> p = at;
    p.p += at.count;
    p.fresh = false;
    batch_at<AHEAD>(sp, p);
    return p;
}
// The batch's first head of this lane among Q's, K's or V's; their number; heads before them.
template <int HEADS, int AXES>
__device__ __forceinline__ void heads_of(const NormRopeArgs& a, const Split& sp, const Place<AXES>& p, int grp, int& h,
                                         int& heads, int& before) {
    const int first = p.seg == 0 ? 0 : p.seg == 1 ? sp.first[1] : sp.first[2];
    h = (p.p - first) * HEADS + grp;
    heads = p.seg == 0 ? a.heads[0] : a.heads[1];
    before = p.seg == 0 ? 0 : p.seg == 1 ? a.heads[0] : a.heads[0] + a.heads[1];
}

// The loads of the next batch (of this token or the warp's next one) are in flight while one
// is worked on: 4 KB a warp, 64 KB an SM.  Measured at B1 N16384 H32 H_kv8 d128 (403 MB):
// batches of 8 passes and 4 blocks an SM 68.7 us (5.9 TB/s, 87% of the copy rate), 4 and 5
// 69.8, 4 and 4 71.3, 2 and 5 83; waiting for each batch 113.  In float32 132 us (805 MB, 6.1 TB/s).  And weights are multiplied into a
// token's cosines and sines once for Q's heads and once for K's.
template <int D, bool F32, bool INTER, int AXES>
__global__ void __launch_bounds__(kThreads, 4)
    qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Split sp) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes, kElem = F32 ? 4 : 2;
    constexpr int kAhead = F32 ? 2 : 8;
    constexpr int kPass = kHeads * D * kElem;  // bytes of a pass in qkv
    __shared__ float2 tab[kWarps][D / 2];
    __shared__ __align__(16) float w[2][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int grp = lane / kLanes;
    int ea, eb;
    lane_groups<D, INTER>(a.rot, lane % kLanes, ea, eb);
    const int gap = (eb - ea) * kElem;
    const int all_heads = a.heads[0] + 2 * a.heads[1];
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t items = a.tokens * sp.chunks, step = gridDim.x * kWarps;
    auto load = [&](const Place<AXES>& at, Raw<F32>(&raw)[kAhead]) {
        int h, heads, before;
        heads_of<kHeads>(a, sp, at, grp, h, heads, before);
        const char* src = static_cast<const char*>(a.qkv) +
                          ((static_cast<size_t>(at.tk) * all_heads + before + h) * D + ea) * kElem;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            raw[u] = load8<F32>(src + u * kPass, src + gap + u * kPass, u < at.count && h + u * kHeads < heads);
    };
    const LaneAxes axis(a, lane);
    Place<AXES> at = place_at<kAhead, AXES>(a, sp, axis, blockIdx.x * kWarps + warp, items);
    Raw<F32> raw[kAhead];
    if (at.it < items) load(at, raw);
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        const float* src = x < D ? a.weight[0] : a.weight[1];
        w[x / D][x % D] = src ? src[x % D] : 1.f;
    }
    __syncthreads();

    float2 c[2], s[2];                          // the token's, of this lane's pairs
    float2 cf[2], cs[2], sf[2], ss[2];          // times the weights of first and second elements
    while (at.it < items) {
        const Place<AXES> next = place_after<kAhead>(a, sp, axis, at, step, items);
        Raw<F32> ahead[kAhead];
        if (next.it < items) load(next, ahead);
        int h, heads, before;
        heads_of<kHeads>(a, sp, at, grp, h, heads, before);
        if (at.seg < 2 && (at.fresh || at.p == sp.first[1])) {
            if (at.fresh) token_angles<D, INTER, AXES>(a, at.pos, tab[warp], lane, c, s);
            const float4 wa = *reinterpret_cast<const float4*>(&w[at.seg][ea]);
            const float4 wb = *reinterpret_cast<const float4*>(&w[at.seg][eb]);
            const float2 wf[2] = {INTER ? make_float2(wa.x, wa.z) : make_float2(wa.x, wa.y),
                                  INTER ? make_float2(wb.x, wb.z) : make_float2(wa.z, wa.w)};
            const float2 ws[2] = {INTER ? make_float2(wa.y, wa.w) : make_float2(wb.x, wb.y),
                                  INTER ? make_float2(wb.y, wb.w) : make_float2(wb.z, wb.w)};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                cf[k] = mul2(c[k], wf[k]);
                cs[k] = mul2(c[k], ws[k]);
                sf[k] = mul2(s[k], wf[k]);
                ss[k] = neg2(mul2(s[k], ws[k]));
            }
        }
        char* dst = static_cast<char*>(at.seg == 0 ? a.out[0] : at.seg == 1 ? a.out[1] : a.out[2]) +
                    (((static_cast<size_t>(at.b) * heads + h) * a.N + at.n) * D + ea) * kElem;
        const size_t out_pass = static_cast<size_t>(a.N) * kPass;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u >= at.count) break;
            if (at.seg < 2) {
                const Quad x = unpack<F32, INTER>(raw[u]);
                const float2 r = both(rsqrtf(fmaf(row_sum<kLanes>(dot(x, x)), 1.f / D, a.eps)));
                Quad y;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    y.first[k] = mul2(r, fma2(x.first[k], cf[k], mul2(x.second[k], ss[k])));
                    y.second[k] = mul2(r, fma2(x.second[k], cs[k], mul2(x.first[k], sf[k])));
                }
                raw[u] = pack<F32, INTER>(y);
            }
            if (h + u * kHeads < heads) store8<F32>(dst, dst + gap, raw[u]);
            dst += out_pass;
        }
        at = next;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) raw[u] = ahead[u];
    }
}

// Many tokens of few heads: a token a group of D / 8 lanes, all of whose heads it works through, pass by pass, so
// that no lane is idle where heads do not fill a pass of one token, no batch ends with Q's or K's heads, and the
// work for a token (its place, position, cosines and sines, four pairs a lane) is shared by 32 / (D / 8) of them.
// By passes of a token / by rows: 63462 tokens of one head at d = 64 80 / 12.7 us, 67419 of 8 / 2 94 / 36 (5.7 TB/s),
// 42840 of 16 / 1 71 / 44, 16384 of 32 / 8 at d = 128 69.6 / 74: there a pass is full and its results lie closer.
// Gradients: 63462 of one head 103 / 19, 53688 of 4 / 2 at d = 128 113 / 61, 16384 of 32 / 8 102 / 104.
struct Rows {
    int all, per, batch;      // heads of a token, Q's, K's and V's; passes of an item; of a batch of loads
    uint32_t groups, items;   // of 32 / (D / 8) tokens; all groups' first passes, then their next ones
    Div by_groups, by_n;
};
// The lane's four pairs, and its place: a batch of passes of its token.
template <int D, int AXES>
struct LanePairs {
    uint64_t f[4];
    int axis[AXES == 2 ? 4 : 1];
    bool turned;
    __device__ __forceinline__ LanePairs(const NormRopeArgs& a, int j) {
        turned = j < a.rot / 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = turned ? a.freq.f[4 * j + i] : 0;
            if constexpr (AXES == 2) axis[i] = turned ? a.axis[4 * j + i] : 0;
        }
    }
    __device__ __forceinline__ void angles(const int (&pos)[AXES == 2 ? 4 : 1], float2 (&c)[2], float2 (&s)[2]) const {
        float cs[4], sn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // as token_angles
            const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos[AXES == 2 ? i : 0])) * f[i];
            sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &sn[i], &cs[i]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            c[k] = make_float2(cs[2 * k], cs[2 * k + 1]);
            s[k] = make_float2(sn[2 * k], sn[2 * k + 1]);
        }
    }
};
template <int AXES>
struct RowPlace {
    uint32_t it, tk, b;
    int n, p, p1, count;
    int pos[AXES == 2 ? 4 : 1];
    bool there, fresh;
};
template <int D, int AXES>
__device__ __forceinline__ void row_place(const NormRopeArgs& a, const Rows& r, const LanePairs<D, AXES>& pairs, uint32_t it,
                                          int grp, RowPlace<AXES>& p) {
    constexpr int kTokens = 32 / (D / 8);
    const uint32_t chunk = r.by_groups.of(min(it, r.items - 1));
    p.it = it;
    p.p = static_cast<int>(chunk) * r.per;
    p.p1 = min(p.p + r.per, r.all);
    p.count = min(r.batch, p.p1 - p.p);
    p.tk = (it - chunk * r.groups) * kTokens + grp;
    p.fresh = true;
    p.there = it < r.items && p.tk < a.tokens;
    if (!p.there) p.tk = 0;
    p.b = r.by_n.of(p.tk);
    p.n = static_cast<int>(p.tk - p.b * r.by_n.d);
    if constexpr (AXES == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p.pos[i] = pairs.turned ? __ldg(a.pos + (static_cast<size_t>(pairs.axis[i]) * a.tokens + p.tk)) : 0;
    } else {
        p.pos[0] = a.pos ? __ldg(a.pos + p.tk) : p.n;
    }
}
template <int D, int AXES>
__device__ __forceinline__ RowPlace<AXES> row_after(const NormRopeArgs& a, const Rows& r, const LanePairs<D, AXES>& pairs,
                                                    const RowPlace<AXES>& at, uint32_t step, int grp) {
    RowPlace<AXES> p = at;
    if (at.p + at.count >= at.p1) {
        row_place(a, r, pairs, at.it + step, grp, p);
    } else {
        p.p += at.count;
        p.count = min(r.batch, at.p1 - p.p);
        p.fresh = false;
    }
    return p;
}
// The lane's weights of Q (seg = 0) or K.
template <int D, bool INTER>
__device__ __forceinline__ void lane_weights(const float (&w)[2][D], int seg, int ea, int eb, float2 (&wf)[2], float2 (&ws)[2]) {
    const float4 wa = *reinterpret_cast<const float4*>(&w[seg][ea]);
    const float4 wb = *reinterpret_cast<const float4*>(&w[seg][eb]);
    wf[0] = INTER ? make_float2(wa.x, wa.z) : make_float2(wa.x, wa.y);
    wf[1] = INTER ? make_float2(wb.x, wb.z) : make_float2(wa.z, wa.w);
    ws[0] = INTER ? make_float2(wa.y, wa.w) : make_float2(wb.x, wb.y);
    ws[1] = INTER ? make_float2(wb.y, wb.w) : make_float2(wb.z, wb.w);
}
// Where head p of a token (b, n) lies among the tensors [B][heads][N][D] of Q, K and V.
__device__ __forceinline__ size_t head_row(const NormRopeArgs& a, int seg, int p, uint32_t b, int n) {
    const int heads = seg == 0 ? a.heads[0] : a.heads[1];
    const int h = seg == 0 ? p : seg == 1 ? p - a.heads[0] : p - a.heads[0] - a.heads[1];
    return (static_cast<size_t>(b) * heads + h) * a.N + n;
}

template <int D, bool F32, bool INTER, int AXES>
__global__ void __launch_bounds__(kThreads, 4)
    qk_norm_rope_rows_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Rows rows) {
    constexpr int kLanes = D / 8, kElem = F32 ? 4 : 2, kAhead = F32 ? 2 : 8;
    __shared__ __align__(16) float w[2][D];
    const int lane = threadIdx.x % 32, grp = lane / kLanes;
    int ea, eb;
    lane_groups<D, INTER>(a.rot, lane % kLanes, ea, eb);
    const int gap = (eb - ea) * kElem;
    const LanePairs<D, AXES> pairs(a, lane % kLanes);
    griddep_wait();
    griddep_launch_dependents();
    auto load = [&](const RowPlace<AXES>& at, Raw<F32>(&raw)[kAhead]) {
        const char* src = static_cast<const char*>(a.qkv) + ((static_cast<size_t>(at.tk) * rows.all + at.p) * D + ea) * kElem;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            raw[u] = load8<F32>(src + u * D * kElem, src + gap + u * D * kElem, u < at.count && at.there);
    };
    RowPlace<AXES> at;
    row_place(a, rows, pairs, blockIdx.x * kWarps + threadIdx.x / 32, grp, at);
    Raw<F32> raw[kAhead];
    load(at, raw);
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        const float* src = x < D ? a.weight[0] : a.weight[1];
        w[x / D][x % D] = src ? src[x % D] : 1.f;
    }
    __syncthreads();

    float2 c[2], s[2];
    while (at.it < rows.items) {
        const RowPlace<AXES> next = row_after(a, rows, pairs, at, gridDim.x * kWarps, grp);
        Raw<F32> ahead[kAhead];
        load(next, ahead);
        if (at.fresh) pairs.angles(at.pos, c, s);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u >= at.count) break;
            const int p = at.p + u, seg = (p >= a.heads[0]) + (p >= a.heads[0] + a.heads[1]);
            if (seg < 2) {
                float2 wf[2], ws[2];
                lane_weights<D, INTER>(w, seg, ea, eb, wf, ws);
                const Quad x = unpack<F32, INTER>(raw[u]);
                const float2 r = both(rsqrtf(fmaf(row_sum<kLanes>(dot(x, x)), 1.f / D, a.eps)));
                Quad y;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    y.first[k] = mul2(r, fma2(x.first[k], mul2(c[k], wf[k]), mul2(x.second[k], neg2(mul2(s[k], ws[k])))));
                    y.second[k] = mul2(r, fma2(x.second[k], mul2(c[k], ws[k]), mul2(x.first[k], mul2(s[k], wf[k]))));
                }
                raw[u] = pack<F32, INTER>(y);
            }
            char* dst = static_cast<char*>(seg == 0 ? a.out[0] : seg == 1 ? a.out[1] : a.out[2]) +
                        (head_row(a, seg, p, at.b, at.n) * D + ea) * kElem;
            if (at.there) store8<F32>(dst, dst + gap, raw[u]);
        }
        at = next;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) raw[u] = ahead[u];
    }
}

// Gradient of a row x (`there`, or zeros) from its output's; seg = 0 (Q) or 1 (K), whose sums of dw it adds to.
template <int LANES>
__device__ __forceinline__ Quad row_gradient(const Quad& x, const Quad& dy, const float2 (&c)[2], const float2 (&s)[2],
                                             const float2 (&wf)[2], const float2 (&ws)[2], float eps, bool there, int seg,
                                             Quad (&dw)[2]) {
    constexpr int D = 8 * LANES;
    Quad g, wg;
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // turned back: the opposite angle
        g.first[k] = fma2(dy.first[k], c[k], mul2(dy.second[k], s[k]));
        g.second[k] = fma2(dy.second[k], c[k], neg2(mul2(dy.first[k], s[k])));
        wg.first[k] = mul2(g.first[k], wf[k]);
        wg.second[k] = mul2(g.second[k], ws[k]);
    }
    const float sq = fmaf(row_sum<LANES>(dot(x, x)), 1.f / D, eps);
    // rows of heads past the end are zeros: with a finite r (for eps = 0 too) they add nothing
    const float r = there ? rsqrtf(sq) : 0.f;
    const float m = row_sum<LANES>(dot(wg, x)) * (1.f / D) * r * r;
    const float2 r2 = both(r), m2 = both(-m);
    Quad dx;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float2 gf = mul2(g.first[k], r2), gs = mul2(g.second[k], r2);
        if (seg == 0) {
            dw[0].first[k] = fma2(gf, x.first[k], dw[0].first[k]);
            dw[0].second[k] = fma2(gs, x.second[k], dw[0].second[k]);
        } else {
            dw[1].first[k] = fma2(gf, x.first[k], dw[1].first[k]);
            dw[1].second[k] = fma2(gs, x.second[k], dw[1].second[k]);
        }
        dx.first[k] = mul2(r2, fma2(m2, x.first[k], wg.first[k]));
        dx.second[k] = mul2(r2, fma2(m2, x.second[k], wg.second[k]));
    }
    return dx;
}
// The block's sums of dw: over the lanes that hold the same elements of other rows, then over its warps in order.
template <int D, bool INTER>
__device__ __forceinline__ void block_sums(const Quad (&dw)[2], float (&sums)[kWarps][2][D], int ea, int eb, float* part) {
    constexpr int kLanes = D / 8;
    const int warp = threadIdx.x / 32, grp = threadIdx.x % 32 / kLanes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Raw<true> v = pack<true, INTER>(dw[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float t = __uint_as_float(v.u[e]);
#pragma unroll
            for (int off = kLanes; off < 32; off <<= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
            if (grp == 0) sums[warp][i][(e < 4 ? ea : eb - 4) + e] = t;
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += sums[k][x / D][x % D];
        part[static_cast<size_t>(blockIdx.x) * 2 * D + x] = v;
    }
}

// Gradient.  Each lane keeps its eight elements' sums of dw over all of the warp's rows; the
// block's warps are then added in order and written as one partial row per block, and
// dweight_sum_kernel adds the blocks in order: no atomics, the same bits every time.
// Measured at B4 N4096 H32 H_kv8 d128 (570 MB): batches of 4 passes and 3 blocks an SM 101 us
// (5.6 TB/s), 2 and 4 112, 1 and 4 157.
template <int D, bool F32, bool INTER, int AXES>
__global__ void __launch_bounds__(kThreads, 3)
    qk_norm_rope_bwd_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Split sp) {
    constexpr int kLanes = D / 8, kHeads = 32 / kLanes, kElem = F32 ? 4 : 2;
    constexpr int kAhead = F32 ? 2 : 4;
    constexpr int kPass = kHeads * D * kElem;
    __shared__ float2 tab[kWarps][D / 2];
    __shared__ __align__(16) float w[2][D];
    __shared__ float sums[kWarps][2][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int grp = lane / kLanes;
    int ea, eb;
    lane_groups<D, INTER>(a.rot, lane % kLanes, ea, eb);
    const int gap = (eb - ea) * kElem;
    const int all_heads = a.heads[0] + 2 * a.heads[1];
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t items = a.tokens * sp.chunks, step = gridDim.x * kWarps;
    const size_t grad_pass = static_cast<size_t>(a.N) * kPass;
    auto load = [&](const Place<AXES>& at, Raw<F32>(&rx)[kAhead], Raw<F32>(&rg)[kAhead]) {
        int h, heads, before;
        heads_of<kHeads>(a, sp, at, grp, h, heads, before);
        const char* src = static_cast<const char*>(a.qkv) +
                          ((static_cast<size_t>(at.tk) * all_heads + before + h) * D + ea) * kElem;
        const char* grad = static_cast<const char*>(at.seg == 0 ? a.grad[0] : at.seg == 1 ? a.grad[1] : a.grad[2]) +
                           (((static_cast<size_t>(at.b) * heads + h) * a.N + at.n) * D + ea) * kElem;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const bool valid = u < at.count && h + u * kHeads < heads;
            rx[u] = load8<F32>(src + u * kPass, src + gap + u * kPass, valid && at.seg < 2);
            rg[u] = load8<F32>(grad, grad + gap, valid);
            grad += grad_pass;
        }
    };
    const LaneAxes axis(a, lane);
    Place<AXES> at = place_at<kAhead, AXES>(a, sp, axis, blockIdx.x * kWarps + warp, items);
    Raw<F32> rx[kAhead], rg[kAhead];
    if (at.it < items) load(at, rx, rg);
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        const float* src = x < D ? a.weight[0] : a.weight[1];
        w[x / D][x % D] = src ? src[x % D] : 1.f;
    }
    __syncthreads();

    float2 c[2], s[2], wf[2], ws[2];
    Quad dw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) dw[i].first[k] = dw[i].second[k] = make_float2(0.f, 0.f);
    while (at.it < items) {
        const Place<AXES> next = place_after<kAhead>(a, sp, axis, at, step, items);
        Raw<F32> nx[kAhead], ng[kAhead];
        if (next.it < items) load(next, nx, ng);
        int h, heads, before;
        heads_of<kHeads>(a, sp, at, grp, h, heads, before);
        if (at.seg < 2 && (at.fresh || at.p == sp.first[1])) {
            if (at.fresh) token_angles<D, INTER, AXES>(a, at.pos, tab[warp], lane, c, s);
            const float4 wa = *reinterpret_cast<const float4*>(&w[at.seg][ea]);
            const float4 wb = *reinterpret_cast<const float4*>(&w[at.seg][eb]);
            wf[0] = INTER ? make_float2(wa.x, wa.z) : make_float2(wa.x, wa.y);
            wf[1] = INTER ? make_float2(wb.x, wb.z) : make_float2(wa.z, wa.w);
            ws[0] = INTER ? make_float2(wa.y, wa.w) : make_float2(wb.x, wb.y);
            ws[1] = INTER ? make_float2(wb.y, wb.w) : make_float2(wb.z, wb.w);
        }
        char* dst = static_cast<char*>(a.dqkv) +
                    ((static_cast<size_t>(at.tk) * all_heads + before + h) * D + ea) * kElem;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u >= at.count) break;
            const bool there = h + u * kHeads < heads;
            if (at.seg < 2) {
                const Quad x = unpack<F32, INTER>(rx[u]), dy = unpack<F32, INTER>(rg[u]);
                const Quad dx = row_gradient<kLanes>(x, dy, c, s, wf, ws, a.eps, there, at.seg, dw);
                rg[u] = pack<F32, INTER>(dx);
            }
            if (there) store8<F32>(dst + u * kPass, dst + gap + u * kPass, rg[u]);
        }
        at = next;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            rx[u] = nx[u];
            rg[u] = ng[u];
        }
    }
    if (a.part == nullptr) return;
    block_sums<D, INTER>(dw, sums, ea, eb, a.part);
}

template <int D, bool F32, bool INTER, int AXES>
__global__ void __launch_bounds__(kThreads, 3)
    qk_norm_rope_rows_bwd_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Rows rows) {
    constexpr int kLanes = D / 8, kElem = F32 ? 4 : 2, kAhead = F32 ? 2 : 4;
    __shared__ __align__(16) float w[2][D];
    __shared__ float sums[kWarps][2][D];
    const int lane = threadIdx.x % 32, grp = lane / kLanes;
    int ea, eb;
    lane_groups<D, INTER>(a.rot, lane % kLanes, ea, eb);
    const int gap = (eb - ea) * kElem;
    const LanePairs<D, AXES> pairs(a, lane % kLanes);
    griddep_wait();
    griddep_launch_dependents();
    auto load = [&](const RowPlace<AXES>& at, Raw<F32>(&rx)[kAhead], Raw<F32>(&rg)[kAhead]) {
        const char* src = static_cast<const char*>(a.qkv) + ((static_cast<size_t>(at.tk) * rows.all + at.p) * D + ea) * kElem;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int p = at.p + u, seg = (p >= a.heads[0]) + (p >= a.heads[0] + a.heads[1]);
            const bool valid = u < at.count && at.there;
            const char* grad = static_cast<const char*>(seg == 0 ? a.grad[0] : seg == 1 ? a.grad[1] : a.grad[2]) +
                               (head_row(a, seg, p, at.b, at.n) * D + ea) * kElem;
            rx[u] = load8<F32>(src + u * D * kElem, src + gap + u * D * kElem, valid && seg < 2);
            rg[u] = load8<F32>(grad, grad + gap, valid);
        }
    };
    RowPlace<AXES> at;
    row_place(a, rows, pairs, blockIdx.x * kWarps + threadIdx.x / 32, grp, at);
    Raw<F32> rx[kAhead], rg[kAhead];
    load(at, rx, rg);
    for (int x = threadIdx.x; x < 2 * D; x += kThreads) {
        const float* src = x < D ? a.weight[0] : a.weight[1];
        w[x / D][x % D] = src ? src[x % D] : 1.f;
    }
    __syncthreads();

    float2 c[2], s[2];
    Quad dw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) dw[i].first[k] = dw[i].second[k] = make_float2(0.f, 0.f);
    while (at.it < rows.items) {
        const RowPlace<AXES> next = row_after(a, rows, pairs, at, gridDim.x * kWarps, grp);
        Raw<F32> nx[kAhead], ng[kAhead];
        load(next, nx, ng);
        if (at.fresh) pairs.angles(at.pos, c, s);
        char* dst = static_cast<char*>(a.dqkv) + ((static_cast<size_t>(at.tk) * rows.all + at.p) * D + ea) * kElem;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (u >= at.count) break;
            const int p = at.p + u, seg = (p >= a.heads[0]) + (p >= a.heads[0] + a.heads[1]);
            if (seg < 2) {
                float2 wf[2], ws[2];
                lane_weights<D, INTER>(w, seg, ea, eb, wf, ws);
                const Quad x = unpack<F32, INTER>(rx[u]), dy = unpack<F32, INTER>(rg[u]);
                rg[u] = pack<F32, INTER>(row_gradient<kLanes>(x, dy, c, s, wf, ws, a.eps, at.there, seg, dw));
            }
            if (at.there) store8<F32>(dst + u * D * kElem, dst + gap + u * D * kElem, rg[u]);
        }
        at = next;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            rx[u] = nx[u];
            rg[u] = ng[u];
        }
    }
    if (a.part == nullptr) return;
    block_sums<D, INTER>(dw, sums, ea, eb, a.part);
}

// Sum of `rows` partial rows of 2 D values: a block owns 8 columns, 32 threads each, which have 16
// rows' loads in flight.
template <int D>
__global__ void __launch_bounds__(256)
    dweight_sum_kernel(const float* __restrict__ part, int rows, float* dq, float* dk) {
    constexpr int kTogether = 16;
    __shared__ float sums[8][8];
    griddep_wait();
    const int col = threadIdx.x % 8, k = threadIdx.x / 8, warp = threadIdx.x / 32;
    const int x = blockIdx.x * 8 + col;
    float v = 0.f;
    for (int r0 = k; r0 < rows; r0 += 32 * kTogether) {
        float t[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            const int r = r0 + 32 * i;
            t[i] = r < rows ? part[static_cast<size_t>(r) * 2 * D + x] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) v += t[i];
    }
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (threadIdx.x % 32 < 8) sums[warp][col] = v;
    __syncthreads();
    if (threadIdx.x < 8) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += sums[i][col];
        float* dst = x < D ? dq : dk;
        if (dst != nullptr) dst[x % D] = v;
    }
}

// Passes of Q, K and V, and how many of a token's a warp takes at a time: the number that gives the
// busiest of `warps` resident warps the least to do, counting three passes more for every run (its
// token's angles and its loads' latency; cut into 24 runs of a pass each, 16384 tokens take 262 us for
// 69).  That is all of a token's passes where there are many tokens, and one pass a warp for one
// token of 40 heads.  Against filling 32 warps an SM, d = 128, H 32 / 8: 512 tokens 5.4 us for 7.1,
// 2000 tokens 11.6 for 13.9, their gradient 19.7 for 20.7, that of 500 tokens 7.6 for 9.2.
int least_per(long long tokens, int all, long long warps, int edge, long long* cost_of) {
    long long least = -1;
    int least_of = all;
    for (int chunks = 1;;) {  // 1, 2, 3, 4, 6, 9, ... 63, all
        const int per = (all + chunks - 1) / chunks;
        const long long runs = tokens * ((all + per - 1) / per);
        const long long cost = (runs + warps - 1) / warps * (per + edge);
        if (least < 0 || cost < least) {
            least = cost;
            least_of = per;
        }
        if (chunks >= all) break;
        chunks += chunks < 4 ? 1 : chunks / 2;
        if (chunks > all || chunks > 63) chunks = all;
    }
    *cost_of = least;
    return least_of;
}
Split split_passes(const NormRopeArgs& a, int d, long long warps, long long* cost_of) {
    const int per_pass = 256 / d;  // heads of one pass
    Split sp;
    sp.first[0] = 0;
    for (int i = 0; i < 3; ++i) sp.first[i + 1] = sp.first[i] + (a.heads[i] + per_pass - 1) / per_pass;
    const int all = sp.first[3];
    sp.per = least_per(a.tokens, all, warps, 3, cost_of);
    sp.chunks = (all + sp.per - 1) / sp.per;
    // against the rows kernels: batches of one pass for K and for V cost their latency once more
    if (sp.first[2] - sp.first[1] == 1) *cost_of += 2 * ((static_cast<long long>(a.tokens) * sp.chunks + warps - 1) / warps);
    sp.by_tokens = make_div(a.tokens);
    sp.by_n = make_div(a.N);
    return sp;
}

// The rows kernels' work, in the same way.
Rows split_rows(const NormRopeArgs& a, int d, int ahead, long long warps, long long* cost_of) {
    const uint32_t together = 256 / d;
    Rows r;
    r.all = a.heads[0] + 2 * a.heads[1];
    r.groups = a.tokens / together + (a.tokens % together != 0);
    r.per = least_per(r.groups, r.all, warps, 4, cost_of);
    const int batches = (r.per + ahead - 1) / ahead;
    r.batch = (r.per + batches - 1) / batches;
    r.items = r.groups * ((r.all + r.per - 1) / r.per);
    r.by_groups = make_div(r.groups);
    r.by_n = make_div(a.N);
    return r;
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

int grid_of(long long warps, int cap) {
    const long long blocks = (warps + kWarps - 1) / kWarps;
    return static_cast<int>(blocks < cap ? blocks : cap);
}

template <int D, bool F32, bool INTER, int AXES>
cudaError_t launch_fwd(const NormRopeArgs& a, cudaStream_t s) {
    static std::atomic<int> known[64], known_rows[64];
    int sms = 0, cap = 0, cap_rows = 0;
    cudaError_t e = resident_ctas(qk_norm_rope_kernel<D, F32, INTER, AXES>, known, &sms, &cap);
    if (e == cudaSuccess) e = resident_ctas(qk_norm_rope_rows_kernel<D, F32, INTER, AXES>, known_rows, &sms, &cap_rows);
    if (e != cudaSuccess) return e;
    long long cost = 0, cost_rows = 0;
    const Split sp = split_passes(a, D, static_cast<long long>(cap) * kWarps, &cost);
    const Rows rows = split_rows(a, D, F32 ? 2 : 8, static_cast<long long>(cap_rows) * kWarps, &cost_rows);
    if (cost_rows < cost)
        return launch_pdl(qk_norm_rope_rows_kernel<D, F32, INTER, AXES>, dim3(grid_of(rows.items, cap_rows)), dim3(kThreads),
                          0, s, a, rows);
    return launch_pdl(qk_norm_rope_kernel<D, F32, INTER, AXES>,
                      dim3(grid_of(static_cast<long long>(a.tokens) * sp.chunks, cap)), dim3(kThreads), 0, s, a, sp);
}

template <int D, bool F32, bool INTER, int AXES>
cudaError_t launch_bwd(NormRopeArgs a, float* const (&dweight)[2], cudaStream_t s) {
    static std::atomic<int> known[64], known_rows[64];
    int sms = 0, cap = 0, cap_rows = 0;
    cudaError_t e = resident_ctas(qk_norm_rope_bwd_kernel<D, F32, INTER, AXES>, known, &sms, &cap);
    if (e == cudaSuccess) e = resident_ctas(qk_norm_rope_rows_bwd_kernel<D, F32, INTER, AXES>, known_rows, &sms, &cap_rows);
    if (e != cudaSuccess) return e;
    long long cost = 0, cost_rows = 0;
    const Split sp = split_passes(a, D, static_cast<long long>(cap) * kWarps, &cost);
    const Rows rows = split_rows(a, D, F32 ? 2 : 4, static_cast<long long>(cap_rows) * kWarps, &cost_rows);
    const bool want = dweight[0] != nullptr || dweight[1] != nullptr, by_rows = a.any_order && cost_rows < cost;
    if (!want) a.part = nullptr;
    if (by_rows) cap = cap_rows;
    if (cap > kBwdMaxBlocks) cap = kBwdMaxBlocks;
    const int grid = grid_of(by_rows ? rows.items : static_cast<long long>(a.tokens) * sp.chunks, cap);
    e = by_rows ? launch_pdl(qk_norm_rope_rows_bwd_kernel<D, F32, INTER, AXES>, dim3(grid), dim3(kThreads), 0, s, a, rows)
                : launch_pdl(qk_norm_rope_bwd_kernel<D, F32, INTER, AXES>, dim3(grid), dim3(kThreads), 0, s, a, sp);
    if (e != cudaSuccess || !want) return e;
    return launch_pdl(dweight_sum_kernel<D>, dim3(2 * D / 8), dim3(256), 0, s, a.part, grid, dweight[0],
                      dweight[1]);
}

// f with the kernel variant's parameters: d, float32, neighbouring pairs, several axes (2) or one.
template <typename F>
cudaError_t pick(const NormRopeArgs& a, int d, int f32, int interleaved, F f) {
    auto axes = [&](auto D, auto F32, auto INTER) {
        return a.axes > 1 ? f(D, F32, INTER, std::integral_constant<int, 2>{})
                          : f(D, F32, INTER, std::integral_constant<int, 1>{});
    };
    auto pairs = [&](auto D, auto F32) {
        return interleaved ? axes(D, F32, std::true_type{}) : axes(D, F32, std::false_type{});
    };
    auto type = [&](auto D) { return f32 ? pairs(D, std::true_type{}) : pairs(D, std::false_type{}); };
    return d == 64 ? type(std::integral_constant<int, 64>{}) : type(std::integral_constant<int, 128>{});
}

}  // namespace

size_t qk_norm_rope_bwd_workspace_bytes(int d) {
    return static_cast<size_t>(kBwdMaxBlocks) * 2 * d * sizeof(float);
}

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int d, int f32, int interleaved, cudaStream_t s) {
    return pick(a, d, f32, interleaved, [&](auto D, auto F32, auto INTER, auto AXES) {
        return launch_fwd<decltype(D)::value, decltype(F32)::value, decltype(INTER)::value, decltype(AXES)::value>(a, s);
    });
}

cudaError_t launch_qk_norm_rope_bwd(const NormRopeArgs& a, float* const (&dweight)[2], int d, int f32,
                                    int interleaved, cudaStream_t s) {
    return pick(a, d, f32, interleaved, [&](auto D, auto F32, auto INTER, auto AXES) {
        return launch_bwd<decltype(D)::value, decltype(F32)::value, decltype(INTER)::value, decltype(AXES)::value>(
            a, dweight, s);
    });
}

}  // namespace fa
