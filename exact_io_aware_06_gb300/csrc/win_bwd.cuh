// win_bwd.cuh -- what the windowed backward's kernels share.
#pragma once

#include <cmath>

#include "layer_ops.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace fa {

struct WinBwdArgs {
    const float* ws_delta;  // [BH][Np], negated: -delta_i
    const float* ws_lse2;   // [BH][Np], negated: -lse_i * log2(e)
    void* dk;
    void* dv;
    int N, Np, n_kv, BH;    // BH: K/V heads (B * H_kv), the grid's head count
    int H, H_kv;            // query heads and K/V heads per batch; H_kv divides H
    WinSplit split;         // sink blocks' pieces
    float* part;            // their dV, dK: [BH][n_part][pieces + 1][2][d / 4][128][4] float32
    float c_log2;           // scale * log2(e), not 0
    float scale;
    DevCtl ctl;
};

namespace {

using BwdArgs = WinBwdArgs;

constexpr int kBlk = 128;  // keys of an item, queries of a step
constexpr float kLog2e = 1.4426950408889634f;

// An item: one K/V head's 128-key block kvb with the query blocks of its window, or a piece of a
// sink block's later query blocks.  Pieces come first, then the key blocks in order: all but a
// head's last ones meet equally many.
struct Item {
    int bh, kvb, i0, n_loc, n_it;
    int slot;  // -1: dK and dV are final; else the part that this item leaves
};
__device__ __forceinline__ int far_items(const BwdArgs& a) { return a.split.n_part * a.split.pieces * a.BH; }
__device__ __forceinline__ Item item_at(const BwdArgs& a, int x) {
    const int n_far = far_items(a), n_q = a.n_kv, reach = a.split.reach;
    Item I;
    I.bh = x % a.BH;
    const int y = x / a.BH;
    if (x < n_far) {
        I.kvb = y % a.split.n_part;
        const int piece = y / a.split.n_part;
        I.i0 = I.kvb + reach + 1 + piece * a.split.per;
        I.n_loc = max(0, min(a.split.per, n_q - I.i0));
        I.slot = 1 + piece;
    } else {
        I.kvb = y - a.split.n_part * a.split.pieces;
        I.i0 = I.kvb;
        I.n_loc = min(n_q - 1, I.kvb + reach) - I.kvb + 1;
        I.slot = I.kvb < a.split.n_part ? 0 : -1;
    }
    // with grouped-query attention, that range for each of the query heads that share this K/V
    // head (dK, dV sum over all of them)
    I.n_it = a.H / a.H_kv * I.n_loc;
    return I;
}
// The query blocks of an item one after the other, without a division a step.
struct Walk {
    int head, blk, end, i0;
    __device__ __forceinline__ Walk(const BwdArgs& a, const Item& I)
        : head((I.bh / a.H_kv) * a.H + (I.bh % a.H_kv) * (a.H / a.H_kv)), blk(I.i0), end(I.i0 + I.n_loc), i0(I.i0) {}
    __device__ __forceinline__ void next() {
        if (++blk == end) {
            blk = i0;
            ++head;
        }
    }
};
// This CTA's k-th item, dealt in alternating order.
__device__ __forceinline__ int item_x(int k) {
    const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    return k * G + ((k & 1) ? G - 1 - c : c);
}

__device__ __forceinline__ void record_timeout(const DevCtl& ctl, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicCAS(ctl.status, kDevOk, kDevTimeout);
}

// Bits below n (all of them for n >= 32, none for n <= 0).
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}
// P^T of this thread's key and a run of 32 NW queries from their raw scores, in their place, and as
// bf16 pairs for dV.  The key's queries are q_first .. q_end - 1, counted from the first of the run;
// nl: -lse log2(e) of the queries.
template <int NW>
__device__ __forceinline__ void probabilities(uint32_t (&r)[NW][32], int q_first, int q_end, uint32_t hide, float2 c2,
                                              const float4* nl, uint32_t (&pk)[16 * NW]) {
    // a warp's keys are neighbours: of two runs of 32 queries mostly one holds a bound of some key
    // and needs the test of every score
    if (__any_sync(0xffffffffu, q_first > 0 || q_end < 32 * NW)) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const uint32_t seen = bits_below(q_end - 32 * w) & ~bits_below(q_first - 32 * w);
            if (__any_sync(0xffffffffu, seen != 0xffffffffu)) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (!(seen & (1u << i))) r[w][i] = hide;
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 8 * NW; ++x) {
        uint32_t* rr = &r[x / 8][4 * (x % 8)];
        const float4 l = nl[x];
        const float2 a = __ffma2_rn(make_float2(__uint_as_float(rr[0]), __uint_as_float(rr[1])), c2, make_float2(l.x, l.y));
        const float2 b = __ffma2_rn(make_float2(__uint_as_float(rr[2]), __uint_as_float(rr[3])), c2, make_float2(l.z, l.w));
        const float p0 = ex2_approx(a.x), p1 = ex2_approx(a.y), p2 = ex2_approx(b.x), p3 = ex2_approx(b.y);
        pk[2 * x] = pack_bf16x2(p0, p1);
        pk[2 * x + 1] = pack_bf16x2(p2, p3);
        rr[0] = __float_as_uint(p0);
        rr[1] = __float_as_uint(p1);
        rr[2] = __float_as_uint(p2);
        rr[3] = __float_as_uint(p3);
    }
}
// dS^T = P^T o (dP^T - delta) of 32 queries as bf16 pairs; nd: -delta.
__device__ __forceinline__ void score_gradients(const uint32_t (&p)[32], const uint32_t (&dp)[32], const float4* nd,
                                                uint32_t (&w)[16]) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const float4 d = nd[x];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int e = 4 * x + 2 * y;
            const float2 g = __fadd2_rn(make_float2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])),
                                        y ? make_float2(d.z, d.w) : make_float2(d.x, d.y));
            const float2 ds = __fmul2_rn(make_float2(__uint_as_float(p[e]), __uint_as_float(p[e + 1])), g);
            w[2 * x + y] = pack_bf16x2(ds.x, ds.y);
        }
    }
}
// A key's queries counted from query q0: from the key on, a window's worth, or all for a sink.
__device__ __forceinline__ void query_range(const WinSplit& sp, int key, int q0, int& q_first, int& q_end) {
    q_first = key - q0;
    const long long end = static_cast<long long>(q_first) + sp.window;
    q_end = key < sp.sinks ? kBlk : static_cast<int>(min(static_cast<long long>(kBlk), end));
}

// 16 TMEM lanes x 64 columns, lane 4 r + q of the warp holding columns 8 j + 2 q, + 1 of rows r
// (x[4 j], x[4 j + 1]) and r + 8 (x[4 j + 2], x[4 j + 3]).
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&x)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
          "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]),
          "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]),
          "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
        : "r"(taddr)
        : "memory");
}
// Lane q of every four holds word q of four 16-byte pieces; afterwards lane q holds piece q.
__device__ __forceinline__ void transpose4(uint32_t& a0, uint32_t& a1, uint32_t& a2, uint32_t& a3, int q) {
    const bool odd = q & 1, high = q & 2;
    uint32_t r = __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
    (odd ? a0 : a1) = r;
    r = __shfl_xor_sync(0xffffffffu, odd ? a2 : a3, 1);
    (odd ? a2 : a3) = r;
    r = __shfl_xor_sync(0xffffffffu, high ? a0 : a2, 2);
    (high ? a0 : a2) = r;
    r = __shfl_xor_sync(0xffffffffu, high ? a1 : a3, 2);
    (high ? a1 : a3) = r;
}

// A warp's 32 rows of D accumulator columns, times a factor and as bf16, on their way from TMEM to
// global memory in pieces of 64 bytes of 8 rows: one row per lane would make every store
// instruction touch 32 lines, and the next TMEM loads of the SM waited 2300 cycles behind them.
template <int D>
struct RowsOut {
    uint32_t w[2][D / 64][2][8];  // rows 16 m + lane / 4 and 8 more, columns 64 c + 8 j + 2 (lane % 4)
    __device__ __forceinline__ void load(uint32_t taddr, float f) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t x[32];
                tmem_ld_rows16(taddr + (static_cast<uint32_t>(16 * m) << 16) + 64 * c, x);
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        w[m][c][h][j] = pack_bf16x2(__uint_as_float(x[4 * j + 2 * h]) * f, __uint_as_float(x[4 * j + 2 * h + 1]) * f);
            }
    }
    // Row r of the warp to row first + row0 + r of `out`, if row0 + r < N.
    __device__ __forceinline__ void store(void* out, size_t first, int row0, int N) {
        const int lane = threadIdx.x % 32, q = lane % 4;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = row0 + 16 * m + 8 * h + lane / 4;
                uint16_t* dst = static_cast<uint16_t*>(out) + (first + row) * D;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        uint32_t(&p)[8] = w[m][c][h];
                        transpose4(p[j], p[j + 1], p[j + 2], p[j + 3], q);  // columns 64 c + 8 (j + q) ..
                        if (row < N)
                            *reinterpret_cast<uint4*>(dst + 64 * c + 8 * (j + q)) = make_uint4(p[j], p[j + 1], p[j + 2], p[j + 3]);
                    }
            }
    }
};

// This thread's key row of dV (which = 0) or dK, unscaled, from TMEM to its place in the
// workspace, where four columns of all rows lie side by side: a warp's store is 512 bytes in a run.
// Rows past N are zeros and fill their places too.
template <int D>
__device__ __forceinline__ void write_part_row(const BwdArgs& a, const Item& I, int which, int row, uint32_t taddr) {
    const size_t part = (static_cast<size_t>(I.bh) * a.split.n_part + I.kvb) * (a.split.pieces + 1) + I.slot;
    uint4* dst = reinterpret_cast<uint4*>(a.part) + (2 * part + which) * (kBlk * D / 4) + row;
#pragma unroll
    for (int h = 0; h < D / 32; ++h) {
        uint32_t r[32];
        tmem_ld32(taddr + 32 * h, r);
#pragma unroll
        for (int x = 0; x < 8; ++x) dst[(8 * h + x) * kBlk] = make_uint4(r[4 * x], r[4 * x + 1], r[4 * x + 2], r[4 * x + 3]);
    }
}

// dV and dK of the blocks that were dealt in parts: the parts added in order, dK times scale,
// rounded once.  Thread t of n (whole warps), eight neighbouring values of a row at a time: a warp
// takes 8 rows x 32 columns, whole lines of the parts and 64-byte runs of the result.
template <int D>
__device__ __forceinline__ void join_parts(const BwdArgs& a, int t, int n) {
    constexpr int kCols = D / 32, kTiles = kCols * (kBlk / 8);  // such tiles of a block's dV or dK
    const WinSplit& sp = a.split;
    const size_t work = static_cast<size_t>(a.BH) * sp.n_part * 2 * kTiles * 32;
    for (size_t x = t; x < work; x += n) {
        const int lane = static_cast<int>(x % 32), tile = static_cast<int>(x / 32 % kTiles);
        const int row = tile / kCols * 8 + lane % 8, vec = tile % kCols * 4 + lane / 8;
        const int which = static_cast<int>(x / (32 * kTiles) % 2);
        const size_t blk = x / (2 * 32 * kTiles);  // bh * n_part + kvb
        const int kvb = static_cast<int>(blk % sp.n_part);
        const size_t bh = blk / sp.n_part;
        const int key = kvb * kBlk + row;
        if (key >= a.N) continue;
        const int slots = 1 + (a.n_kv - 1 - sp.reach - kvb + sp.per - 1) / sp.per;
        const float4* src =
            reinterpret_cast<const float4*>(a.part) + (blk * (sp.pieces + 1) * 2 + which) * (kBlk * D / 4) + 2 * vec * kBlk + row;
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
#pragma unroll 4
        for (int i = 0; i < slots; ++i) {
            const float4 y = src[0], z = src[kBlk];
            u.x += y.x, u.y += y.y, u.z += y.z, u.w += y.w;
            w.x += z.x, w.y += z.y, w.z += z.z, w.w += z.w;
            src += 2 * (kBlk * D / 4);
        }
        const float f = which ? a.scale : 1.f;
        static_cast<uint4*>(which ? a.dk : a.dv)[(bh * a.N + key) * (D / 8) + vec] =
            make_uint4(pack_bf16x2(u.x * f, u.y * f), pack_bf16x2(u.z * f, u.w * f), pack_bf16x2(w.x * f, w.y * f),
                       pack_bf16x2(w.z * f, w.w * f));
    }
}

}  // namespace

// dK and dV of the windowed backward for d = 64; grid: CTAs.
cudaError_t launch_bwd_window_main64(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                                     const CUtensorMap& dk, const CUtensorMap& dv, const WinBwdArgs& a, int grid,
                                     cudaStream_t s);
// dQ, and the join of the parts that the dK/dV kernel has left.
int launch_bwd_window_dq(const void* q, const void* k, const void* v, const void* dO, void* dq, const WinBwdArgs& a, int d,
                         cudaStream_t s);

}  // namespace fa
