// bwd_tile.cuh -- what the backward kernels over lists of 128-row blocks share (the windowed ones and cross
// attention's).  Which blocks meet is the arguments' matter: for an argument type A with
//     c_log2, scale, ws_delta, ws_lse2 (rows [heads][Np] of N), dk, dv, part, ctl
// the kernels call the overloads
//     item_count(a), item_at(a, x)       dK/dV: an Item
//     walk_of(a, I)                      its query blocks one after the other: head, blk, next()
//     query_range(a, I, key, q0, ..)     which queries from q0 on a key meets
//     key_rows(a), part_of(a, I)         rows of a head of dK and dV; an item's parts of dV (twice that) and dK (+ 1)
//     hides(a)                           whether hidden keys may hold anything, an infinity or a NaN
#pragma once

#include <cmath>

#include "internal.h"
#include "layer_ops.h"
#include "ptx.cuh"
#include "rows_out.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kBlk = 128;  // keys of an item, queries of a step
constexpr float kLog2e = 1.4426950408889634f;

// An item of dK/dV: a K/V head's 128-key block kvb and query blocks that meet it.
struct Item {
    int bh, kvb, i0, n_loc, n_it;
    int slot;  // -1: dK and dV are final; else the part that this item leaves
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
// bf16 pairs for dV (the type of dO, the product's other operand).  The key's queries are q_first .. q_end - 1, counted from the first of the run;
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
// dS^T = P^T o (dP^T - delta) of 32 queries as bf16 pairs (the type of Q, the other operand of dK's product: a step's error
// relative to 64 bits 2.4e-3, of which the gradients' own rounding is 1.7e-3); P before its rounding; nd: -delta.
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

// This thread's row of an accumulator, unscaled, from TMEM to its place in the workspace (`there`: if it is one of
// the tensor's), where four columns of all rows lie side by side: a warp's store is 512 bytes in a run.
template <int D>
__device__ __forceinline__ void write_part_row(float* parts, size_t part, int row, bool there, uint32_t taddr) {
    uint4* dst = reinterpret_cast<uint4*>(parts) + part * (kBlk * D / 4) + row;
#pragma unroll
    for (int h = 0; h < D / 32; ++h) {
        uint32_t r[32];
        tmem_ld32(taddr + 32 * h, r);
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (there) dst[(8 * h + x) * kBlk] = make_uint4(r[4 * x], r[4 * x + 1], r[4 * x + 2], r[4 * x + 3]);
    }
}

__device__ __forceinline__ float dot8(const uint4& x, const uint4& y) {
    const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sum = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), sum);
        sum = fmaf(__uint_as_float(a[e] & 0xFFFF0000u), __uint_as_float(b[e] & 0xFFFF0000u), sum);
    }
    return sum;
}
template <int FROM, int TO>
__device__ __forceinline__ float lanes_sum(float x) {  // over the lanes that differ in bits FROM .. TO / 2
#pragma unroll
    for (int off = FROM; off < TO; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

int grid_for(size_t work, int threads, int max_blocks) {
    size_t b = (work + threads - 1) / threads;
    if (b > static_cast<size_t>(max_blocks)) b = max_blocks;
    return static_cast<int>(b < 1 ? 1 : b);
}

}  // namespace
}  // namespace fa
