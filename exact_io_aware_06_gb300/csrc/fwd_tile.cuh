// fwd_tile.cuh -- pieces of the forward kernels whose query tiles of 128 rows meet lists of key blocks (the
// windowed ones and cross attention's): the online softmax of a block, O on its way out.
#pragma once

#include <cmath>
#include <type_traits>

#include "fwd_sizes.h"
#include "internal.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kTau = 8.0f;   // lazy-rescale threshold, log2 units

__device__ __forceinline__ void record_timeout(const DevCtl& ctl, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicCAS(ctl.status, kDevOk, kDevTimeout);
}

// Store a box from shared to global memory through the tensor map, in the thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit_group() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All of this thread's committed bulk operations have read shared memory / have completed.
__device__ __forceinline__ void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 consecutive TMEM columns of this thread's lane into r[OFF..], no wait.
template <int OFF, int NC>
__device__ __forceinline__ void ld32_at(uint32_t taddr, uint32_t (&r)[NC]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[OFF + 0]), "=r"(r[OFF + 1]), "=r"(r[OFF + 2]), "=r"(r[OFF + 3]),
          "=r"(r[OFF + 4]), "=r"(r[OFF + 5]), "=r"(r[OFF + 6]), "=r"(r[OFF + 7]),
          "=r"(r[OFF + 8]), "=r"(r[OFF + 9]), "=r"(r[OFF + 10]), "=r"(r[OFF + 11]),
          "=r"(r[OFF + 12]), "=r"(r[OFF + 13]), "=r"(r[OFF + 14]), "=r"(r[OFF + 15]),
          "=r"(r[OFF + 16]), "=r"(r[OFF + 17]), "=r"(r[OFF + 18]), "=r"(r[OFF + 19]),
          "=r"(r[OFF + 20]), "=r"(r[OFF + 21]), "=r"(r[OFF + 22]), "=r"(r[OFF + 23]),
          "=r"(r[OFF + 24]), "=r"(r[OFF + 25]), "=r"(r[OFF + 26]), "=r"(r[OFF + 27]),
          "=r"(r[OFF + 28]), "=r"(r[OFF + 29]), "=r"(r[OFF + 30]), "=r"(r[OFF + 31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float min3f(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Max (or, for a negative score scale, min) of NC raw scores: four 3-input chains.
template <int NC>
__device__ __forceinline__ float extreme(const uint32_t (&r)[NC], bool want_max) {
    float a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = __uint_as_float(r[k]);
    if (want_max) {
#pragma unroll
        for (int i = 4; i + 8 <= NC; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                a[k] = max3f(a[k], __uint_as_float(r[i + 2 * k]), __uint_as_float(r[i + 2 * k + 1]));
        a[0] = max3f(a[0], __uint_as_float(r[NC - 4]), __uint_as_float(r[NC - 3]));
        a[1] = max3f(a[1], __uint_as_float(r[NC - 2]), __uint_as_float(r[NC - 1]));
        return max3f(a[0], a[1], fmaxf(a[2], a[3]));
    }
#pragma unroll
    for (int i = 4; i + 8 <= NC; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            a[k] = min3f(a[k], __uint_as_float(r[i + 2 * k]), __uint_as_float(r[i + 2 * k + 1]));
    a[0] = min3f(a[0], __uint_as_float(r[NC - 4]), __uint_as_float(r[NC - 3]));
    a[1] = min3f(a[1], __uint_as_float(r[NC - 2]), __uint_as_float(r[NC - 1]));
    return min3f(a[0], a[1], fminf(a[2], a[3]));
}

// Bits below n (all of them for n >= 32, none for n <= 0).
__device__ __forceinline__ uint32_t bits_below(int n) {
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// One key block for one row: NC raw scores (columns colS ..) to P (columns colP ..), the reference
// maximum, the sum and, where the reference moves, O.  `taken` is called once the scores are in
// registers; `free` before P and O are written, true when P V of the tile's last block is done.
// Returns false when `free` did.  With `half` O is rescaled first, and it is called once the first 64 columns of
// P are in TMEM, so that P V can begin.
// P is rounded to bf16, the type of V, as one matrix product takes operands of one type: each weight is off by up to 2^-8
// of itself, o by that of sum w |v| at most (its error relative to 64 bits 2.1e-3 to 2.35e-3, where P kept in
// float32 would leave 1.7e-3).  The sum l adds up P before that rounding; maximum, sum and O are float32.
struct NoHalf {};
template <int D, int NC, class Taken, class Free, class Half = NoHalf>
__device__ __forceinline__ bool softmax_block(uint32_t lane_base, uint32_t colS, uint32_t colP, uint32_t colO, float c,
                                              bool c_pos, uint32_t mask_bits, int hi, int lo, int sink, bool first,
                                              float& m_ref, float& l, Taken taken, Free free, Half half = {}) {
    uint32_t r[NC];
    ld32_at<0>(lane_base + colS, r);
    if constexpr (NC >= 64) ld32_at<32>(lane_base + colS + 32, r);
    if constexpr (NC == 128) {
        ld32_at<64>(lane_base + colS + 64, r);
        ld32_at<96>(lane_base + colS + 96, r);
    }
    tmem_wait_ld();
    reg_fence(r);
    taken();
    // Keys hi and below, of those the ones from lo on or below `sink`, counted in the block.  (Tests
    // for the runs of 32 keys that hold a bound only, and no exponentials where no row of the warp
    // sees a key, were both slower, by 1.5% and 25%: branches among the runs keep the compiler from
    // interleaving them.)
    if (hi < NC - 1 || (lo > 0 && sink < NC)) {
#pragma unroll
        for (int w = 0; w < NC / 32; ++w) {
            const uint32_t seen = bits_below(hi + 1 - 32 * w) & (~bits_below(lo - 32 * w) | bits_below(sink - 32 * w));
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (!(seen & (1u << i))) r[32 * w + i] = mask_bits;
        }
    }
    const float mt = c * extreme(r, c_pos);
    float alpha = 1.f;
    const bool bump = mt > m_ref + kTau;
    if (bump) {
        alpha = (m_ref == -INFINITY) ? 0.f : ex2_approx(m_ref - mt);
        m_ref = mt;
        l *= alpha;
    }
    constexpr bool kHalf = !std::is_same<Half, NoHalf>::value;
    if constexpr (kHalf) {
        if (!first && __any_sync(0xffffffffu, bump)) {  // (with the scores in registers: few columns at a time)
#pragma unroll 1
            for (int q = 0; q < D; q += 8) {
                uint32_t ov[8];
                tmem_ld8(lane_base + colO + q, ov);
#pragma unroll
                for (int i = 0; i < 8; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                tmem_st8(lane_base + colO + q, ov);
            }
        }
    }
    const float ref = (m_ref == -INFINITY) ? 0.f : m_ref;
    const float2 c2 = make_float2(c, c), nref2 = make_float2(-ref, -ref);
    float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
    for (int h = 0; h < (NC + 63) / 64; ++h) {
        constexpr int kW = NC < 64 ? NC / 2 : 32;
        uint32_t pk[kW];
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const int e = 64 * h + 2 * i;
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), c2, nref2);
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            if (i & 1)
                acc1 = __fadd2_rn(acc1, p);
            else
                acc0 = __fadd2_rn(acc0, p);
            pk[i] = pack_bf16x2(p.x, p.y);
        }
        if (h == 0 && !free()) return false;
        if constexpr (NC < 64)
            tmem_st16(lane_base + colP, pk);
        else
            tmem_st32(lane_base + colP + 32 * h, pk);
        if constexpr (kHalf) {
            if (h == 0) {
                tmem_st_wait();
                half();
            }
        }
    }
    if (!kHalf && !first && __any_sync(0xffffffffu, bump)) {
#pragma unroll
        for (int q4 = 0; q4 < D / 32; ++q4) {
            uint32_t ov[32];
            tmem_ld32(lane_base + colO + 32 * q4, ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(lane_base + colO + 32 * q4, ov);
        }
    }
    l += (acc0.x + acc0.y) + (acc1.x + acc1.y);
    tmem_st_wait();
    return true;
}

// A warp's 32 rows of O, times `f`, from TMEM to global memory, 64 columns at a time: each lane writes
// its row's 128 bytes into the warp's own 4 KB of shared memory (16-byte granule g of row r at
// g ^ (r % 8)), one lane stores the box by TMA, and the next box waits until that has been read.
// Rows past N are not written by the store.  (Each lane storing its row itself takes 32 lines an
// instruction, in the way of the warps' next TMEM loads.)
template <int D>
__device__ __forceinline__ void store_rows(const CUtensorMap& tm_o, uint32_t box, uint32_t taddr, float f, int row0, int bh,
                                           int N) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        uint32_t ov[2][32];
        tmem_ld32_async(taddr + 64 * c, ov[0]);
        tmem_ld32_async(taddr + 64 * c + 32, ov[1]);
        tmem_wait_ld();
        reg_fence(ov[0]);
        reg_fence(ov[1]);
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const uint32_t* x = ov[g / 4] + 8 * (g % 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 128 + ((g ^ (lane & 7)) << 4)),
                         "r"(pack_bf16x2(__uint_as_float(x[0]) * f, __uint_as_float(x[1]) * f)),
                         "r"(pack_bf16x2(__uint_as_float(x[2]) * f, __uint_as_float(x[3]) * f)),
                         "r"(pack_bf16x2(__uint_as_float(x[4]) * f, __uint_as_float(x[5]) * f)),
                         "r"(pack_bf16x2(__uint_as_float(x[6]) * f, __uint_as_float(x[7]) * f))
                         : "memory");
        }
        fence_proxy_async_smem();  // the lanes' writes -> visible to the TMA unit
        __syncwarp();
        if (lane == 0 && row0 < N) {
            tma_store_3d(&tm_o, box, 64 * c, row0, bh);
            bulk_commit_group();
        }
    }
}

}  // namespace
}  // namespace fa
