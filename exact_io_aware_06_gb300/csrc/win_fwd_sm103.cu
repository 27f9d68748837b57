// win_fwd_sm103.cu -- forward of attention under a causal sliding window with sinks, on the
// sm_103a tensor core (tcgen05 + TMEM + TMA).
//
// Query i sees key j iff j <= i and (j > i - W or j < S): the W newest keys and the first S.
// The online softmax is the plain forward's (fwd_sm103.cu): per row a running reference
// maximum, sum and unnormalised output, lazily rescaled, o / l and lse = m + ln l at the end.
//
// Bound by the tensor pipe and the thread that feeds it, so the work is to visit only key
// blocks that hold a visible key, and as little as possible of those:
//   * Item = two query tiles of 128 rows (one head), as in the plain forward: K_j and V_j
//     are loaded once for both.  An item's list of 128-key blocks is the sinks' blocks, then
//     the window's, from the first row's first key to the last row's diagonal.  The two
//     tiles' ranges differ by one block at either end, and a tile leaves out the block that
//     it sees nothing of: without that, W = 512 would cost 6 blocks per tile for 5.
//   * Up to 32 sinks in front of a window that has left them behind take a short block: S of
//     32 keys and P V of two K steps instead of 128 and eight, a quarter of the softmax work.
//   * Blocks that are visible whole need no mask; the others take a row's visible keys as four
//     32-bit words, made by shifts from the row's two bounds, and one bit test per score.
// Warp roles, TMEM columns, the K/V bundle ring and the order of MMAs are the plain
// forward's; O leaves through shared memory and TMA stores.  Every wait is bounded, and a wait
// that runs out is recorded and ends the CTA with its copies and MMAs drained.
#include <cmath>
#include <type_traits>

#include "layer_ops.h"
#include "ptx.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kBM = 128;       // query rows per tile
constexpr int kBN = 128;       // keys per block
constexpr int kShort = 32;     // keys of a short sink block
constexpr int kStages = 2;     // K/V ring depth
constexpr int kThreads = 384;  // 12 warps
constexpr float kTau = 8.0f;   // lazy-rescale threshold, log2 units

struct WinArgs {
    float* lse;
    int N, n_pairs, BH, n_items;
    int window, sinks;
    float c_log2;  // scale * log2(e), not 0
    int H, H_kv;
    DevCtl ctl;
};

template <int D>
struct Cfg {
    static constexpr int kChunks = D / 64;             // 128-byte swizzle columns per row
    static constexpr int kChunkBytes = 128 * 128;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kOffQ = 0;                    // Q0, Q1
    static constexpr int kOffK = 2 * kTileBytes;       // K[kStages]
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffO = kOffV + kStages * kTileBytes;  // 4 KB per softmax warp: 32 rows x 128 bytes
    static constexpr int kSmemBytes = kOffO + 8 * 4096;
    static constexpr int kSmemAlloc = kSmemBytes + 1024;
    static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kIdescS = idesc_bf16(kBM, kBN, false, false);
    static constexpr uint32_t kIdescShort = idesc_bf16(kBM, kShort, false, false);
    static constexpr uint32_t kIdescO = idesc_bf16(kBM, D, false, true);
};

struct Bars {
    uint64_t q_full, q_free;
    uint64_t kv_full[kStages], kv_empty[kStages];
    uint64_t s_full[2], p_full[2], o_done[2];
    uint64_t drain;
};

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

// Which key blocks a pair of query tiles visits.  List index n: blocks 0 .. n_sink - 1, then
// lo .. ; the first is a short one if `shorty`.  Tile 0 leaves out the last entry when tile 1
// has a diagonal block of its own, tile 1 leaves out entry skip1 (-1: none).
struct Plan {
    int n;          // entries
    int n_sink, lo;
    int skip1;
    bool shorty, two;
    __device__ __forceinline__ int block(int i) const { return i < n_sink ? i : lo + i - n_sink; }
    __device__ __forceinline__ bool active(int t, int i) const {
        return t ? (two && i != skip1) : (!two || i != n - 1);
    }
};
__device__ __forceinline__ Plan plan_of(const WinArgs& a, int r0) {
    Plan p;
    p.two = r0 + kBM < a.N;
    p.lo = max(0, static_cast<int>(static_cast<long long>(r0) - a.window + 1)) / kBN;
    const int lo1 = max(0, static_cast<int>(static_cast<long long>(r0) + kBM - a.window + 1)) / kBN;
    const int last = r0 / kBN + (p.two ? 1 : 0);
    p.shorty = a.sinks > 0 && a.sinks <= kShort && p.lo > 0;
    p.n_sink = min(p.lo, a.sinks / kBN + (a.sinks % kBN ? 1 : 0));
    p.n = p.n_sink + last - p.lo + 1;
    // tile 1 sees nothing of block lo if its window starts behind it and no sink lies in it
    p.skip1 = (p.two && lo1 > p.lo && static_cast<long long>(p.lo) * kBN >= a.sinks) ? p.n_sink : -1;
    return p;
}

// One key block for one row: NC raw scores (columns colS ..) to P in the same columns, the
// reference maximum, the sum and, where the reference moves, O.
template <int D, int NC>
__device__ __forceinline__ void softmax_block(uint32_t lane_base, uint32_t colS, uint32_t colO, float c, bool c_pos,
                                              uint32_t mask_bits, int hi, int lo, int sink, bool first, float& m_ref,
                                              float& l) {
    uint32_t r[NC];
    ld32_at<0>(lane_base + colS, r);
    if constexpr (NC == 128) {
        ld32_at<32>(lane_base + colS + 32, r);
        ld32_at<64>(lane_base + colS + 64, r);
        ld32_at<96>(lane_base + colS + 96, r);
    }
    tmem_wait_ld();
    reg_fence(r);
    // keys hi and below, of those the ones from lo on or below `sink`, counted in the block
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
        if constexpr (NC < 64)
            tmem_st16(lane_base + colS, pk);
        else
            tmem_st32(lane_base + colS + 32 * h, pk);
    }
    if (!first && __any_sync(0xffffffffu, bump)) {
        // O_t += P V of this tile's previous block has completed: it precedes these scores in
        // issue order
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
}

// Persistent: a CTA works through items, its k-th being x = k * gridDim.x + (blockIdx.x, or
// gridDim.x - 1 - blockIdx.x in odd rounds); items run from the last pair of every head to
// the first, the heaviest first (the first W / 256 pairs of a head see fewer keys).  Every
// barrier counts its phases across items: q_full, q_free per item, kv_full, kv_empty per
// bundle, s_full, p_full per block that the tile visits, o_done per item of the tile.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    win_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                   const WinArgs args) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Bars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int N = args.N, n_items = args.n_items, G = static_cast<int>(gridDim.x);
    auto item_x = [&](int k) {
        return k * G + ((k & 1) ? G - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x));
    };
    auto item_bh = [&](int x) { return x % args.BH; };
    auto item_r0 = [&](int x) { return (args.n_pairs - 1 - x / args.BH) * 2 * kBM; };

    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(smem_u32(&bars.q_full), 1);
        mbar_init(smem_u32(&bars.q_free), 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bars.kv_full[s]), 1);
            mbar_init(smem_u32(&bars.kv_empty[s]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bars.s_full[t]), 1);
            mbar_init(smem_u32(&bars.p_full[t]), 128);
            mbar_init(smem_u32(&bars.o_done[t]), 1);
        }
        mbar_init(smem_u32(&bars.drain), 1);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_o);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint64_t lim = args.ctl.wait_ns;
    griddep_wait();
    griddep_launch_dependents();

    // 384 threads x 168 registers at launch: 128 * 120 + 256 * 184 <= 384 * 168
    if (warp < 4) {
        regs_dec<120>();
        if (warp == 0) {
            // ============================================================ TMA producer
            if (lane == 0) {
                const uint32_t qf = smem_u32(&bars.q_full);
                int gb = 0, kq = 0;  // bundles and items issued
                bool ok = true;
                const volatile int never = 0;
                for (int k = 0; ok; ++k) {
                    const int x = item_x(k);
                    if (x >= n_items) break;
                    const int bh = item_bh(x), r0 = item_r0(x);
                    const int bh_kv = (bh / args.H) * args.H_kv + (bh % args.H) / (args.H / args.H_kv);
                    const Plan P = plan_of(args, r0);
                    if (kq > 0 && !mbar_wait(smem_u32(&bars.q_free), (kq - 1) & 1, lim, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    const int n_q = P.two ? 2 : 1;
                    mbar_arrive_expect_tx(qf, n_q * C::kTileBytes);
                    for (int t = 0; t < n_q; ++t)
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_3d(smem_base + C::kOffQ + t * C::kTileBytes + c * C::kChunkBytes, &tm_q, qf,
                                        c * 64, r0 + t * kBM, bh);
                    ++kq;
                    // bundle n = {K of entry n (n < P.n), V of entry n - 1 (n >= 1)}
                    for (int n = 0; n <= P.n; ++n, ++gb) {
                        const int u = gb % kStages;
                        if (gb >= kStages &&
                            !mbar_wait(smem_u32(&bars.kv_empty[u]), ((gb / kStages) & 1) ^ 1, lim, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb = smem_u32(&bars.kv_full[u]);
                        mbar_arrive_expect_tx(fb, ((n < P.n ? 1 : 0) + (n >= 1 ? 1 : 0)) * C::kTileBytes);
                        if (n < P.n)
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_3d(smem_base + C::kOffK + u * C::kTileBytes + c * C::kChunkBytes, &tm_k, fb,
                                            c * 64, P.block(n) * kBN, bh_kv);
                        if (n >= 1)
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_3d(smem_base + C::kOffV + u * C::kTileBytes + c * C::kChunkBytes, &tm_v, fb,
                                            c * 64, P.block(n - 1) * kBN, bh_kv);
                    }
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                // the last Q and the newest bundle of every slot have landed before exit
                if (kq > 0) mbar_wait(qf, (kq - 1) & 1, kDrainWaitNs, &never);
                for (int n = max(0, gb - kStages); n < gb; ++n)
                    mbar_wait(smem_u32(&bars.kv_full[n % kStages]), (n / kStages) & 1, kDrainWaitNs, &never);
            }
        } else if (warp == 1) {
            // ============================================================ MMA issuer
            if (lane == 0) {
                constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
                const uint32_t q_lo = sdesc_sw128_lo(smem_base + C::kOffQ, 16);
                const uint32_t k_lo = sdesc_sw128_lo(smem_base + C::kOffK, 16);
                const uint32_t v_lo = sdesc_sw128_lo(smem_base + C::kOffV, C::kChunkBytes);
                // S_t = Q_t K^T of the block in slot u
                auto issue_s = [&](int t, int u, uint32_t idesc) {
                    const uint32_t ql = q_lo + t * (C::kTileBytes >> 4), kl = k_lo + u * (C::kTileBytes >> 4);
                    const uint32_t col = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off16 = ((kk * 32) / 128 * C::kChunkBytes + (kk * 32) % 128) >> 4;
                        if (kk == 0)
                            mma_ss_w<false, -1>(col, ql, kl, kDescHi, idesc, 0u);
                        else
                            mma_ss_w<false, 1>(col, ql + off16, kl + off16, kDescHi, idesc);
                    }
                    mma_commit(smem_u32(&bars.s_full[t]));
                };
                // O_t += P_t V of the block in slot u, over `steps` K steps of 16 keys
                auto issue_pv = [&](int t, int u, bool acc, auto steps_c) {
                    constexpr int kSteps = decltype(steps_c)::value;
                    const uint32_t vl = v_lo + u * (C::kTileBytes >> 4);
                    const uint32_t colO = tmem + (t ? C::kColO1 : C::kColO0), colP = tmem + (t ? C::kColS1 : C::kColS0);
#pragma unroll
                    for (int kk = 0; kk < kSteps; ++kk) {
                        if (kk == 0)
                            mma_ts_w<false, -1>(colO, colP, vl, kDescHi, C::kIdescO, acc ? 1u : 0u);
                        else
                            mma_ts_w<false, 1>(colO, colP + kk * 8, vl + ((kk * 16 * 128) >> 4), kDescHi, C::kIdescO);
                    }
                };
                using Full = std::integral_constant<int, kBN / 16>;
                using Short = std::integral_constant<int, kShort / 16>;
                int gb = 0, kq = 0;
                int cnt[2] = {0, 0};  // blocks of each tile whose P V was issued, over all items
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    const int x = item_x(k);
                    if (x >= n_items) break;
                    const Plan P = plan_of(args, item_r0(x));
                    ok = mbar_wait(smem_u32(&bars.q_full), kq & 1, lim, &abort_flag);
                    if (ok) ok = mbar_wait(smem_u32(&bars.kv_full[gb % kStages]), (gb / kStages) & 1, lim, &abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const int u0 = gb % kStages;
                    const uint32_t id0 = P.shorty ? C::kIdescShort : C::kIdescS;
                    if (P.active(0, 0)) issue_s(0, u0, id0);
                    if (P.active(1, 0)) issue_s(1, u0, id0);
                    if (P.n == 1) mma_commit(smem_u32(&bars.q_free));
                    mma_commit(smem_u32(&bars.kv_empty[u0]));
                    bool acc0 = false, acc1 = false;
                    for (int n = 1; ok && n <= P.n; ++n) {
                        const int g = gb + n, u = g % kStages;
                        ok = mbar_wait(smem_u32(&bars.kv_full[u]), (g / kStages) & 1, lim, &abort_flag);
                        if (!ok) break;
                        const bool more = n < P.n;
                        const bool pv0 = P.active(0, n - 1), pv1 = P.active(1, n - 1);
                        const bool s0 = more && P.active(0, n), s1 = more && P.active(1, n);
                        const bool shorty = P.shorty && n == 1;  // the P V of a short block
                        if (pv0 && pv1 && s0 && s1 && !shorty && n + 1 < P.n) {
                            // inside: both tiles, P V then the next scores
                            ok = mbar_wait(smem_u32(&bars.p_full[0]), cnt[0] & 1, lim, &abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            issue_pv(0, u, acc0, Full{});
                            issue_s(0, u, C::kIdescS);
                            ok = mbar_wait(smem_u32(&bars.p_full[1]), cnt[1] & 1, lim, &abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            issue_pv(1, u, acc1, Full{});
                            issue_s(1, u, C::kIdescS);
                            acc0 = acc1 = true;
                            ++cnt[0];
                            ++cnt[1];
                        } else {
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                const bool pv = t ? pv1 : pv0, s = t ? s1 : s0;
                                bool& acc = t ? acc1 : acc0;
                                if (pv) {
                                    ok = mbar_wait(smem_u32(&bars.p_full[t]), cnt[t] & 1, lim, &abort_flag);
                                    if (!ok) break;
                                    tc_fence_after();
                                    if (shorty)
                                        issue_pv(t, u, acc, Short{});
                                    else
                                        issue_pv(t, u, acc, Full{});
                                    acc = true;
                                    ++cnt[t];
                                    // the tile's last entry: the item's last, or tile 0's one before it
                                    if (n == P.n || (t == 0 && P.two && n == P.n - 1))
                                        mma_commit(smem_u32(&bars.o_done[t]));
                                }
                                if (s) {
                                    tc_fence_after();
                                    issue_s(t, u, C::kIdescS);
                                }
                            }
                            if (!ok) break;
                            if (n == P.n - 1) mma_commit(smem_u32(&bars.q_free));  // the item's last scores
                        }
                        mma_commit(smem_u32(&bars.kv_empty[u]));
                    }
                    gb += P.n + 1;
                    ++kq;
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                mma_commit(smem_u32(&bars.drain));
                const volatile int never = 0;
                mbar_wait(smem_u32(&bars.drain), 0, kDrainWaitNs, &never);
            }
        }
        // warps 2-3 have no role
    } else {
        regs_inc<184>();
        // ================================================================ softmax warpgroups
        const int t = (warp - 4) / 4;
        const int wq = warp % 4;
        const int row_in_tile = wq * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t colS = t ? C::kColS1 : C::kColS0;
        const uint32_t colO = t ? C::kColO1 : C::kColO0;
        const float c = args.c_log2;
        const bool c_pos = c >= 0.f;
        const uint32_t mask_bits = c_pos ? 0xff800000u : 0x7f800000u;  // -inf after the multiply by c
        int gj = 0;  // blocks of this tile before the current item
        int kd = 0;  // items of this tile
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int x = item_x(k);
            if (x >= n_items) break;
            const int bh = item_bh(x), r0 = item_r0(x);
            const Plan P = plan_of(args, r0);
            if (t == 1 && !P.two) continue;
            const int qrow = r0 + t * kBM + row_in_tile;
            float m_ref = -INFINITY, l = 0.f;
            bool first = true;
            for (int n = 0; n < P.n; ++n) {
                if (!P.active(t, n)) continue;
                ok = mbar_wait(smem_u32(&bars.s_full[t]), gj & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const int kv0 = P.block(n) * kBN;
                // the row's bounds within the block (a window beyond the row's start: none)
                const int hi = qrow - kv0;
                const int lo = static_cast<int>(max(-1ll, static_cast<long long>(hi) - args.window + 1));
                const int sink = args.sinks - kv0;
                if (n == 0 && P.shorty)
                    softmax_block<D, kShort>(lane_base, colS, colO, c, c_pos, mask_bits, hi, lo, sink, first, m_ref, l);
                else
                    softmax_block<D, kBN>(lane_base, colS, colO, c, c_pos, mask_bits, hi, lo, sink, first, m_ref, l);
                first = false;
                ++gj;
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.p_full[t]));
            }
            if (ok) {
                ok = mbar_wait(smem_u32(&bars.o_done[t]), kd & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                ++kd;
            }
            if (!ok) {
                if (lane == 0) record_timeout(args.ctl, &abort_flag);
                break;
            }
            tc_fence_after();
            // O_t is read before this warp publishes the next item's first P, so the next item's
            // first P V (which overwrites O_t) comes after these loads
            const float inv = 1.f / l;
            // The warp's 32 rows go out 64 columns at a time: each lane writes its row's 128 bytes
            // into the warp's own 4 KB (16-byte granule g of row r at g ^ (r % 8)), one lane stores
            // the box, and the next box waits until that has been read.  Rows past N are not
            // written by the store.  (Each lane storing its row itself: 32 lines an instruction,
            // in the way of the warps' next TMEM loads.)
            const uint32_t box = smem_base + C::kOffO + (warp - 4) * 4096;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t ov[2][32];
                tmem_ld32_async(lane_base + colO + 64 * c, ov[0]);
                tmem_ld32_async(lane_base + colO + 64 * c + 32, ov[1]);
                tmem_wait_ld();
                reg_fence(ov[0]);
                reg_fence(ov[1]);
                if (lane == 0) bulk_wait_read_all();
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const uint32_t* f = ov[g / 4] + 8 * (g % 4);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 128 + ((g ^ (lane & 7)) << 4)),
                                 "r"(pack_bf16x2(__uint_as_float(f[0]) * inv, __uint_as_float(f[1]) * inv)),
                                 "r"(pack_bf16x2(__uint_as_float(f[2]) * inv, __uint_as_float(f[3]) * inv)),
                                 "r"(pack_bf16x2(__uint_as_float(f[4]) * inv, __uint_as_float(f[5]) * inv)),
                                 "r"(pack_bf16x2(__uint_as_float(f[6]) * inv, __uint_as_float(f[7]) * inv))
                                 : "memory");
                }
                fence_proxy_async_smem();  // the lanes' writes -> visible to the TMA unit
                __syncwarp();
                const int row0 = r0 + t * kBM + wq * 32;
                if (lane == 0 && row0 < N) {
                    tma_store_3d(&tm_o, box, 64 * c, row0, bh);
                    bulk_commit_group();
                }
            }
            if (qrow < N && args.lse != nullptr)
                args.lse[static_cast<size_t>(bh) * N + qrow] = (m_ref + log2f(l)) * 0.69314718055994530942f;
        }
        // the stores complete before the CTA's shared memory goes away
        if (lane == 0) bulk_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int D>
int launch_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv, int N,
                float c_log2, int window, int sinks, DevCtl ctl, cudaStream_t s) {
    using C = Cfg<D>;
    const int BH = B * H, BH_kv = B * H_kv;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap tq, tk, tv, to;
    int rc = make_map_3d(&tq, q, dt, 2, D, N, BH, 64, kBM);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, D, N, BH_kv, 64, kBN);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, D, N, BH_kv, 64, kBN);
    if (rc == 0) rc = make_map_3d(&to, o, dt, 2, D, N, BH, 64, 32);
    if (rc != 0) return rc;
    int dev = 0, sms = 152;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    static std::atomic<uint64_t> smem_done;
    if (e == cudaSuccess) e = allow_smem(win_fwd_kernel<D>, C::kSmemAlloc, smem_done);
    if (e != cudaSuccess) return static_cast<int>(e);
    WinArgs a;
    a.lse = lse;
    a.N = N;
    a.n_pairs = (N + 2 * kBM - 1) / (2 * kBM);
    a.BH = BH;
    a.n_items = a.n_pairs * BH;
    a.window = window;
    a.sinks = sinks < N ? sinks : N;
    // a scale of 0 makes all scores 0; the mask multiplies -inf by c, which has to stay -inf
    a.c_log2 = c_log2 == 0.f ? 1e-30f : c_log2;
    a.H = H;
    a.H_kv = H_kv;
    a.ctl = ctl;
    const int grid = a.n_items < sms ? a.n_items : sms;
    return static_cast<int>(
        launch_pdl(win_fwd_kernel<D>, dim3(grid), dim3(kThreads), C::kSmemAlloc, s, tq, tk, tv, to, a));
}

}  // namespace

int launch_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv, int N,
                      int d, float c_log2, int window, int sinks, DevCtl ctl, cudaStream_t s) {
    if (d == 64) return launch_impl<64>(q, k, v, o, lse, B, H, H_kv, N, c_log2, window, sinks, ctl, s);
    return launch_impl<128>(q, k, v, o, lse, B, H, H_kv, N, c_log2, window, sinks, ctl, s);
}

}  // namespace fa
