// bwd_main128.cuh -- dK and dV for d = 128, over the blocks that the arguments name (bwd_tile.cuh).
//
// Per key block j (128 keys, TMEM lanes) and query block i (128 queries):
//     S^T = K Q^T,  P^T = exp(S^T - lse),  dV += P^T dO,   dP^T = V dO^T,
//     dS^T = P^T o (dP^T - delta),  dK += dS^T Q.
// S^T, dP^T, dV and dK fill TMEM, P^T and dS^T are written over S^T and
// dP^T, and roles and the order of MMAs are the plain backward's.  Q and dO have rings of their own,
// and the issuing thread waits for the next Q behind dV and for the next dO behind dK: with both under
// one barrier, in front of dV, it waited 530 of a pair's 2800 cycles for them.  Measured (N8191 W1024,
// 16 sinks, H16 H_kv4): 110 us, 2640 cycles a pair of blocks inside an item, of which the tensor pipe
// works 2152.
#pragma once

#include <type_traits>

#include "bwd_tile.cuh"

namespace fa {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 384;
constexpr int kQStages = 2;
constexpr int kChunks = kD / 64;                    // 128-byte swizzle columns per row
constexpr int kTile = kBlk * kD * 2;                // bf16 128 x d tile
// shared memory map (offsets from a 1 KB aligned base)
constexpr int kOffK = 0, kOffV = kTile, kOffQ = 2 * kTile, kOffDO = kOffQ + kQStages * kTile;
constexpr int kOffL = kOffDO + kQStages * kTile;          // kQStages x 512 B
constexpr int kOffDelta = kOffL + kQStages * kBlk * 4;    // kQStages x 512 B
constexpr int kSmemAlloc = kOffDelta + kQStages * kBlk * 4 + 1024;
static_assert(kSmemAlloc <= 232448, "smem");
// TMEM columns
constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescSS = idesc_bf16(128, 128, false, false);  // S^T, dP^T
constexpr uint32_t kIdescTS = idesc_bf16(128, kD, false, true);    // dV, dK

struct Bars {
    uint64_t k_full, k_empty, v_full, v_empty;
    uint64_t q_full[kQStages], q_empty[kQStages], do_full[kQStages], do_empty[kQStages];
    uint64_t s_full, dp_full, p_full;
    uint64_t ds_full[2];  // one per parity, as a waiter may fall one phase behind
    uint64_t all_done, drain;
};

template <class Args>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_main_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const Args args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Bars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const sb_ptr = smem_raw + (sb - smem_u32(smem_raw));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int N = key_rows(args), Np = args.Np;
    // Persistent: every role computes this CTA's sequence of items on its own and passes over those
    // without query blocks (a later sink block has fewer pieces); query blocks are numbered
    // g = 0, 1, 2, ... across items: stages and barrier phases follow g, the K/V tile and the
    // dK/dV accumulators follow the count of items done.
    const int n_items = item_count(args);
    const uint64_t lim = args.ctl.wait_ns;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(smem_u32(&bars.k_full), 1);
        mbar_init(smem_u32(&bars.k_empty), 1);
        mbar_init(smem_u32(&bars.v_full), 1);
        mbar_init(smem_u32(&bars.v_empty), 1);
        for (int s = 0; s < kQStages; ++s) {
            mbar_init(smem_u32(&bars.q_full[s]), 1);
            mbar_init(smem_u32(&bars.q_empty[s]), 1);
            mbar_init(smem_u32(&bars.do_full[s]), 1);
            mbar_init(smem_u32(&bars.do_empty[s]), 1);
        }
        mbar_init(smem_u32(&bars.s_full), 1);
        mbar_init(smem_u32(&bars.dp_full), 1);
        mbar_init(smem_u32(&bars.p_full), 256);
        mbar_init(smem_u32(&bars.ds_full[0]), 256);
        mbar_init(smem_u32(&bars.ds_full[1]), 256);
        mbar_init(smem_u32(&bars.all_done), 1);
        mbar_init(smem_u32(&bars.drain), 1);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_do);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    griddep_wait();               // delta and lse come from the kernel before this one
    griddep_launch_dependents();  // and so may a kernel that needs nothing else start

    if (warp == 0) {
        // ================================================================ Q / dO producer
        // The rings run across item boundaries: they wait only for their own stages.  A stage of dO is
        // free after dV, one of Q (with lse and delta) after dK.
        if (lane == 0) {
            int g = 0, nq = 0, ndo = 0;  // pairs; Q, dO loads issued
            bool ok = true;
            for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
                const auto I = item_at(args, x);
                auto at = walk_of(args, I);
                for (int i = 0; i < I.n_it; ++i, ++g, at.next()) {
                    const int s = g % kQStages;
                    const int qb = at.blk, qh = at.head;
                    const uint32_t par = ((g / kQStages) & 1) ^ 1;
                    if (g >= kQStages && !mbar_wait(smem_u32(&bars.do_empty[s]), par, lim, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t df = smem_u32(&bars.do_full[s]);
                    mbar_arrive_expect_tx(df, kTile);
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_3d(sb + kOffDO + s * kTile + c * 16384, &tm_do, df, 64 * c, qb * kBlk, qh);
                    ndo = g + 1;
                    if (g >= kQStages && !mbar_wait(smem_u32(&bars.q_empty[s]), par, lim, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t qf = smem_u32(&bars.q_full[s]);
                    mbar_arrive_expect_tx(qf, kTile + 2 * kBlk * 4);
                    for (int c = 0; c < kChunks; ++c)
                        tma_load_3d(sb + kOffQ + s * kTile + c * 16384, &tm_q, qf, 64 * c, qb * kBlk, qh);
                    const size_t row = static_cast<size_t>(qh) * Np + static_cast<size_t>(qb) * kBlk;
                    bulk_load(sb + kOffL + s * kBlk * 4, args.ws_lse2 + row, kBlk * 4, qf);
                    bulk_load(sb + kOffDelta + s * kBlk * 4, args.ws_delta + row, kBlk * 4, qf);
                    nq = g + 1;
                }
            }
            if (!ok) record_timeout(args.ctl, &abort_flag);
            // drain: the newest load of every stage has landed
            const volatile int never = 0;
            for (int q = max(0, nq - kQStages); q < nq; ++q)
                mbar_wait(smem_u32(&bars.q_full[q % kQStages]), (q / kQStages) & 1, kDrainWaitNs, &never);
            for (int q = max(0, ndo - kQStages); q < ndo; ++q)
                mbar_wait(smem_u32(&bars.do_full[q % kQStages]), (q / kQStages) & 1, kDrainWaitNs, &never);
        }
    } else if (warp == 3) {
        // ================================================================ K / V producer
        // An item's K goes in once the previous item's last S has read its own, its V once its
        // last dP has.
        if (lane == 0) {
            int kc = 0, v_issued = 0;
            bool ok = true;
            for (int k = 0, x = item_x(0); x < n_items; x = item_x(++k)) {
                const auto I = item_at(args, x);
                if (I.n_it == 0) continue;
                if (kc > 0 && !mbar_wait(smem_u32(&bars.k_empty), (kc - 1) & 1, lim, &abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t kf = smem_u32(&bars.k_full);
                mbar_arrive_expect_tx(kf, kTile);
                for (int c = 0; c < kChunks; ++c)
                    tma_load_3d(sb + kOffK + c * 16384, &tm_k, kf, 64 * c, I.kvb * kBlk, I.bh);
                ++kc;
                if (v_issued > 0 && !mbar_wait(smem_u32(&bars.v_empty), (v_issued - 1) & 1, lim, &abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t vf = smem_u32(&bars.v_full);
                mbar_arrive_expect_tx(vf, kTile);
                for (int c = 0; c < kChunks; ++c)
                    tma_load_3d(sb + kOffV + c * 16384, &tm_v, vf, 64 * c, I.kvb * kBlk, I.bh);
                ++v_issued;
            }
            if (!ok) record_timeout(args.ctl, &abort_flag);
            // drain: the newest K and V loads have landed (also for an item the consumers gave up on)
            const volatile int never = 0;
            if (kc > 0) mbar_wait(smem_u32(&bars.k_full), (kc - 1) & 1, kDrainWaitNs, &never);
            if (v_issued > 0) mbar_wait(smem_u32(&bars.v_full), (v_issued - 1) & 1, kDrainWaitNs, &never);
        }
    } else if (warp == 1) {
        // ================================================================ MMA issuer
        if (lane == 0) {
            // Operand descriptors as low words built once (see sdesc_sw128_lo): K-major
            // (leading byte offset 16) for S^T and dP^T, MN-major (16384) for dV and dK.
            constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
            constexpr uint32_t kStage16 = kTile >> 4;
            const uint32_t k_lo = sdesc_sw128_lo(sb + kOffK, 16), v_lo = sdesc_sw128_lo(sb + kOffV, 16);
            const uint32_t q_lo = sdesc_sw128_lo(sb + kOffQ, 16), q_mn = sdesc_sw128_lo(sb + kOffQ, 16384);
            const uint32_t do_lo = sdesc_sw128_lo(sb + kOffDO, 16), do_mn = sdesc_sw128_lo(sb + kOffDO, 16384);
            // S^T = K_j Q^T or dP^T = V_j dO^T of the block in stage s
            auto issue_ss = [&](uint32_t col, uint32_t a_lo, uint32_t b_lo, int s, uint64_t& bar) {
                const uint32_t bl = b_lo + s * kStage16;
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk) {
                    const uint32_t off16 = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                    if (kk == 0)
                        mma_ss_w<false, -1>(tmem + col, a_lo, bl, kDescHi, kIdescSS, 0u);
                    else
                        mma_ss_w<false, 1>(tmem + col, a_lo + off16, bl + off16, kDescHi, kIdescSS);
                }
                mma_commit(smem_u32(&bar));
            };
            // dV += P^T dO or dK += dS^T Q: A from the two halves of S^T's or dP^T's columns
            auto issue_ts = [&](uint32_t col, uint32_t colA, uint32_t b_mn, bool acc) {
#pragma unroll
                for (int kk = 0; kk < kBlk / 16; ++kk) {
                    if (kk == 0)
                        mma_ts_w<false, -1>(tmem + col, tmem + colA, b_mn, kDescHi, kIdescTS, acc ? 1u : 0u);
                    else
                        mma_ts_w<false, 1>(tmem + col, tmem + colA + 64 * (kk >> 2) + 8 * (kk & 3), b_mn + 128 * kk,
                                           kDescHi, kIdescTS);
                }
            };
            int g = 0, kc = 0;
            bool ok = true;
            for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
                const auto I = item_at(args, x);
                if (I.n_it == 0) continue;
                // the item's first scores; S and dP of the previous item's last block were read by
                // its dV and dK, issued before these by this thread
                ok = mbar_wait(smem_u32(&bars.k_full), kc & 1, lim, &abort_flag);
                if (ok) ok = mbar_wait(smem_u32(&bars.q_full[g % kQStages]), (g / kQStages) & 1, lim, &abort_flag);
                if (!ok) break;
                tc_fence_after();
                issue_ss(kColS, k_lo, q_lo, g % kQStages, bars.s_full);
                if (I.n_it == 1) mma_commit(smem_u32(&bars.k_empty));
                ok = mbar_wait(smem_u32(&bars.v_full), kc & 1, lim, &abort_flag);
                if (ok) ok = mbar_wait(smem_u32(&bars.do_full[g % kQStages]), (g / kQStages) & 1, lim, &abort_flag);
                if (!ok) break;
                tc_fence_after();
                issue_ss(kColDP, v_lo, do_lo, g % kQStages, bars.dp_full);
                if (I.n_it == 1) mma_commit(smem_u32(&bars.v_empty));
                // One query block: dV_i, the next block's S, dK_i, the next block's dP.  MORE: a
                // next block exists; LAST2: it is the item's last, so this block issues the item's
                // last S and dP and releases K and V after them.  Both compile-time: the item's
                // last two blocks run outside the loop, which keeps its body free of the release
                // commits.
                auto block = [&](int i, auto more_c, auto last2_c) -> bool {
                    constexpr bool more = decltype(more_c)::value, last2 = decltype(last2_c)::value;
                    const int gi = g + i, s = gi % kQStages, s1 = (gi + 1) % kQStages;
                    // P of an item's first block is computed after the P/dS warps have read the
                    // previous item's dV and dK, so dV, dK may then be overwritten
                    const uint32_t par1 = ((gi + 1) / kQStages) & 1;
                    if (!mbar_wait(smem_u32(&bars.p_full), gi & 1, lim, &abort_flag)) return false;
                    tc_fence_after();
                    issue_ts(kColDV, kColS, do_mn + s * kStage16, i > 0);
                    mma_commit(smem_u32(&bars.do_empty[s]));
                    if constexpr (more) {  // the P/dS warps keep P_i in registers
                        if (!mbar_wait(smem_u32(&bars.q_full[s1]), par1, lim, &abort_flag)) return false;
                        tc_fence_after();
                        issue_ss(kColS, k_lo, q_lo, s1, bars.s_full);
                        if constexpr (last2) mma_commit(smem_u32(&bars.k_empty));
                    }
                    if (!mbar_wait(smem_u32(&bars.ds_full[gi & 1]), (gi >> 1) & 1, lim, &abort_flag)) return false;
                    if (more && !mbar_wait(smem_u32(&bars.do_full[s1]), par1, lim, &abort_flag)) return false;
                    tc_fence_after();
                    issue_ts(kColDK, kColDP, q_mn + s * kStage16, i > 0);
                    mma_commit(smem_u32(&bars.q_empty[s]));  // Q_i, lse_i, delta_i consumed
                    if constexpr (more) {
                        issue_ss(kColDP, v_lo, do_lo, s1, bars.dp_full);
                        if constexpr (last2) mma_commit(smem_u32(&bars.v_empty));
                    }
                    return true;
                };
                using T = std::true_type;
                using F = std::false_type;
                int i = 0;
                for (; i + 2 < I.n_it && ok; ++i) ok = block(i, T{}, F{});
                if (ok && I.n_it >= 2) ok = block(I.n_it - 2, T{}, T{});
                if (ok) ok = block(I.n_it - 1, F{}, F{});
                if (!ok) break;
                mma_commit(smem_u32(&bars.all_done));  // the item's dV, dK are complete
                g += I.n_it;
                ++kc;
            }
            if (!ok) record_timeout(args.ctl, &abort_flag);
            mma_commit(smem_u32(&bars.drain));
            const volatile int never = 0;
            mbar_wait(smem_u32(&bars.drain), 0, kDrainWaitNs, &never);
        }
    } else if (warp >= 4) {
        // ================================================================ P / dS warpgroups
        const int half = (warp - 4) / 4;          // query columns 64*half .. 64*half+63
        const int wq = warp % 4;
        const int key_in_blk = wq * 32 + lane;
        const uint32_t lb = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float2 c2 = make_float2(args.c_log2, args.c_log2);
        const uint32_t hide = args.c_log2 >= 0.f ? 0xff800000u : 0x7f800000u;  // -inf after the multiply by c
        bool ok = true;
        int g = 0, kc = 0;
        for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
            const auto I = item_at(args, x);
            if (I.n_it == 0) continue;
            const int key = I.kvb * kBlk + key_in_blk;
            auto at = walk_of(args, I);
            for (int i = 0; i < I.n_it; ++i, at.next()) {
                const int gi = g + i, s = gi % kQStages;
                int q_first, q_end;
                query_range(args, I, key, at.blk * kBlk + 64 * half, q_first, q_end);
                ok = mbar_wait(smem_u32(&bars.q_full[s]), (gi / kQStages) & 1, lim, &abort_flag);
                if (ok) ok = mbar_wait(smem_u32(&bars.s_full), gi & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                // -lse_i * log2(e) and -delta_i of this block's 64 queries
                const float4* nl = reinterpret_cast<const float4*>(sb_ptr + kOffL + s * kBlk * 4) + 16 * half;
                const float4* nd = reinterpret_cast<const float4*>(sb_ptr + kOffDelta + s * kBlk * 4) + 16 * half;
                uint32_t p[2][32], pk[32];  // scores, then P^T
                tmem_ld32_async(lb + kColS + 64 * half, p[0]);
                tmem_ld32_async(lb + kColS + 64 * half + 32, p[1]);
                tmem_wait_ld();
                reg_fence(p[0]);
                reg_fence(p[1]);
                probabilities(p, q_first, q_end, hide, c2, nl, pk);
                // P^T of this half goes inside the columns this half read (the other half's
                // scores may still be unread): queries 64h..64h+63 -> columns 64h..64h+31
                tmem_st32(lb + kColS + 64 * half, pk);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.p_full));

                // dS^T = P^T o (dP^T - delta)
                ok = mbar_wait(smem_u32(&bars.dp_full), gi & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                // in two 32-column loads; the second runs while the first 32 queries' dS is stored
                uint32_t r[32];
                tmem_ld32_async(lb + kColDP + 64 * half, r);
                tmem_wait_ld();
                reg_fence(r);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[16];
                    if (hides(args) && q_end <= 0) {  // a hidden key's dP may be anything: no gradient
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = 0u;
                    }
                    score_gradients(p[h], r, nd + 8 * h, w);
                    if (h == 0) tmem_ld32_async(lb + kColDP + 64 * half + 32, r);
                    tmem_st16(lb + kColDP + 64 * half + 16 * h, w);
                    if (h == 0) {
                        tmem_wait_ld();
                        reg_fence(r);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.ds_full[gi & 1]));
            }
            if (!ok) break;
            // epilogue: warps 4-7 store dV, warps 8-11 dK (times scale).  Their TMEM reads finish
            // before these warps compute the next item's first P.
            ok = mbar_wait(smem_u32(&bars.all_done), kc & 1, lim, &abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t col = half ? kColDK : kColDV;
            if (I.slot >= 0) {
                write_part_row<kD>(args.part, 2 * part_of(args, I) + half, key_in_blk, key < N, lb + col);
            } else {
                RowsOut<kD> rows;
                rows.load(lb + col, half ? args.scale : 1.0f);
                rows.store(half ? args.dk : args.dv, static_cast<size_t>(I.bh) * N, I.kvb * kBlk + wq * 32, N);
            }
            tc_fence_before();
            g += I.n_it;
            ++kc;
        }
        if (!ok && lane == 0) record_timeout(args.ctl, &abort_flag);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace
}  // namespace fa
