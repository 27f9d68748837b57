// win_bwd_sm103.cu -- backward of attention under a causal sliding window with sinks, by
// recomputation on the sm_103a tensor core.
//
// The mathematics are the plain backward's (bwd_sm103.cu), over the pairs (i, j) that the
// forward saw, j <= i and (j > i - W or j < S):
//     P_ij = exp(S_ij - lse_i),  dV = P^T dO,  dP = dO V^T,  delta_i = dO_i . O_i,
//     dS = P o (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q.
//
// Kernels on one stream: win_bwd_prep (delta and padded -lse log2 e), the main kernel (dK and dV in
// TMEM per 128-key block: here for d = 128, win_bwd64_sm103.cu for d = 64), and a query-parallel
// kernel for dQ (win_bwd_dq_sm103.cu), which also joins the sinks' parts.  Nothing is summed by
// atomics: the same bits every time.  (For d = 64 the plain backward's scheme, dQ partials added to a
// float32 accumulator by TMA reductions, was also measured: the main kernel took 79 us of a B4 H16
// N2048 W512 step, zeroing and converting the accumulator 13 more; dK/dV and dQ take 52 and 42.)
//
// What the window changes:
//   * A key block j meets the query blocks j .. j + (W + 126) / 128 only.
//   * A block that holds sinks meets all later query blocks too: N / 128 of them where the
//     others meet W / 128, so that one CTA would still be at it long after the rest are done.
//     Its later query blocks are dealt in pieces, as items of their own, first of all; the
//     pieces of a block leave float32 dK and dV in the workspace, and an idle warp of the dQ
//     kernel adds them in order and rounds once.
//   * The visible queries of a key row are a range; blocks that hold its ends take them as
//     bit words made by shifts.
//   * dS is taken from P before its rounding to bf16: with P rounded first, dQ and dK carried two
//     bf16 roundings before their own.
//
// The d = 128 main kernel: S^T, dP^T, dV and dK fill TMEM, P^T and dS^T are written over S^T and
// dP^T, and roles and the order of MMAs are the plain backward's.  Q and dO have rings of their own,
// and the issuing thread waits for the next Q behind dV and for the next dO behind dK: with both under
// one barrier, in front of dV, it waited 530 of a pair's 2800 cycles for them.  Measured (N8191 W1024,
// 16 sinks, H16 H_kv4): 110 us, 2640 cycles a pair of blocks inside an item, of which the tensor pipe
// works 2152.
#include <type_traits>

#include "win_bwd.cuh"

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

__global__ void __launch_bounds__(kThreads, 1)
    win_bwd_main_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                        const BwdArgs args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Bars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const sb_ptr = smem_raw + (sb - smem_u32(smem_raw));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int N = args.N, Np = args.Np;
    // Persistent: every role computes this CTA's sequence of items on its own and passes over those
    // without query blocks (a later sink block has fewer pieces); query blocks are numbered
    // g = 0, 1, 2, ... across items: stages and barrier phases follow g, the K/V tile and the
    // dK/dV accumulators follow the count of items done.
    const int n_items = far_items(args) + args.n_kv * args.BH;
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

    if (warp == 0) {
        // ================================================================ Q / dO producer
        // The rings run across item boundaries: they wait only for their own stages.  A stage of dO is
        // free after dV, one of Q (with lse and delta) after dK.
        if (lane == 0) {
            int g = 0, nq = 0, ndo = 0;  // pairs; Q, dO loads issued
            bool ok = true;
            for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
                const Item I = item_at(args, x);
                Walk at(args, I);
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
                const Item I = item_at(args, x);
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
                const Item I = item_at(args, x);
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
            const Item I = item_at(args, x);
            if (I.n_it == 0) continue;
            const int key = I.kvb * kBlk + key_in_blk;
            Walk at(args, I);
            for (int i = 0; i < I.n_it; ++i, at.next()) {
                const int gi = g + i, s = gi % kQStages;
                int q_first, q_end;
                query_range(args.split, key, at.blk * kBlk + 64 * half, q_first, q_end);
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
                write_part_row<kD>(args, I, half, key_in_blk, lb + col);
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

// ---------------------------------------------------------------- pre / post passes
// -delta_i and -lse_i * log2(e) (rows past N: 0 and -inf, so that recomputed P is exactly 0 there).
// Both are stored negated so the main kernels add them with packed FMA/FADD.  D / 8 threads per row.
//
// delta_i = dO_i . O_i takes the O that the forward rounded to bf16, which is off by up to 2^-8 |O| |dO|
// beside dP's spread: little against dS's own rounding where many keys average out in O, as much as
// it at four keys.  A head's first kFirst rows, which see kFirst keys at most and have the largest
// gradients, take delta_i = sum_j P_ij dP_ij instead, in `extra` CTAs beside the others, a warp a row
// (dQ's error relative to 64 bits, N1024 W512 d64: 2.54e-3 -> 2.46e-3 for 1% of a step).  So do all rows
// of sequences of up to kShort, and under a window and sinks of up to kNarrow keys in all, in a kernel
// of their own.
constexpr int kFirst = 16, kNarrow = 24, kShort = 128;

struct PrepArgs {
    const uint4 *o, *dO, *q, *k, *v;
    const float* lse;
    float *ws_delta, *ws_lse2;
    int BH, H, H_kv, N, Np;
    int window, sinks;
    float c_log2;
    int extra;
};

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

// sum_j P_ij dP_ij of row i < min(N, kFirst) of query head bh, by one warp: D / 8 lanes a key, two
// such rounds of keys at a time.
template <int D>
__device__ __forceinline__ float delta_of_first(const PrepArgs& a, int bh, int i) {
    constexpr int kT = D / 8, kSlots = 32 / kT;
    const int lane = threadIdx.x % 32, part = lane % kT;
    const int lo = max(0, static_cast<int>(max(-1ll, static_cast<long long>(i) - a.window + 1)));
    const int front = min(a.sinks, lo), n = front + i - lo + 1;  // sinks in front of the window; keys
    const size_t row = static_cast<size_t>(bh) * a.N + i;
    const size_t kv = static_cast<size_t>((bh / a.H) * a.H_kv + (bh % a.H) / (a.H / a.H_kv)) * a.N;
    const uint4 q = a.q[row * kT + part], d = a.dO[row * kT + part], zero = make_uint4(0, 0, 0, 0);
    const float nl = -a.lse[row] * kLog2e;
    float delta = 0.f;
    for (int t = lane / kT; t - lane / kT < n; t += 2 * kSlots) {
        uint4 k[2], v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int x = t + u * kSlots;
            const size_t at = (kv + (x < front ? x : lo + x - front)) * kT + part;
            k[u] = x < n ? a.k[at] : zero;
            v[u] = x < n ? a.v[at] : zero;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float p = ex2_approx(fmaf(lanes_sum<1, kT>(dot8(q, k[u])), a.c_log2, nl));
            const float dp = lanes_sum<1, kT>(dot8(d, v[u]));
            if (t + u * kSlots < n) delta = fmaf(p, dp, delta);
        }
    }
    return lanes_sum<kT, 32>(delta);
}

template <int D>
__global__ void __launch_bounds__(256, 8) win_bwd_prep_kernel(const PrepArgs a) {
    griddep_wait();               // O, dO may come from the kernel before this one
    griddep_launch_dependents();  // the main kernel may launch and set up meanwhile
    constexpr int kT = D / 8;     // threads per row (8 or 16): the shuffles stay inside a warp
    const int N = a.N, Np = a.Np, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (static_cast<int>(blockIdx.x) < a.extra) {
        const long long rows = static_cast<long long>(a.BH) * kFirst, step = a.extra * 8;
        for (long long r = blockIdx.x * 8 + warp; r < rows; r += step) {
            const int bh = static_cast<int>(r / kFirst), i = static_cast<int>(r % kFirst);
            if (i >= N) continue;
            const float delta = delta_of_first<D>(a, bh, i);
            if (lane == 0) a.ws_delta[static_cast<size_t>(bh) * Np + i] = -delta;
        }
        return;
    }
    const int part = lane % kT;
    const size_t tid = static_cast<size_t>(blockIdx.x - a.extra) * blockDim.x + threadIdx.x;
    const size_t nthreads = static_cast<size_t>(gridDim.x - a.extra) * blockDim.x;
    const size_t rows = static_cast<size_t>(a.BH) * Np;
    for (size_t base = tid; base < rows * kT; base += nthreads) {
        const size_t r = base / kT;
        const int bh = static_cast<int>(r / Np), i = static_cast<int>(r % Np);
        float sum = 0.f;
        if (i < N) {
            const size_t src = (static_cast<size_t>(bh) * N + i) * kT + part;
            sum = dot8(a.o[src], a.dO[src]);
        }
        sum = lanes_sum<1, kT>(sum);
        if (part == 0) {
            if (i >= N || i >= kFirst) a.ws_delta[r] = -sum;
            a.ws_lse2[r] = (i < N) ? -a.lse[static_cast<size_t>(bh) * N + i] * kLog2e : -INFINITY;
        }
    }
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same rows of the workspace for few keys: delta_i = sum_j P_ij dP_ij.  A warp takes 16
// query rows with the keys that any of them sees, eight at a time: S and dP as m16n8k16 products of
// the same layout, multiplied element by element.  Against dO . o, a step of B4 H16 N2048 d64: W2 83 ->
// 92 us and dQ's error 3.8e-3 -> 2.35e-3, W16 84 -> 95 and 2.5e-3 -> 2.34e-3 (W32 84 -> 100 and 2.48e-3 ->
// 2.36e-3, hence kNarrow).  The order of d in a product is free, so that a lane
// (row or key g, t) loads its operands as 16 neighbouring bytes: values 32 c + 8 t .. + 7, of which the
// first four serve one product and the rest the next.  Bound by memory: q, k, v and dO are read here
// (and by the kernels after this one, from L2) where the other kernel reads o and dO.
template <int D>
__global__ void __launch_bounds__(256) win_bwd_narrow_prep_kernel(const PrepArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kC = D / 32, kT = D / 8;  // 16-byte loads of a lane and of a row
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int N = a.N, Np = a.Np, tiles_head = Np / 16;
    const long long tiles = static_cast<long long>(a.BH) * tiles_head;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (long long x = static_cast<long long>(blockIdx.x) * 8 + warp; x < tiles; x += static_cast<long long>(gridDim.x) * 8) {
        const int bh = static_cast<int>(x / tiles_head), i0 = static_cast<int>(x % tiles_head) * 16;
        const size_t q_row = static_cast<size_t>(bh) * N;
        const size_t k_row = static_cast<size_t>((bh / a.H) * a.H_kv + (bh % a.H) / (a.H / a.H_kv)) * N;
        uint4 q[2][kC], d[2][kC];  // rows i0 + g, i0 + g + 8
        float nl[2], delta[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = i0 + g + 8 * r;
            const size_t at = (q_row + i) * kT + t;
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                q[r][c] = i < N ? a.q[at + 4 * c] : zero;
                d[r][c] = i < N ? a.dO[at + 4 * c] : zero;
            }
            nl[r] = i < N ? -a.lse[q_row + i] * kLog2e : -INFINITY;
        }
        const int start = max(0, i0 - a.window + 1) & ~7, end = min(i0 + 16, N);  // the window's keys
        const int front = min(a.sinks, start);                                    // sinks before them
        for (int kt = front > 0 ? 0 : start; kt < end; kt = kt < front && kt + 8 >= front ? start : kt + 8) {
            const bool of_front = kt < front;
            const int key = kt + g;  // this lane's
            const bool there = key < N;
            const size_t at = (k_row + key) * kT + t;
            float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kC; ++c) {
                const uint4 k = there ? a.k[at + 4 * c] : zero, v = there ? a.v[at + 4 * c] : zero;
                mma_bf16(s, q[0][c].x, q[1][c].x, q[0][c].y, q[1][c].y, k.x, k.y);
                mma_bf16(s, q[0][c].z, q[1][c].z, q[0][c].w, q[1][c].w, k.z, k.w);
                mma_bf16(dp, d[0][c].x, d[1][c].x, d[0][c].y, d[1][c].y, v.x, v.y);
                mma_bf16(dp, d[0][c].z, d[1][c].z, d[0][c].w, d[1][c].w, v.z, v.w);
            }
            // rows g, g + 8 and keys 2 t, 2 t + 1
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + g + 8 * (e / 2), j = kt + 2 * t + e % 2;
                const bool seen = of_front ? j < front : j <= i && (j > i - a.window || j < a.sinks);
                if (seen) delta[e / 2] = fmaf(ex2_approx(fmaf(s[e], a.c_log2, nl[e / 2])), dp[e], delta[e / 2]);
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
}

int grid_for(size_t work, int threads, int max_blocks) {
    size_t b = (work + threads - 1) / threads;
    if (b > static_cast<size_t>(max_blocks)) b = max_blocks;
    return static_cast<int>(b < 1 ? 1 : b);
}

}  // namespace

namespace {

// delta and lse rows in bytes; the parts follow
size_t rows_bytes(int BH, int N) {
    return 2 * static_cast<size_t>(BH) * static_cast<size_t>(round_up(N, kBlk)) * sizeof(float);
}

}  // namespace

// How a sink block's later query blocks are dealt: pieces no shorter than a window's run of
// blocks, at most 64 a block, and together about two per SM, which keeps any one of them
// below the mean load of a CTA (B1 H_kv1 N131072 W1024: 1024 later blocks in 64 pieces of 16
// against 60 blocks a CTA).  Two per SM of 152, whatever the current device: the workspace's size and
// the order of the sums follow from the sizes alone.
WinSplit win_split(int B, int H_kv, int N, int window, int sinks) {
    const int n_q = (N + kBlk - 1) / kBlk;
    WinSplit sp;
    sp.window = window;
    sp.sinks = sinks < N ? sinks : N;
    const long long reach = (static_cast<long long>(window) + kBlk - 2) / kBlk;
    sp.reach = static_cast<int>(reach < n_q - 1 ? reach : n_q - 1);
    const int later = n_q - 1 - sp.reach;  // of block 0; one fewer for each block after it
    const int n_sink = (sp.sinks + kBlk - 1) / kBlk;
    sp.n_part = n_sink < later ? n_sink : later;
    sp.per = 1;
    sp.pieces = 0;
    if (sp.n_part > 0) {
        const long long blocks = static_cast<long long>(B) * H_kv * sp.n_part;
        long long most = (304 + blocks - 1) / blocks;
        if (most > 64) most = 64;
        sp.per = static_cast<int>((later + most - 1) / most);
        if (sp.per < sp.reach + 1) sp.per = sp.reach + 1;
        sp.pieces = (later + sp.per - 1) / sp.per;
    }
    return sp;
}

size_t bwd_window_workspace_bytes(int B, int H, int H_kv, int N, int d, int window, int sinks) {
    const WinSplit sp = win_split(B, H_kv, N, window, sinks);
    return rows_bytes(B * H, N) +
           static_cast<size_t>(B) * H_kv * sp.n_part * (sp.pieces + 1) * 2 * kBlk * d * sizeof(float);
}

int launch_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                      void* dq, void* dk, void* dv, void* workspace, int B, int H, int H_kv, int N, int d, float scale,
                      int window, int sinks, DevCtl ctl, cudaStream_t s) {
    const WinSplit sp = win_split(B, H_kv, N, window, sinks);
    const int BH = B * H, BH_kv = B * H_kv;  // query heads; K/V heads
    const int Np = round_up(N, kBlk);
    float* ws_delta = static_cast<float*>(workspace);
    float* ws_lse2 = ws_delta + static_cast<size_t>(BH) * Np;

    int sms = 152, dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    PrepArgs pa;
    pa.o = static_cast<const uint4*>(o);
    pa.dO = static_cast<const uint4*>(dO);
    pa.q = static_cast<const uint4*>(q);
    pa.k = static_cast<const uint4*>(k);
    pa.v = static_cast<const uint4*>(v);
    pa.lse = lse;
    pa.ws_delta = ws_delta;
    pa.ws_lse2 = ws_lse2;
    pa.BH = BH;
    pa.H = H;
    pa.H_kv = H_kv;
    pa.N = N;
    pa.Np = Np;
    pa.window = window;
    pa.sinks = sp.sinks;
    pa.c_log2 = scale == 0.f ? 1e-30f : scale * kLog2e;
    if (N <= kShort || static_cast<long long>(window) + sp.sinks <= kNarrow) {
        pa.extra = 0;
        e = launch_pdl(d == 64 ? win_bwd_narrow_prep_kernel<64> : win_bwd_narrow_prep_kernel<128>,
                       dim3(grid_for(static_cast<size_t>(BH) * Np / 16, 8, sms * 4)), dim3(256), 0, s, pa);
    } else {
        pa.extra = grid_for(static_cast<size_t>(BH) * kFirst, 8, 2 * sms);
        const int others = grid_for(static_cast<size_t>(BH) * Np * (d / 8), 256, sms * 8 - pa.extra);
        e = launch_pdl(d == 64 ? win_bwd_prep_kernel<64> : win_bwd_prep_kernel<128>, dim3(others + pa.extra), dim3(256), 0,
                       s, pa);
    }
    if (e != cudaSuccess) return static_cast<int>(e);

    CUtensorMap tq, tk, tv, tdo, tdk, tdv;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = make_map_3d(&tq, q, dt, 2, d, N, BH, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, d, N, BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, d, N, BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tdo, dO, dt, 2, d, N, BH, 64, kBlk);
    // d = 64: dK, dV written in boxes of a warp's 32 rows
    if (rc == 0 && d == 64) rc = make_map_3d(&tdk, dk, dt, 2, d, N, BH_kv, 64, 32);
    if (rc == 0 && d == 64) rc = make_map_3d(&tdv, dv, dt, 2, d, N, BH_kv, 64, 32);
    if (rc != 0) return rc;
    BwdArgs a;
    a.ws_delta = ws_delta;
    a.ws_lse2 = ws_lse2;
    a.dk = dk;
    a.dv = dv;
    a.N = N;
    a.Np = Np;
    a.n_kv = Np / kBlk;
    a.BH = BH_kv;
    a.H = H;
    a.H_kv = H_kv;
    a.split = sp;
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + rows_bytes(BH, N));
    a.c_log2 = scale == 0.f ? 1e-30f : scale * kLog2e;  // not 0: the mask multiplies -inf by it
    a.scale = scale;
    a.ctl = ctl;
    // persistent: one CTA per SM (fewer if there are fewer items), each looping over items.  An
    // ordinary launch, as of the causal plain backward: the deal takes it that every CTA
    // starts together.
    const int n_items = (a.n_kv + sp.n_part * sp.pieces) * BH_kv;
    const int grid = n_items < sms ? n_items : sms;
    if (d == 64) {
        e = launch_bwd_window_main64(tq, tk, tv, tdo, tdk, tdv, a, grid, s);
    } else {
        static std::atomic<uint64_t> smem_done;
        e = allow_smem(win_bwd_main_kernel, kSmemAlloc, smem_done);
        if (e != cudaSuccess) return static_cast<int>(e);
        win_bwd_main_kernel<<<grid, kThreads, kSmemAlloc, s>>>(tq, tk, tv, tdo, a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return static_cast<int>(e);
    return launch_bwd_window_dq(q, k, v, dO, dq, a, d, s);
}

}  // namespace fa
