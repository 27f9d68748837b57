// win_bwd64_sm103.cu -- dK and dV of the windowed backward for d = 64.
//
// Per key block j (128 keys, TMEM lanes) and query block i (128 queries):
//     S^T = K Q^T,  P^T = exp(S^T - lse),  dV += P^T dO,   dP^T = V dO^T,
//     dS^T = P^T o (dP^T - delta),  dK += dS^T Q.
// At d = 64 the four products are 24 MMAs, 1076 cycles of the tensor pipe, and everything around
// them longer: the plain backward's schedule, with P^T and dS^T written over S^T and dP^T, runs
// S, P, dV, dP, dS, dK of a pair mostly one after the other (4400 cycles a pair in items of five).
// TMEM has room for more: S^T and dP^T (128 columns each), P^T, dS^T, dV and dK (64 each) are all 512.
//   * The tensor core goes on with the next pair's S^T and dP^T as soon as the P/dS warps have this
//     pair's in registers.
//   * Two issuing threads: S^T and dP^T in one, dV and dK in the other; neither writes columns that
//     the other's MMAs read or write.
//   * A warpgroup of its own takes an item's dV and dK out, through shared memory and TMA stores, or
//     as float32 parts to the workspace; the next item's MMAs wait for its TMEM loads only.
//   * K and V have two buffers, for the next item's loads.
//
//   * Four warpgroups on P and dS, 32 queries each: two of 64 took 2450 cycles a pair at half of the
//     issue slots and exponentials that they could have had.  Four take 2100: loads, exponentials and
//     stores of the sixteen warps run in step.  (Publishing P behind the load of dP, or dS behind the
//     next scores' load, changed nothing.)  Measured (B4 H16 N2048 W512, 4 sinks): 52 us.
//
// Warp 0 TMA for Q, dO, lse, delta (three stages), warp 3 TMA for K, V, warps 1 and 2 MMA, warps 4-19 P
// and dS (thread = key), warps 20-23 dV and dK out.
#include "win_bwd.cuh"

namespace fa {
namespace {

constexpr int kD = 64;
constexpr int kPdsThreads = 512;
constexpr int kThreads = 256 + kPdsThreads;
constexpr int kQStages = 3;
constexpr int kTile = kBlk * kD * 2;
constexpr int kOffK = 0, kOffV = 2 * kTile, kOffQ = 4 * kTile, kOffDO = kOffQ + kQStages * kTile;
constexpr int kOffOut = kOffDO + kQStages * kTile;           // dV, dK of a warp's 32 rows: 4 x 8 KB
constexpr int kOffL = kOffOut + 4 * 8192;                    // kQStages x 512 B
constexpr int kOffDelta = kOffL + kQStages * kBlk * 4;
constexpr int kSmemAlloc = kOffDelta + kQStages * kBlk * 4 + 1024;
static_assert(kSmemAlloc + 1024 <= 232448, "smem");
constexpr uint32_t kColS = 0, kColDP = 128, kColP = 256, kColDS = 320, kColDV = 384, kColDK = 448;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescSS = idesc_bf16(128, 128, false, false);  // S^T, dP^T
constexpr uint32_t kIdescTS = idesc_bf16(128, kD, false, true);    // dV, dK

struct Bars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t q_full[kQStages], q_empty[kQStages];
    // of S^T and dP^T: written, read by the P/dS warps; of P^T and dS^T: written, read by dV / dK
    uint64_t s_full, s_free, dp_full, dp_free;
    uint64_t p_full, p_empty, ds_full, ds_empty;
    uint64_t all_done, acc_read;  // an item's dV, dK complete; read out of TMEM
    uint64_t drain, drain2;
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    win_bwd64_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                     const BwdArgs args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Bars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const sb_ptr = smem_raw + (sb - smem_u32(smem_raw));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int N = args.N, Np = args.Np;
    // As in the d = 128 kernel every role goes through this CTA's items on its own; query blocks are
    // numbered g = 0, 1, 2, ... across items, items (those with query blocks) kc = 0, 1, ...
    const int n_items = far_items(args) + args.n_kv * args.BH;
    const uint64_t lim = args.ctl.wait_ns;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&bars.k_full[b]), 1);
            mbar_init(smem_u32(&bars.k_empty[b]), 1);
            mbar_init(smem_u32(&bars.v_full[b]), 1);
            mbar_init(smem_u32(&bars.v_empty[b]), 1);
        }
        for (int s = 0; s < kQStages; ++s) {
            mbar_init(smem_u32(&bars.q_full[s]), 1);
            mbar_init(smem_u32(&bars.q_empty[s]), 1);
        }
        mbar_init(smem_u32(&bars.s_full), 1);
        mbar_init(smem_u32(&bars.s_free), kPdsThreads);
        mbar_init(smem_u32(&bars.dp_full), 1);
        mbar_init(smem_u32(&bars.dp_free), kPdsThreads);
        mbar_init(smem_u32(&bars.p_full), kPdsThreads);
        mbar_init(smem_u32(&bars.p_empty), 1);
        mbar_init(smem_u32(&bars.ds_full), kPdsThreads);
        mbar_init(smem_u32(&bars.ds_empty), 1);
        mbar_init(smem_u32(&bars.all_done), 1);
        mbar_init(smem_u32(&bars.acc_read), 128);
        mbar_init(smem_u32(&bars.drain), 1);
        mbar_init(smem_u32(&bars.drain2), 1);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_do);
        tma_prefetch_desc(&tm_dk);
        tma_prefetch_desc(&tm_dv);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    griddep_wait();  // delta and lse come from the kernel before this one

    // 768 threads x 80 registers at launch: 40 + 4 * 88 + 88 = 6 * 80
    if (warp < 4) {
        regs_dec<40>();
        if (warp == 0) {
            // ============================================================ Q / dO producer
            if (lane == 0) {
                int g = 0;
                bool ok = true;
                for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
                    const Item I = item_at(args, x);
                    Walk at(args, I);
                    for (int i = 0; i < I.n_it; ++i, ++g, at.next()) {
                        const int s = g % kQStages;
                        const int qb = at.blk, qh = at.head;
                        if (g >= kQStages &&
                            !mbar_wait(smem_u32(&bars.q_empty[s]), ((g / kQStages) & 1) ^ 1, lim, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t qf = smem_u32(&bars.q_full[s]);
                        mbar_arrive_expect_tx(qf, 2 * kTile + 2 * kBlk * 4);
                        tma_load_3d(sb + kOffQ + s * kTile, &tm_q, qf, 0, qb * kBlk, qh);
                        tma_load_3d(sb + kOffDO + s * kTile, &tm_do, qf, 0, qb * kBlk, qh);
                        const size_t row = static_cast<size_t>(qh) * Np + static_cast<size_t>(qb) * kBlk;
                        bulk_load(sb + kOffL + s * kBlk * 4, args.ws_lse2 + row, kBlk * 4, qf);
                        bulk_load(sb + kOffDelta + s * kBlk * 4, args.ws_delta + row, kBlk * 4, qf);
                    }
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                // the newest load of every stage has landed before exit
                const volatile int never = 0;
                for (int q = max(0, g - kQStages); q < g; ++q)
                    mbar_wait(smem_u32(&bars.q_full[q % kQStages]), (q / kQStages) & 1, kDrainWaitNs, &never);
            }
        } else if (warp == 3) {
            // ============================================================ K / V producer
            if (lane == 0) {
                int kc = 0, kn = 0, vn = 0;  // items, K and V loads issued
                bool ok = true;
                for (int k = 0, x = item_x(0); x < n_items; x = item_x(++k)) {
                    const Item I = item_at(args, x);
                    if (I.n_it == 0) continue;
                    const int b = kc & 1;
                    const uint32_t par = ((kc >> 1) & 1) ^ 1;
                    if (kc >= 2 && !mbar_wait(smem_u32(&bars.k_empty[b]), par, lim, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t kf = smem_u32(&bars.k_full[b]);
                    mbar_arrive_expect_tx(kf, kTile);
                    tma_load_3d(sb + kOffK + b * kTile, &tm_k, kf, 0, I.kvb * kBlk, I.bh);
                    kn = kc + 1;
                    if (kc >= 2 && !mbar_wait(smem_u32(&bars.v_empty[b]), par, lim, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t vf = smem_u32(&bars.v_full[b]);
                    mbar_arrive_expect_tx(vf, kTile);
                    tma_load_3d(sb + kOffV + b * kTile, &tm_v, vf, 0, I.kvb * kBlk, I.bh);
                    vn = ++kc;
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                const volatile int never = 0;
                for (int i = max(0, kn - 2); i < kn; ++i)
                    mbar_wait(smem_u32(&bars.k_full[i & 1]), (i >> 1) & 1, kDrainWaitNs, &never);
                for (int i = max(0, vn - 2); i < vn; ++i)
                    mbar_wait(smem_u32(&bars.v_full[i & 1]), (i >> 1) & 1, kDrainWaitNs, &never);
            }
        } else if (warp == 1) {
            // ============================================================ S^T, dP^T issuer
            if (lane == 0) {
                constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
                constexpr uint32_t kStage16 = kTile >> 4;
                const uint32_t k_lo = sdesc_sw128_lo(sb + kOffK, 16), v_lo = sdesc_sw128_lo(sb + kOffV, 16);
                const uint32_t q_lo = sdesc_sw128_lo(sb + kOffQ, 16), do_lo = sdesc_sw128_lo(sb + kOffDO, 16);
                auto issue = [&](uint32_t col, uint32_t a_lo, uint32_t b_lo, uint64_t& bar) {
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk) {
                        if (kk == 0)
                            mma_ss_w<false, -1>(tmem + col, a_lo, b_lo, kDescHi, kIdescSS, 0u);
                        else
                            mma_ss_w<false, 1>(tmem + col, a_lo + 2 * kk, b_lo + 2 * kk, kDescHi, kIdescSS);
                    }
                    mma_commit(smem_u32(&bar));
                };
                int g = 0, kc = 0;
                bool ok = true;
                for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
                    const Item I = item_at(args, x);
                    if (I.n_it == 0) continue;
                    const int b = kc & 1;
                    ok = mbar_wait(smem_u32(&bars.k_full[b]), (kc >> 1) & 1, lim, &abort_flag);
                    if (ok) ok = mbar_wait(smem_u32(&bars.v_full[b]), (kc >> 1) & 1, lim, &abort_flag);
                    for (int i = 0; i < I.n_it && ok; ++i, ++g) {
                        const int s = g % kQStages;
                        const bool last = i + 1 == I.n_it;
                        ok = mbar_wait(smem_u32(&bars.q_full[s]), (g / kQStages) & 1, lim, &abort_flag);
                        if (ok && g > 0) ok = mbar_wait(smem_u32(&bars.s_free), (g - 1) & 1, lim, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        issue(kColS, k_lo + b * kStage16, q_lo + s * kStage16, bars.s_full);
                        if (last) mma_commit(smem_u32(&bars.k_empty[b]));
                        if (g > 0) ok = mbar_wait(smem_u32(&bars.dp_free), (g - 1) & 1, lim, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        issue(kColDP, v_lo + b * kStage16, do_lo + s * kStage16, bars.dp_full);
                        if (last) mma_commit(smem_u32(&bars.v_empty[b]));
                    }
                    ++kc;
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                mma_commit(smem_u32(&bars.drain));
                const volatile int never = 0;
                mbar_wait(smem_u32(&bars.drain), 0, kDrainWaitNs, &never);
            }
        } else {
            // ============================================================ dV, dK issuer
            if (lane == 0) {
                constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
                constexpr uint32_t kStage16 = kTile >> 4;
                const uint32_t q_mn = sdesc_sw128_lo(sb + kOffQ, 16384), do_mn = sdesc_sw128_lo(sb + kOffDO, 16384);
                auto issue = [&](uint32_t col, uint32_t colA, uint32_t b_mn, bool acc, uint64_t& bar) {
#pragma unroll
                    for (int kk = 0; kk < kBlk / 16; ++kk) {
                        if (kk == 0)
                            mma_ts_w<false, -1>(tmem + col, tmem + colA, b_mn, kDescHi, kIdescTS, acc ? 1u : 0u);
                        else
                            mma_ts_w<false, 1>(tmem + col, tmem + colA + 8 * kk, b_mn + 128 * kk, kDescHi, kIdescTS);
                    }
                    mma_commit(smem_u32(&bar));
                };
                int g = 0, kc = 0;
                bool ok = true;
                for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
                    const Item I = item_at(args, x);
                    if (I.n_it == 0) continue;
                    for (int i = 0; i < I.n_it; ++i, ++g) {
                        const int s = g % kQStages;
                        ok = mbar_wait(smem_u32(&bars.q_full[s]), (g / kQStages) & 1, lim, &abort_flag);
                        // the last item's dV and dK have been read out
                        if (ok && i == 0 && kc > 0)
                            ok = mbar_wait(smem_u32(&bars.acc_read), (kc - 1) & 1, lim, &abort_flag);
                        if (ok) ok = mbar_wait(smem_u32(&bars.p_full), g & 1, lim, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        issue(kColDV, kColP, do_mn + s * kStage16, i > 0, bars.p_empty);
                        ok = mbar_wait(smem_u32(&bars.ds_full), g & 1, lim, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        issue(kColDK, kColDS, q_mn + s * kStage16, i > 0, bars.ds_empty);
                        // the stage's other readers (S^T, dP^T, lse, delta) were done before dS^T was
                        mma_commit(smem_u32(&bars.q_empty[s]));
                    }
                    if (!ok) break;
                    mma_commit(smem_u32(&bars.all_done));
                    ++kc;
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                mma_commit(smem_u32(&bars.drain2));
                const volatile int never = 0;
                mbar_wait(smem_u32(&bars.drain2), 0, kDrainWaitNs, &never);
            }
        }
    } else if (warp < 20) {
        regs_inc<88>();
        // ================================================================ P / dS warpgroups
        // (runs of 32 queries)
        const int part = (warp - 4) / 4;          // queries 32*part .. 32*part+31
        const int wq = warp % 4;
        const int key_in_blk = wq * 32 + lane;
        const uint32_t lb = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float2 c2 = make_float2(args.c_log2, args.c_log2);
        const uint32_t hide = args.c_log2 >= 0.f ? 0xff800000u : 0x7f800000u;  // -inf after the multiply by c
        bool ok = true;
        int g = 0;
        for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
            const Item I = item_at(args, x);
            const int key = I.kvb * kBlk + key_in_blk;
            Walk at(args, I);
            for (int i = 0; i < I.n_it; ++i, ++g, at.next()) {
                const int s = g % kQStages;
                int q_first, q_end;
                query_range(args.split, key, at.blk * kBlk + 32 * part, q_first, q_end);
                ok = mbar_wait(smem_u32(&bars.q_full[s]), (g / kQStages) & 1, lim, &abort_flag);
                if (ok) ok = mbar_wait(smem_u32(&bars.s_full), g & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                // -lse_i * log2(e) and -delta_i of these queries
                const float4* nl = reinterpret_cast<const float4*>(sb_ptr + kOffL + s * kBlk * 4) + 8 * part;
                const float4* nd = reinterpret_cast<const float4*>(sb_ptr + kOffDelta + s * kBlk * 4) + 8 * part;
                uint32_t p[1][32];  // scores, then P^T
                {
                    uint32_t pk[16];
                    tmem_ld32_async(lb + kColS + 32 * part, p[0]);
                    tmem_wait_ld();
                    reg_fence(p[0]);
                    tc_fence_before();
                    mbar_arrive(smem_u32(&bars.s_free));
                    probabilities(p, q_first, q_end, hide, c2, nl, pk);
                    if (g > 0) {  // dV of the last pair has read P^T
                        ok = mbar_wait(smem_u32(&bars.p_empty), (g - 1) & 1, lim, &abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    tmem_st16(lb + kColP + 16 * part, pk);
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(smem_u32(&bars.p_full));
                }
                // dS^T = P^T o (dP^T - delta)
                ok = mbar_wait(smem_u32(&bars.dp_full), g & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                uint32_t r[32];
                tmem_ld32_async(lb + kColDP + 32 * part, r);
                tmem_wait_ld();
                reg_fence(r);
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.dp_free));
                uint32_t w[16];
                score_gradients(p[0], r, nd, w);
                if (g > 0) {  // dK of the last pair has read dS^T
                    ok = mbar_wait(smem_u32(&bars.ds_empty), (g - 1) & 1, lim, &abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                }
                tmem_st16(lb + kColDS + 16 * part, w);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.ds_full));
            }
        }
        if (!ok && lane == 0) record_timeout(args.ctl, &abort_flag);
    } else {
        regs_inc<88>();
        // ================================================================ dV, dK out
        const int wq = warp % 4;
        const uint32_t lb = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t box = sb + kOffOut + wq * 8192;  // this warp's rows: dV, then dK
        bool ok = true;
        int kc = 0;
        for (int k = 0, x = item_x(0); x < n_items; x = item_x(++k)) {
            const Item I = item_at(args, x);
            if (I.n_it == 0) continue;
            ok = mbar_wait(smem_u32(&bars.all_done), kc & 1, lim, &abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++kc;
            tc_fence_after();
            if (I.slot >= 0) {
                write_part_row<kD>(args, I, 0, wq * 32 + lane, lb + kColDV);
                write_part_row<kD>(args, I, 1, wq * 32 + lane, lb + kColDK);
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.acc_read));
                continue;
            }
            // 128-byte rows, 16-byte granule g of row r at g ^ (r % 8); the last item's stores have
            // read them
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int m = 0; m < 2; ++m) {  // dV; dK times scale
                const float f = m ? args.scale : 1.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[32];
                    tmem_ld32(lb + (m ? kColDK : kColDV) + 32 * h, r);
                    if (m == 1 && h == 1) {
                        tc_fence_before();
                        mbar_arrive(smem_u32(&bars.acc_read));
                    }
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4) {
                        const float* x = reinterpret_cast<const float*>(r) + 8 * c4;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + m * 4096 + lane * 128 +
                                                                                      (((4 * h + c4) ^ (lane & 7)) << 4)),
                                     "r"(pack_bf16x2(x[0] * f, x[1] * f)), "r"(pack_bf16x2(x[2] * f, x[3] * f)),
                                     "r"(pack_bf16x2(x[4] * f, x[5] * f)), "r"(pack_bf16x2(x[6] * f, x[7] * f))
                                     : "memory");
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            const int row0 = I.kvb * kBlk + wq * 32;
            if (lane == 0 && row0 < N) {
                tma_store_3d(&tm_dv, box, 0, row0, I.bh);
                tma_store_3d(&tm_dk, box + 4096, 0, row0, I.bh);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        }
        // the stores complete before the CTA's shared memory goes away
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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

cudaError_t launch_bwd_window_main64(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& dO,
                                     const CUtensorMap& dk, const CUtensorMap& dv, const WinBwdArgs& a, int grid,
                                     cudaStream_t s) {
    static std::atomic<uint64_t> smem_done;
    const cudaError_t e = allow_smem(win_bwd64_kernel, kSmemAlloc, smem_done);
    if (e != cudaSuccess) return e;
    // set up while win_bwd_prep runs: 0.8% of a step (the d = 128 kernel lost as much that way)
    return launch_pdl(win_bwd64_kernel, dim3(grid), dim3(kThreads), kSmemAlloc, s, q, k, v, dO, dk, dv, a);
}

}  // namespace fa
