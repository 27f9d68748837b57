// win_fwd64_sm103.cu -- the windowed forward (win_fwd_sm103.cu) for d = 64.
//
// At d = 64 the two products of a tile and a key block are 12 MMAs, half of d = 128's, and the
// softmax the same; with P written over S a tile's scores, softmax and P V run one after the other
// (1550 cycles a tile and block).  TMEM has room for more here: S 2 x 128, P (bf16) 2 x 64 and
// O 2 x 64 columns are all 512.  So
//   * P has columns of its own, and S_t of the next block is computed as soon as the softmax warps
//     have S_t in registers (s_free), beside softmax and P V;
//   * two threads issue MMAs, one S of both tiles, the other P V of both: they share no columns that
//     either writes, and neither waits for the other's barriers;
//   * K and V have rings of their own, three blocks deep, each released by its one reader;
//   * P_t is rewritten and O_t rescaled once P V of the tile's last block is done (pv_done).
// Measured: B4 H16 N1000 W256, 4 sinks 18.6 us (3 of them until the first scores: every CTA's first
// loads at once), B4 H16 N2048 W512, 4 sinks 36 us; a block takes two tiles 1900 cycles, a masked one
// 2600.
#include <type_traits>

#include "win_fwd.cuh"

namespace fa {
namespace {

constexpr int D = 64;
constexpr int kStages = 3;
constexpr int kTileBytes = kBM * D * 2;
constexpr int kOffQ = 0, kOffK = 2 * kTileBytes, kOffV = kOffK + kStages * kTileBytes;
constexpr int kOffO = kOffV + kStages * kTileBytes;  // 4 KB per softmax warp: 32 rows x 128 bytes
constexpr int kSmemAlloc = kOffO + 8 * 4096 + 1024;
constexpr uint32_t kColS = 0, kColP = 256, kColO = 384;  // + 128, 64, 64 for the second tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescS = idesc_bf16(kBM, kBN, false, false);
constexpr uint32_t kIdescShort = idesc_bf16(kBM, kShort, false, false);
constexpr uint32_t kIdescO = idesc_bf16(kBM, D, false, true);

struct Bars {
    uint64_t q_full, q_free;
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
    uint64_t drain, drain2;
};

// Persistent as the d = 128 kernel; phases: q_full, q_free per item, the rings' per block of the
// item's list, the tiles' per block that the tile visits.
__global__ void __launch_bounds__(kThreads, 1)
    win_fwd64_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                     const WinArgs args) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Bars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
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
            mbar_init(smem_u32(&bars.k_full[s]), 1);
            mbar_init(smem_u32(&bars.k_empty[s]), 1);
            mbar_init(smem_u32(&bars.v_full[s]), 1);
            mbar_init(smem_u32(&bars.v_empty[s]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bars.s_full[t]), 1);
            mbar_init(smem_u32(&bars.s_free[t]), 128);
            mbar_init(smem_u32(&bars.p_full[t]), 128);
            mbar_init(smem_u32(&bars.pv_done[t]), 1);
        }
        mbar_init(smem_u32(&bars.drain), 1);
        mbar_init(smem_u32(&bars.drain2), 1);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_o);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), kTmemCols);
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
                int g = 0, kq = 0;         // blocks, and items whose Q was issued
                int gk = 0, gv = 0;        // K and V loads issued
                bool ok = true;
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
                    mbar_arrive_expect_tx(qf, n_q * kTileBytes);
                    for (int t = 0; t < n_q; ++t)
                        tma_load_3d(sb + kOffQ + t * kTileBytes, &tm_q, qf, 0, r0 + t * kBM, bh);
                    ++kq;
                    for (int n = 0; n < P.n; ++n, ++g) {
                        const int u = g % kStages, row = P.block(n) * kBN;
                        const uint32_t par = ((g / kStages) & 1) ^ 1;
                        if (g >= kStages && !mbar_wait(smem_u32(&bars.k_empty[u]), par, lim, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t kf = smem_u32(&bars.k_full[u]);
                        mbar_arrive_expect_tx(kf, kTileBytes);
                        tma_load_3d(sb + kOffK + u * kTileBytes, &tm_k, kf, 0, row, bh_kv);
                        gk = g + 1;
                        if (g >= kStages && !mbar_wait(smem_u32(&bars.v_empty[u]), par, lim, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t vf = smem_u32(&bars.v_full[u]);
                        mbar_arrive_expect_tx(vf, kTileBytes);
                        tma_load_3d(sb + kOffV + u * kTileBytes, &tm_v, vf, 0, row, bh_kv);
                        gv = g + 1;
                    }
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                // the last Q and the newest load of every slot have landed before exit
                const volatile int never = 0;
                if (kq > 0) mbar_wait(qf, (kq - 1) & 1, kDrainWaitNs, &never);
                for (int i = max(0, gk - kStages); i < gk; ++i)
                    mbar_wait(smem_u32(&bars.k_full[i % kStages]), (i / kStages) & 1, kDrainWaitNs, &never);
                for (int i = max(0, gv - kStages); i < gv; ++i)
                    mbar_wait(smem_u32(&bars.v_full[i % kStages]), (i / kStages) & 1, kDrainWaitNs, &never);
            }
        } else if (warp == 1) {
            // ============================================================ S issuer
            if (lane == 0) {
                constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
                const uint32_t q_lo = sdesc_sw128_lo(sb + kOffQ, 16), k_lo = sdesc_sw128_lo(sb + kOffK, 16);
                int g = 0, kq = 0;
                int cnt[2] = {0, 0};  // blocks of each tile, over all items
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    const int x = item_x(k);
                    if (x >= n_items) break;
                    const Plan P = plan_of(args, item_r0(x));
                    ok = mbar_wait(smem_u32(&bars.q_full), kq & 1, lim, &abort_flag);
                    for (int n = 0; ok && n < P.n; ++n, ++g) {
                        const int u = g % kStages;
                        ok = mbar_wait(smem_u32(&bars.k_full[u]), (g / kStages) & 1, lim, &abort_flag);
                        if (!ok) break;
                        const uint32_t kl = k_lo + u * (kTileBytes >> 4);
                        const uint32_t idesc = n == 0 && P.shorty ? kIdescShort : kIdescS;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!P.active(t, n)) continue;
                            // the tile's last scores are in registers
                            if (cnt[t] > 0) ok = mbar_wait(smem_u32(&bars.s_free[t]), (cnt[t] - 1) & 1, lim, &abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t ql = q_lo + t * (kTileBytes >> 4);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                if (kk == 0)
                                    mma_ss_w<false, -1>(tmem + kColS + 128 * t, ql, kl, kDescHi, idesc, 0u);
                                else
                                    mma_ss_w<false, 1>(tmem + kColS + 128 * t, ql + 2 * kk, kl + 2 * kk, kDescHi, idesc);
                            }
                            mma_commit(smem_u32(&bars.s_full[t]));
                            ++cnt[t];
                        }
                        if (!ok) break;
                        mma_commit(smem_u32(&bars.k_empty[u]));
                    }
                    if (ok) mma_commit(smem_u32(&bars.q_free));
                    ++kq;
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                mma_commit(smem_u32(&bars.drain));
                const volatile int never = 0;
                mbar_wait(smem_u32(&bars.drain), 0, kDrainWaitNs, &never);
            }
        } else if (warp == 2) {
            // ============================================================ P V issuer
            if (lane == 0) {
                constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
                const uint32_t v_lo = sdesc_sw128_lo(sb + kOffV, kTileBytes);
                auto issue_pv = [&](int t, uint32_t vl, bool acc, auto steps_c) {
                    constexpr int kSteps = decltype(steps_c)::value;
                    const uint32_t colO = tmem + kColO + 64 * t, colP = tmem + kColP + 64 * t;
#pragma unroll
                    for (int kk = 0; kk < kSteps; ++kk) {
                        if (kk == 0)
                            mma_ts_w<false, -1>(colO, colP, vl, kDescHi, kIdescO, acc ? 1u : 0u);
                        else
                            mma_ts_w<false, 1>(colO, colP + 8 * kk, vl + 128 * kk, kDescHi, kIdescO);
                    }
                    mma_commit(smem_u32(&bars.pv_done[t]));
                };
                int g = 0;
                int cnt[2] = {0, 0};
                bool ok = true;
                for (int k = 0; ok; ++k) {
                    const int x = item_x(k);
                    if (x >= n_items) break;
                    const Plan P = plan_of(args, item_r0(x));
                    bool acc[2] = {false, false};
                    for (int n = 0; n < P.n; ++n, ++g) {
                        const int u = g % kStages;
                        ok = mbar_wait(smem_u32(&bars.v_full[u]), (g / kStages) & 1, lim, &abort_flag);
                        if (!ok) break;
                        const uint32_t vl = v_lo + u * (kTileBytes >> 4);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!P.active(t, n)) continue;
                            // P of an item's first block is published after O_t of the item before
                            // has been read, so O_t may then be overwritten
                            ok = mbar_wait(smem_u32(&bars.p_full[t]), cnt[t] & 1, lim, &abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            if (n == 0 && P.shorty)
                                issue_pv(t, vl, acc[t], std::integral_constant<int, kShort / 16>{});
                            else
                                issue_pv(t, vl, acc[t], std::integral_constant<int, kBN / 16>{});
                            acc[t] = true;
                            ++cnt[t];
                        }
                        if (!ok) break;
                        mma_commit(smem_u32(&bars.v_empty[u]));
                    }
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                mma_commit(smem_u32(&bars.drain2));
                const volatile int never = 0;
                mbar_wait(smem_u32(&bars.drain2), 0, kDrainWaitNs, &never);
            }
        }
        // warp 3 has no role
    } else {
        regs_inc<184>();
        // ================================================================ softmax warpgroups
        const int t = (warp - 4) / 4;
        const int wq = warp % 4;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t colS = kColS + 128 * t, colP = kColP + 64 * t, colO = kColO + 64 * t;
        const float c = args.c_log2;
        const bool c_pos = c >= 0.f;
        const uint32_t mask_bits = c_pos ? 0xff800000u : 0x7f800000u;  // -inf after the multiply by c
        int gj = 0;  // blocks of this tile, over all items
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int x = item_x(k);
            if (x >= n_items) break;
            const int bh = item_bh(x), r0 = item_r0(x);
            const Plan P = plan_of(args, r0);
            if (t == 1 && !P.two) continue;
            const int qrow = r0 + t * kBM + wq * 32 + lane;
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
                auto taken = [&] {
                    tc_fence_before();
                    mbar_arrive(smem_u32(&bars.s_free[t]));
                };
                // P V of the tile's last block (of this item; an item's first follows the end of the
                // item before) has read P_t and written O_t
                auto free = [&] {
                    if (first) return true;
                    const bool done = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.pv_done[t]), (gj - 1) & 1, lim, &abort_flag));
                    tc_fence_after();
                    return done;
                };
                if (n == 0 && P.shorty)
                    ok = softmax_block<D, kShort>(lane_base, colS, colP, colO, c, c_pos, mask_bits, hi, lo, sink, first, m_ref,
                                                  l, taken, free);
                else
                    ok = softmax_block<D, kBN>(lane_base, colS, colP, colO, c, c_pos, mask_bits, hi, lo, sink, first, m_ref, l,
                                               taken, free);
                if (!ok) break;
                first = false;
                ++gj;
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.p_full[t]));
            }
            if (ok) {
                ok = mbar_wait(smem_u32(&bars.pv_done[t]), (gj - 1) & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!ok) {
                if (lane == 0) record_timeout(args.ctl, &abort_flag);
                break;
            }
            tc_fence_after();
            // O_t is read before this warp publishes the next item's first P
            store_rows<D>(tm_o, sb + kOffO + (warp - 4) * 4096, lane_base + colO, 1.f / l, r0 + t * kBM + wq * 32, bh, N);
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
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

int launch_fwd_window64(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv, int N,
                        float c_log2, int window, int sinks, DevCtl ctl, cudaStream_t s) {
    CUtensorMap m[4];
    const int rc = win_maps(m, q, k, v, o, B, H, H_kv, N, D);
    if (rc != 0) return rc;
    const WinArgs a = win_args(lse, B, H, H_kv, N, c_log2, window, sinks, ctl);
    static std::atomic<uint64_t> smem_done;
    int dev = 0, sms = 152;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = allow_smem(win_fwd64_kernel, kSmemAlloc, smem_done);
    if (e != cudaSuccess) return static_cast<int>(e);
    return static_cast<int>(launch_pdl(win_fwd64_kernel, dim3(a.n_items < sms ? a.n_items : sms), dim3(kThreads), kSmemAlloc,
                                       s, m[0], m[1], m[2], m[3], a));
}

}  // namespace fa
