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
// This kernel is for d = 128, whose S (P in its place) and O fill TMEM; d = 64 has room for P of its
// own and another schedule (win_fwd64_sm103.cu).  Warp roles, TMEM columns, the K/V bundle ring and
// the order of MMAs are the plain forward's; O leaves through shared memory and TMA stores.  Every
// wait is bounded, and a wait that runs out is recorded and ends the CTA with its copies and MMAs
// drained.
// Measured: N16384 W4096, 4 sinks, H32 H_kv8 623 us on a cool GPU, 1546 TFLOP/s of visible pairs (80% of
// the bf16 peak), 660-683 us (1412-1460) called for a second or more, when the power cap lowers the clock;
// N8191 W1024, 16 sinks, H16 71 us.
#include <type_traits>

#include "win_fwd.cuh"

namespace fa {
namespace {

constexpr int kStages = 2;     // K/V ring depth

constexpr int D = 128;

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

// Persistent: a CTA works through items, its k-th being x = k * gridDim.x + (blockIdx.x, or
// gridDim.x - 1 - blockIdx.x in odd rounds); items run from the last pair of every head to
// the first, the heaviest first (the first W / 256 pairs of a head see fewer keys).  Every
// barrier counts its phases across items: q_full, q_free per item, kv_full, kv_empty per
// bundle, s_full, p_full per block that the tile visits, o_done per item of the tile.
__global__ void __launch_bounds__(kThreads, 1)
    win_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                   const WinArgs args) {
    using C = Cfg;
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
                // P overwrites S, and O_t += P V of the tile's last block precedes these scores in
                // issue order: nothing to say and nothing to wait for
                auto taken = [] {};
                auto free = [] { return true; };
                if (n == 0 && P.shorty)
                    softmax_block<D, kShort>(lane_base, colS, colS, colO, c, c_pos, mask_bits, hi, lo, sink, first, m_ref, l,
                                             taken, free);
                else
                    softmax_block<D, kBN>(lane_base, colS, colS, colO, c, c_pos, mask_bits, hi, lo, sink, first, m_ref, l,
                                          taken, free);
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
            store_rows<D>(tm_o, smem_base + C::kOffO + (warp - 4) * 4096, lane_base + colO, inv, r0 + t * kBM + wq * 32, bh, N);
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

}  // namespace

int launch_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv, int N,
                      int d, float c_log2, int window, int sinks, DevCtl ctl, cudaStream_t s) {
    if (d == 64) return launch_fwd_window64(q, k, v, o, lse, B, H, H_kv, N, c_log2, window, sinks, ctl, s);
    CUtensorMap m[4];
    const int rc = win_maps(m, q, k, v, o, B, H, H_kv, N, 128);
    if (rc != 0) return rc;
    const WinArgs a = win_args(lse, B, H, H_kv, N, c_log2, window, sinks, ctl);
    static std::atomic<uint64_t> smem_done;
    int dev = 0, sms = 152;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = allow_smem(win_fwd_kernel, Cfg::kSmemAlloc, smem_done);
    if (e != cudaSuccess) return static_cast<int>(e);
    return static_cast<int>(launch_pdl(win_fwd_kernel, dim3(a.n_items < sms ? a.n_items : sms), dim3(kThreads),
                                       Cfg::kSmemAlloc, s, m[0], m[1], m[2], m[3], a));
}

}  // namespace fa
