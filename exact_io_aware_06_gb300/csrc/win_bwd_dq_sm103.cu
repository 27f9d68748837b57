// win_bwd_dq_sm103.cu -- dQ of the windowed backward, query-parallel, over the
// key blocks that a 128-query block sees, those of the sinks and those of the window:
//     S_ij = Q_i K_j^T,  P_ij = exp(S_ij - lse_i),  dP_ij = dO_i V_j^T,
//     dS_ij = P_ij o (dP_ij - delta_i),  dQ_i = scale * sum_j dS_ij K_j.
// dQ_i accumulates in TMEM over the sweep and is written once as bf16: no atomics.
//
// Three products of 128 x 128 x d per pair of blocks, 24 MMAs at d = 128: 1614 cycles of the tensor pipe.
// The plain backward's dQ kernel writes dS over S, so that the next scores wait for this block's
// dS and dQ: 3850 cycles a pair.  Here:
//   * dS has two TMEM buffers of its own, and the tensor core goes on with the next block's S
//     and dP as soon as the dS warps have taken this block's into registers.
//   * Two issuing threads, S and dP in one, dQ in the other: a single thread issues S and dP of
//     pair g + 1 (1034 cycles), then waits for dS of g and issues dQ (1100), 2970 cycles a pair.
//   * K is read twice, up to two pairs apart: its ring is three deep, V's two (with Q and dO
//     224 KB).
//   * Persistent, one CTA per SM, items from the last query blocks to the first: the next
//     item's Q, dO and first S, dP are under way while this one ends, and a warpgroup of its
//     own writes dQ (which took 3000 cycles of the dS warps' time per item).
// Measured: d = 128 (N8191 W1024, 16 sinks, H16 H_kv4) 79 us, 1810 cycles a pair inside an item;
// d = 64 (B4 H16 N2048 W512, 4 sinks) 42 us.
//
// An idle warp joins the parts of dK and dV that the kernel before has left (join_parts).
//
// Warp 0 TMA, warps 1 and 2 MMA, warps 4-7 and 8-11 one query row per thread, for keys 0-63 /
// 64-127 of block j, warps 12-15 write dQ.  TMEM: S 0-127, dP 128-255, dQ 256-383, dS (bf16)
// 384-447 and 448-511.
#include "win_bwd.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr int kKStages = 3, kVStages = 2;
template <int D>
struct Cfg {
    static constexpr int kTile = kBlk * D * 2;
    static constexpr int kOffQ = 0, kOffDO = kTile, kOffK = 2 * kTile, kOffV = kOffK + kKStages * kTile;
    static constexpr int kSmemAlloc = kOffV + kVStages * kTile + 1024;
    static constexpr uint32_t kIdescDQ = idesc_bf16(128, D, false, true);  // dQ += dS K
};
static_assert(Cfg<128>::kSmemAlloc + 1024 <= 232448, "smem");
constexpr uint32_t kColS = 0, kColDP = 128, kColDQ = 256, kColDS = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescSS = idesc_bf16(128, 128, false, false);  // S, dP
constexpr uint32_t kIdescShort = idesc_bf16(128, 32, false, false);  // of up to 32 sinks

struct DqArgs {
    WinBwdArgs w;
    void* dq;
    int n_items;  // 128-query blocks of all query heads
};

struct DqBars {
    uint64_t q_full, q_free;
    uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t sp_full, sp_free;  // S, dP written; read by the dS warps
    uint64_t ds_full[2], ds_empty[2];  // one per dS buffer: a waiter cannot fall two phases behind
    uint64_t all_done, dq_read;        // an item's dQ complete; read out of TMEM
    uint64_t drain, drain2;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    win_bwd_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                      const DqArgs dq_args) {
    using C = Cfg<D>;
    constexpr int kTile = C::kTile, kOffQ = C::kOffQ, kOffDO = C::kOffDO, kOffK = C::kOffK, kOffV = C::kOffV;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) DqBars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const WinBwdArgs& args = dq_args.w;
    const int N = args.N, Np = args.Np, n_items = dq_args.n_items;
    const int q_heads = args.BH / args.H_kv * args.H;
    const uint64_t lim = args.ctl.wait_ns;
    struct QItem {
        int bh, bh_kv, qb, lo, n_sink, n_kv;
        bool shorty;  // the first block is that of up to 32 sinks, in front of the window
        __device__ __forceinline__ int block(int j) const { return j < n_sink ? j : lo + j - n_sink; }
    };
    auto item_at = [&](int x) {
        QItem I;
        I.bh = x % q_heads;
        I.qb = args.n_kv - 1 - x / q_heads;
        // grouped-query attention: query head bh reads K/V head bh_kv of its group
        I.bh_kv = (I.bh / args.H) * args.H_kv + (I.bh % args.H) / (args.H / args.H_kv);
        // key blocks: the sinks' in front of the window, then lo .. qb
        I.lo = max(0, static_cast<int>(static_cast<long long>(I.qb) * kBlk - args.split.window + 1)) / kBlk;
        I.n_sink = min(I.lo, (args.split.sinks + kBlk - 1) / kBlk);
        I.n_kv = I.n_sink + I.qb - I.lo + 1;
        I.shorty = I.n_sink > 0 && args.split.sinks <= 32;
        return I;
    };

    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(smem_u32(&bars.q_full), 1);
        mbar_init(smem_u32(&bars.q_free), 1);
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(smem_u32(&bars.k_full[s]), 1);
            mbar_init(smem_u32(&bars.k_empty[s]), 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(smem_u32(&bars.v_full[s]), 1);
            mbar_init(smem_u32(&bars.v_empty[s]), 1);
        }
        mbar_init(smem_u32(&bars.sp_full), 1);
        mbar_init(smem_u32(&bars.sp_free), 256);
        mbar_init(smem_u32(&bars.ds_full[0]), 256);
        mbar_init(smem_u32(&bars.ds_full[1]), 256);
        mbar_init(smem_u32(&bars.ds_empty[0]), 1);
        mbar_init(smem_u32(&bars.ds_empty[1]), 1);
        mbar_init(smem_u32(&bars.all_done), 1);
        mbar_init(smem_u32(&bars.dq_read), 128);
        mbar_init(smem_u32(&bars.drain), 1);
        mbar_init(smem_u32(&bars.drain2), 1);
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

    // 512 threads x 128 registers at launch: 72 + 2 * 160 + 120 = 4 * 128
    if (warp < 4) {
        regs_dec<72>();
        if (warp == 0) {
            // ============================================================ producer
            if (lane == 0) {
                const uint32_t qf = smem_u32(&bars.q_full);
                int g = 0, n = 0;  // pairs and items whose loads were issued
                int gk = 0, gv = 0;
                bool ok = true;
                for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
                    const QItem I = item_at(x);
                    if (n > 0 && !mbar_wait(smem_u32(&bars.q_free), (n - 1) & 1, lim, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(qf, 2 * kTile);
                    for (int c = 0; c < D / 64; ++c) {
                        tma_load_3d(sb + kOffQ + c * 16384, &tm_q, qf, 64 * c, I.qb * kBlk, I.bh);
                        tma_load_3d(sb + kOffDO + c * 16384, &tm_do, qf, 64 * c, I.qb * kBlk, I.bh);
                    }
                    ++n;
                    for (int j = 0; j < I.n_kv; ++j, ++g) {
                        const int sk = g % kKStages, sv = g % kVStages, row = I.block(j) * kBlk;
                        // V's slot is free once dP of g - 2 is done, K's after dQ of g - 3, issued later
                        if (g >= kVStages &&
                            !mbar_wait(smem_u32(&bars.v_empty[sv]), ((g / kVStages) & 1) ^ 1, lim, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t vf = smem_u32(&bars.v_full[sv]);
                        mbar_arrive_expect_tx(vf, kTile);
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(sb + kOffV + sv * kTile + c * 16384, &tm_v, vf, 64 * c, row, I.bh_kv);
                        gv = g + 1;
                        if (g >= kKStages &&
                            !mbar_wait(smem_u32(&bars.k_empty[sk]), ((g / kKStages) & 1) ^ 1, lim, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t kf = smem_u32(&bars.k_full[sk]);
                        mbar_arrive_expect_tx(kf, kTile);
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(sb + kOffK + sk * kTile + c * 16384, &tm_k, kf, 64 * c, row, I.bh_kv);
                        gk = g + 1;
                    }
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                // the newest load of every stage has landed before exit
                const volatile int never = 0;
                if (n > 0) mbar_wait(qf, (n - 1) & 1, kDrainWaitNs, &never);
                for (int i = max(0, gk - kKStages); i < gk; ++i)
                    mbar_wait(smem_u32(&bars.k_full[i % kKStages]), (i / kKStages) & 1, kDrainWaitNs, &never);
                for (int i = max(0, gv - kVStages); i < gv; ++i)
                    mbar_wait(smem_u32(&bars.v_full[i % kVStages]), (i / kVStages) & 1, kDrainWaitNs, &never);
            }
        } else if (warp == 1) {
            // ============================================================ MMA issuer
            if (lane == 0) {
                constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
                constexpr uint32_t kStage16 = kTile >> 4;
                const uint32_t q_lo = sdesc_sw128_lo(sb + kOffQ, 16), do_lo = sdesc_sw128_lo(sb + kOffDO, 16);
                const uint32_t k_lo = sdesc_sw128_lo(sb + kOffK, 16), v_lo = sdesc_sw128_lo(sb + kOffV, 16);
                // S = Q K_j^T and dP = dO V_j^T of pair g (both operands K-major along d)
                auto issue_sp = [&](int g, int item, bool first, bool last, uint32_t idesc) -> bool {
                    const int sk = g % kKStages, sv = g % kVStages;
                    if (first && !mbar_wait(smem_u32(&bars.q_full), item & 1, lim, &abort_flag)) return false;
                    if (!mbar_wait(smem_u32(&bars.k_full[sk]), (g / kKStages) & 1, lim, &abort_flag)) return false;
                    if (!mbar_wait(smem_u32(&bars.v_full[sv]), (g / kVStages) & 1, lim, &abort_flag)) return false;
                    if (g > 0 && !mbar_wait(smem_u32(&bars.sp_free), (g - 1) & 1, lim, &abort_flag)) return false;
                    tc_fence_after();
                    const uint32_t kl = k_lo + sk * kStage16, vl = v_lo + sv * kStage16;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off16 = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                        if (kk == 0)
                            mma_ss_w<false, -1>(tmem + kColS, q_lo, kl, kDescHi, idesc, 0u);
                        else
                            mma_ss_w<false, 1>(tmem + kColS, q_lo + off16, kl + off16, kDescHi, idesc);
                    }
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off16 = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                        if (kk == 0)
                            mma_ss_w<false, -1>(tmem + kColDP, do_lo, vl, kDescHi, idesc, 0u);
                        else
                            mma_ss_w<false, 1>(tmem + kColDP, do_lo + off16, vl + off16, kDescHi, idesc);
                    }
                    mma_commit(smem_u32(&bars.sp_full));
                    mma_commit(smem_u32(&bars.v_empty[sv]));
                    if (last) mma_commit(smem_u32(&bars.q_free));
                    return true;
                };
                int g = 0, item = 0;
                bool ok = true;
                for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k), ++item) {
                    const QItem I = item_at(x);
                    for (int j = 0; j < I.n_kv && ok; ++j, ++g)
                        ok = issue_sp(g, item, j == 0, j + 1 == I.n_kv, I.shorty && j == 0 ? kIdescShort : kIdescSS);
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                mma_commit(smem_u32(&bars.drain));
                const volatile int never = 0;
                mbar_wait(smem_u32(&bars.drain), 0, kDrainWaitNs, &never);
            }
        } else if (warp == 2) {
            // ============================================================ dQ issuer
            // Its MMAs read dS (TMEM) and K and write dQ: nothing that the other thread's write.
            if (lane == 0) {
                constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
                const uint32_t k_mn = sdesc_sw128_lo(sb + kOffK, 16384);
                int g = 0, item = 0;
                bool ok = true;
                for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k), ++item) {
                    const QItem I = item_at(x);
                    for (int j = 0; j < I.n_kv; ++j, ++g) {
                        const int sk = g % kKStages;
                        ok = mbar_wait(smem_u32(&bars.k_full[sk]), (g / kKStages) & 1, lim, &abort_flag);
                        // the last item's dQ has been read out
                        if (ok && j == 0 && item > 0)
                            ok = mbar_wait(smem_u32(&bars.dq_read), (item - 1) & 1, lim, &abort_flag);
                        if (ok) ok = mbar_wait(smem_u32(&bars.ds_full[g & 1]), (g >> 1) & 1, lim, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        // dQ += dS_j K_j: A = dS from TMEM (queries x keys), B = K_j MN-major
                        const uint32_t km = k_mn + sk * (kTile >> 4), ds = tmem + kColDS + 64 * (g & 1);
#pragma unroll
                        for (int kk = 0; kk < kBlk / 16; ++kk) {
                            if (kk == 2 && I.shorty && j == 0) break;
                            if (kk == 0)
                                mma_ts_w<false, -1>(tmem + kColDQ, ds, km, kDescHi, C::kIdescDQ, j > 0 ? 1u : 0u);
                            else
                                mma_ts_w<false, 1>(tmem + kColDQ, ds + 8 * kk, km + 128 * kk, kDescHi, C::kIdescDQ);
                        }
                        mma_commit(smem_u32(&bars.ds_empty[g & 1]));
                        mma_commit(smem_u32(&bars.k_empty[sk]));  // S of this pair read K before dS was made
                        if (j + 1 == I.n_kv) mma_commit(smem_u32(&bars.all_done));
                    }
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                mma_commit(smem_u32(&bars.drain2));
                const volatile int never = 0;
                mbar_wait(smem_u32(&bars.drain2), 0, kDrainWaitNs, &never);
            }
        } else if (args.split.n_part > 0) {
            // ============================================================ the sinks' parts
            join_parts<D>(args, static_cast<int>(blockIdx.x) * 32 + lane, static_cast<int>(gridDim.x) * 32);
        }
    } else if (warp < 12) {
        regs_inc<160>();
        // ================================================================ dS warpgroups
        const int half = (warp - 4) / 4;  // keys 64*half .. 64*half+63 of each block
        const int wq = warp % 4;
        const int row = wq * 32 + lane;
        const uint32_t lb = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float2 c2 = make_float2(args.c_log2, args.c_log2);
        const uint32_t hide = args.c_log2 >= 0.f ? 0xff800000u : 0x7f800000u;  // -inf after the multiply by c
        bool ok = true;
        int g = 0;
        // an item's row values, loaded one item ahead; padded rows exist up to Np
        auto row_at = [&](int x) {
            const QItem I = item_at(x);
            return static_cast<size_t>(I.bh) * Np + I.qb * kBlk + row;
        };
        float next_nl = 0.f, next_nd = 0.f;
        if (item_x(0) < n_items) {
            next_nl = args.ws_lse2[row_at(item_x(0))];
            next_nd = args.ws_delta[row_at(item_x(0))];
        }
        for (int k = 0, x = item_x(0); x < n_items && ok; x = item_x(++k)) {
            const QItem I = item_at(x);
            const int qrow = I.qb * kBlk + row;
            const float nl = next_nl, nd = next_nd;
            if (item_x(k + 1) < n_items) {
                next_nl = args.ws_lse2[row_at(item_x(k + 1))];
                next_nd = args.ws_delta[row_at(item_x(k + 1))];
            }
            const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
            for (int j = 0; j < I.n_kv; ++j, ++g) {
                ok = mbar_wait(smem_u32(&bars.sp_full), g & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                // dQ of pair g - 2 has read this pair's dS buffer
                auto buffer_free = [&]() -> bool {
                    if (g < 2) return true;
                    const bool done = mbar_wait(smem_u32(&bars.ds_empty[g & 1]), ((g >> 1) & 1) ^ 1, lim, &abort_flag);
                    if (!__all_sync(0xffffffffu, done)) return false;
                    tc_fence_after();
                    return true;
                };
                // NW runs of 32 keys from this half's first on
                auto pair = [&](auto nw) -> bool {
                    constexpr int NW = decltype(nw)::value;
                    uint32_t rs[NW][32], rp[NW][32];
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        tmem_ld32_async(lb + kColS + 64 * half + 32 * w, rs[w]);
                        tmem_ld32_async(lb + kColDP + 64 * half + 32 * w, rp[w]);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        reg_fence(rs[w]);
                        reg_fence(rp[w]);
                    }
                    tc_fence_before();
                    mbar_arrive(smem_u32(&bars.sp_free));
                    // the row's keys, counted from this half's first: from `first` or below `sink`, to `last`
                    const int key0 = I.block(j) * kBlk + 64 * half;
                    const int last = qrow - key0, sink = args.split.sinks - key0;
                    const int first = static_cast<int>(max(-1ll, static_cast<long long>(last) - args.split.window + 1));
                    const bool edge = __any_sync(0xffffffffu, last < 32 * NW - 1 || (first > 0 && sink < 32 * NW));
                    // a warp's rows are neighbours: of its two runs of 32 keys mostly one holds a bound of
                    // some row and needs the test of every score
                    if (edge) {
#pragma unroll
                        for (int w = 0; w < NW; ++w) {
                            const uint32_t seen =
                                bits_below(last + 1 - 32 * w) & (~bits_below(first - 32 * w) | bits_below(sink - 32 * w));
                            if (__any_sync(0xffffffffu, seen != 0xffffffffu)) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!(seen & (1u << i))) rs[w][i] = hide;
                            }
                        }
                    }
                    uint32_t pk[16 * NW];
#pragma unroll
                    for (int i = 0; i < 16 * NW; ++i) {
                        const int e = 2 * (i % 16);
                        const uint32_t* S = rs[i / 16];
                        const uint32_t* P = rp[i / 16];
                        const float2 a = __ffma2_rn(make_float2(__uint_as_float(S[e]), __uint_as_float(S[e + 1])), c2, nl2);
                        const float2 p = make_float2(ex2_approx(a.x), ex2_approx(a.y));
                        const float2 d = __fadd2_rn(make_float2(__uint_as_float(P[e]), __uint_as_float(P[e + 1])), nd2);
                        const float2 ds = __fmul2_rn(p, d);
                        pk[i] = pack_bf16x2(ds.x, ds.y);
                    }
                    if (!buffer_free()) return false;
                    const uint32_t dst = lb + kColDS + 64 * (g & 1) + 32 * half;
                    if constexpr (NW == 2)
                        tmem_st32(dst, pk);
                    else
                        tmem_st16(dst, pk);
                    tmem_st_wait();
                    return true;
                };
                if (!(I.shorty && j == 0)) {
                    ok = pair(std::integral_constant<int, 2>{});
                } else if (half == 0) {
                    ok = pair(std::integral_constant<int, 1>{});
                } else {  // no keys
                    mbar_arrive(smem_u32(&bars.sp_free));
                    ok = buffer_free();
                }
                if (!ok) break;
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.ds_full[g & 1]));
            }
        }
        if (!ok && lane == 0) record_timeout(args.ctl, &abort_flag);
    } else {
        regs_dec<120>();
        // ================================================================ dQ out
        const int wq = warp % 4;
        const uint32_t lb = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        bool ok = true;
        int item = 0;
        for (int k = 0, x = item_x(0); x < n_items; x = item_x(++k), ++item) {
            const QItem I = item_at(x);
            ok = mbar_wait(smem_u32(&bars.all_done), item & 1, lim, &abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            RowsOut<D> rows;
            rows.load(lb + kColDQ, args.scale);
            tc_fence_before();
            mbar_arrive(smem_u32(&bars.dq_read));
            rows.store(dq_args.dq, static_cast<size_t>(I.bh) * N, I.qb * kBlk + wq * 32, N);
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

template <int D>
int launch_impl(const void* q, const void* k, const void* v, const void* dO, const DqArgs& a, cudaStream_t s) {
    const int BH_kv = a.w.BH, BH = BH_kv / a.w.H_kv * a.w.H, N = a.w.N;
    CUtensorMap tq, tk, tv, tdo;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = make_map_3d(&tq, q, dt, 2, D, N, BH, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, D, N, BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, D, N, BH_kv, 64, kBlk);
    if (rc == 0) rc = make_map_3d(&tdo, dO, dt, 2, D, N, BH, 64, kBlk);
    if (rc != 0) return rc;
    static std::atomic<uint64_t> smem_done;
    cudaError_t e = allow_smem(win_bwd_dq_kernel<D>, Cfg<D>::kSmemAlloc, smem_done);
    int dev = 0, sms = 152;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    // An ordinary launch.  Launched with programmatic serialization, its CTAs taking over the SMs as
    // those of the dK/dV kernel finish (of which dQ needs nothing), a step took 2-3% longer.
    win_bwd_dq_kernel<D><<<a.n_items < sms ? a.n_items : sms, kThreads, Cfg<D>::kSmemAlloc, s>>>(tq, tk, tv, tdo, a);
    return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_bwd_window_dq(const void* q, const void* k, const void* v, const void* dO, void* dq, const WinBwdArgs& a, int d,
                         cudaStream_t s) {
    DqArgs x;
    x.w = a;
    x.dq = dq;
    x.n_items = a.n_kv * (a.BH / a.H_kv * a.H);
    return d == 64 ? launch_impl<64>(q, k, v, dO, x, s) : launch_impl<128>(q, k, v, dO, x, s);
}

}  // namespace fa
