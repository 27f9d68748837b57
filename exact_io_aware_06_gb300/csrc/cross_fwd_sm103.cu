// cross_fwd_sm103.cu -- forward of attention to another sequence's keys (an encoder's states, a prefix
// that requests share) on the sm_103a tensor core (tcgen05 + TMEM + TMA).
//
//     O = softmax(scale Q K^T over the keys j < len_b) V,  lse = m + ln l,
// by the online softmax of the plain forward (fwd_sm103.cu): a running reference maximum, sum and
// unnormalised output a row, lazily rescaled.  Optionally merged with (o_own, lse_own), the same queries'
// attention to other keys: lse = ln(e^lse + e^lse_own), O weighted by e^(lse_x - lse).
#include <type_traits>

#include "cross_fwd.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kThreads = 384;
constexpr int kMaxCtas = 152;

template <int D>
struct Cfg {
    static constexpr int kStages = D == 64 ? 4 : 2;  // 128 KB of K and V either way
    static constexpr int kChunks = D / 64;           // 128-byte swizzle columns per row
    static constexpr int kChunkBytes = 128 * 128;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffO = kOffV + kStages * kTileBytes;  // 4 KB per softmax warp
    static constexpr int kSmemAlloc = kOffO + 8 * 4096 + 1024;
    static constexpr uint32_t kColS = 0, kColO = 256;  // + 128, + D for the second tile
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kIdescS = idesc_bf16(kBM, kBN, false, false);
    static constexpr uint32_t kIdescO = idesc_bf16(kBM, D, false, true);
};
static_assert(Cfg<128>::kSmemAlloc + 1536 <= 232448, "smem");

template <int STAGES>
struct Bars {
    uint64_t q_full, q_free;
    uint64_t kv_full[STAGES], kv_empty[STAGES];
    uint64_t s_full[2], p_full[2], o_done[2];
    uint64_t merge_ml, merge_done;  // one tile: warpgroup 1's state is in shared memory; its O was read
    uint64_t drain;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// 32 columns of this thread's row of the accumulator(s) at `first` (and `second`), weighted.
__device__ __forceinline__ void weighted32(uint32_t first, float w0, uint32_t second, float w1, bool two, float (&x)[32]) {
    uint32_t r[32];
    tmem_ld32(first, r);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(r[e]) * w0;
    if (two) {
        tmem_ld32(second, r);
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(r[e]), w1, x[e]);
    }
}
// x times 1 and the row's own O (when f_own is not 0), as bf16.
__device__ __forceinline__ void store32(const CrossArgs& a, const float (&x)[32], float f_own, size_t at) {
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + at);
    const uint4* own = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o_own) + at);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[8 * g + e];
        if (f_own != 0.f) {
            const uint4 v = own[g];
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[2 * e] = fmaf(__uint_as_float(u[e] << 16), f_own, y[2 * e]);
                y[2 * e + 1] = fmaf(__uint_as_float(u[e] & 0xFFFF0000u), f_own, y[2 * e + 1]);
            }
        }
        out[g] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                     const CrossArgs args) {
    using C = Cfg<D>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) Bars<kStages> bars;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ float merge_m[kBM], merge_l[kBM];

    const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

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
        mbar_init(smem_u32(&bars.merge_ml), 128);
        mbar_init(smem_u32(&bars.merge_done), 128);
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
    Walk walk(args);
    Segment seg;

    // 384 threads x 168 registers at launch: 128 * 120 + 256 * 184 <= 384 * 168
    if (warp < 4) {
        regs_dec<120>();
        if (warp == 0) {
            // ============================================================ TMA producer
            if (lane == 0) {
                const uint32_t qf = smem_u32(&bars.q_full);
                const int q_rows = args.nb > 1 ? args.nb * args.R : kBM;  // of a box
                int gb = 0, kq = 0;  // bundles and segments issued
                bool ok = true;
                const volatile int never = 0;
                while (ok && walk.next(args, seg)) {
                    if (kq > 0 && !mbar_wait(smem_u32(&bars.q_free), (kq - 1) & 1, lim, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    const int n_q = seg.solo ? 1 : 2, bh_kv = seg.b * args.H_kv + seg.h;
                    mbar_arrive_expect_tx(qf, n_q * C::kChunks * q_rows * 128);
                    for (int t = 0; t < n_q; ++t) {
                        const TileRows T = tile_rows(args, seg.b, 2 * seg.pair + t);
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_4d(smem_base + C::kOffQ + t * C::kTileBytes + c * C::kChunkBytes, &tm_q, qf, c * 64, T.r0,
                                        seg.h, T.b);
                    }
                    ++kq;
                    // bundle n = {K of block n (n < seg.n), V of block n - 1 (n >= 1)}
                    for (int n = 0; n <= seg.n; ++n, ++gb) {
                        const int u = gb % kStages;
                        if (gb >= kStages &&
                            !mbar_wait(smem_u32(&bars.kv_empty[u]), ((gb / kStages) & 1) ^ 1, lim, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb = smem_u32(&bars.kv_full[u]);
                        mbar_arrive_expect_tx(fb, ((n < seg.n ? 1 : 0) + (n >= 1 ? 1 : 0)) * C::kTileBytes);
                        if (n < seg.n)
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_3d(smem_base + C::kOffK + u * C::kTileBytes + c * C::kChunkBytes, &tm_k, fb, c * 64,
                                            (seg.k0 + n) * kBN, bh_kv);
                        if (n >= 1)
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_3d(smem_base + C::kOffV + u * C::kTileBytes + c * C::kChunkBytes, &tm_v, fb, c * 64,
                                            (seg.k0 + n - 1) * kBN, bh_kv);
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
                // S in the columns of tile (or warpgroup) t from query tile q and K in slot u
                auto issue_s = [&](int t, int q, int u) {
                    const uint32_t ql = q_lo + q * (C::kTileBytes >> 4), kl = k_lo + u * (C::kTileBytes >> 4);
                    const uint32_t col = tmem + C::kColS + 128 * t;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off16 = ((kk * 32) / 128 * C::kChunkBytes + (kk * 32) % 128) >> 4;
                        if (kk == 0)
                            mma_ss_w<false, -1>(col, ql, kl, kDescHi, C::kIdescS, 0u);
                        else
                            mma_ss_w<false, 1>(col, ql + off16, kl + off16, kDescHi, C::kIdescS);
                    }
                    mma_commit(smem_u32(&bars.s_full[t]));
                };
                auto issue_pv = [&](int t, int u, bool acc) {
                    const uint32_t vl = v_lo + u * (C::kTileBytes >> 4);
                    const uint32_t colO = tmem + C::kColO + D * t, colP = tmem + C::kColS + 128 * t;
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk) {
                        if (kk == 0)
                            mma_ts_w<false, -1>(colO, colP, vl, kDescHi, C::kIdescO, acc ? 1u : 0u);
                        else
                            mma_ts_w<false, 1>(colO, colP + kk * 8, vl + ((kk * 16 * 128) >> 4), kDescHi, C::kIdescO);
                    }
                };
                int gb = 0, kq = 0;
                int c0 = 0, c1 = 0;  // blocks of warpgroup 0 / 1 before the segment
                bool ok = true;
                // Block j of two tiles: P_t V_j, then the next block's scores, tile by tile; the last two
                // blocks run outside the loop, which keeps its body free of branches.
                auto block = [&](int j, int g1, uint32_t p0, uint32_t p1, auto more_c, auto last2_c) -> bool {
                    constexpr bool more = decltype(more_c)::value, last2 = decltype(last2_c)::value;
                    const int u = g1 % kStages;
                    if (!mbar_wait(smem_u32(&bars.kv_full[u]), (g1 / kStages) & 1, lim, &abort_flag)) return false;
                    if (!mbar_wait(smem_u32(&bars.p_full[0]), p0, lim, &abort_flag)) return false;
                    tc_fence_after();
                    issue_pv(0, u, j > 0);
                    if constexpr (more)
                        issue_s(0, 0, u);
                    else
                        mma_commit(smem_u32(&bars.o_done[0]));
                    if (!mbar_wait(smem_u32(&bars.p_full[1]), p1, lim, &abort_flag)) return false;
                    tc_fence_after();
                    issue_pv(1, u, j > 0);
                    if constexpr (more)
                        issue_s(1, 1, u);
                    else
                        mma_commit(smem_u32(&bars.o_done[1]));
                    if constexpr (last2) mma_commit(smem_u32(&bars.q_free));
                    mma_commit(smem_u32(&bars.kv_empty[u]));
                    return true;
                };
                using T = std::true_type;
                using F = std::false_type;
                while (ok && walk.next(args, seg)) {
                    const int n = seg.n;
                    ok = mbar_wait(smem_u32(&bars.q_full), kq & 1, lim, &abort_flag);
                    if (ok) ok = mbar_wait(smem_u32(&bars.kv_full[gb % kStages]), (gb / kStages) & 1, lim, &abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const int u0 = gb % kStages;
                    issue_s(0, 0, u0);
                    if (!seg.solo) issue_s(1, 1, u0);
                    if (n == 1) mma_commit(smem_u32(&bars.q_free));
                    mma_commit(smem_u32(&bars.kv_empty[u0]));
                    if (seg.solo) {
                        // One tile: block i belongs to warpgroup i % 2, whose S, P and O columns it uses.
                        for (int i = 1; i <= n; ++i) {
                            const int g = gb + i, u = g % kStages;
                            ok = mbar_wait(smem_u32(&bars.kv_full[u]), (g / kStages) & 1, lim, &abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            if (i < n) {
                                issue_s(i & 1, 0, u);
                                if (i == n - 1) mma_commit(smem_u32(&bars.q_free));
                            }
                            const int j = i - 1, t = j & 1;
                            ok = mbar_wait(smem_u32(&bars.p_full[t]), ((t ? c1 : c0) + j / 2) & 1, lim, &abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            issue_pv(t, u, j >= 2);
                            if (j + 2 >= n) mma_commit(smem_u32(&bars.o_done[t]));  // the warpgroup's last
                            mma_commit(smem_u32(&bars.kv_empty[u]));
                        }
                        c0 += (n + 1) / 2;
                        c1 += n / 2;
                    } else {
                        int j = 0;
                        for (; j + 2 < n && ok; ++j) ok = block(j, gb + j + 1, (c0 + j) & 1, (c1 + j) & 1, T{}, F{});
                        if (ok && n >= 2) ok = block(n - 2, gb + n - 1, (c0 + n - 2) & 1, (c1 + n - 2) & 1, T{}, T{});
                        if (ok) ok = block(n - 1, gb + n, (c0 + n - 1) & 1, (c1 + n - 1) & 1, F{}, F{});
                        c0 += n;
                        c1 += n;
                    }
                    gb += n + 1;
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
        const int row = wq * 32 + lane;  // of the tile
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t colS = C::kColS + 128 * t, colO = C::kColO + D * t;
        const float c = args.c_log2;
        const bool c_pos = c >= 0.f;
        const uint32_t mask_bits = c_pos ? 0xff800000u : 0x7f800000u;  // -inf after the multiply by c
        int gb = 0;          // bundles before the segment
        int gj = 0, kd = 0;  // this warpgroup's blocks before the segment, and segments with any
        int ns = 0;          // solo segments
        bool ok = true;
        while (ok && walk.next(args, seg)) {
            const int n = seg.n, step = seg.solo ? 2 : 1;
            const TileRows T = tile_rows(args, seg.b, 2 * seg.pair + (seg.solo ? 0 : t));
            const bool busy = wq * 32 < T.rows;  // some of the warp's rows are in use
            float m_ref = -INFINITY, l = 0.f;
            int i = 0;
            for (int j = seg.solo ? t : 0; j < n; j += step, ++i) {
                ok = mbar_wait(smem_u32(&bars.s_full[t]), (gj + i) & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const int kv0 = (seg.k0 + j) * kBN, valid = seg.len - kv0;
                if (valid < kBN && seg.len < args.N_kv) {
                    // What the caller left behind the sequence's end (an infinity, a NaN) would reach O as
                    // 0 * V: the block's rows of V from there on are made zeros before P V.
                    const int g = gb + j + 1, u = g % kStages;
                    ok = mbar_wait(smem_u32(&bars.kv_full[u]), (g / kStages) & 1, lim, &abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t vb = smem_base + C::kOffV + u * C::kTileBytes;
                    const int r1 = min(kBN, args.N_kv - kv0);
                    for (int x = max(valid, 0) * 8 + (warp % 4) * 32 + lane; x < r1 * 8; x += 128)
#pragma unroll
                        for (int ch = 0; ch < C::kChunks; ++ch)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + ch * C::kChunkBytes + x * 16), "r"(0)
                                         : "memory");
                    fence_proxy_async_smem();
                }
                if (busy)
                    softmax_block<D, kBN>(lane_base, colS, colS, colO, c, c_pos, mask_bits, valid - 1, -1, 0, i == 0, m_ref, l,
                                          [] {}, [] { return true; });
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.p_full[t]));
            }
            gj += i;
            gb += n + 1;
            if (ok && i > 0) {
                ok = mbar_wait(smem_u32(&bars.o_done[t]), kd & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                ++kd;
            }
            if (!ok) break;
            tc_fence_after();
            float w0 = 1.f, w1 = 0.f;
            bool two = false;
            if (seg.solo) {
                // Two states over disjoint keys: m = max(m_0, m_1), l and O weighted by 2^(m_t - m).
                if (t == 1) {
                    merge_m[row] = m_ref;
                    merge_l[row] = l;
                    mbar_arrive(smem_u32(&bars.merge_ml));
                    // O_1 stays in TMEM until warpgroup 0 has read it
                    ok = mbar_wait(smem_u32(&bars.merge_done), ns & 1, lim, &abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    ++ns;
                    continue;
                }
                ok = mbar_wait(smem_u32(&bars.merge_ml), ns & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                ++ns;
                if (!ok) break;
                tc_fence_after();
                two = n >= 2;
                const float m1 = merge_m[row], l1 = merge_l[row], mm = fmaxf(m_ref, m1);
                w0 = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - mm);
                w1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - mm);
                l = w0 * l + w1 * l1;
                m_ref = mm;
            }
            // O_t is read before this warp publishes the next segment's first P, so the next segment's
            // first P V (which overwrites O_t) comes after these loads
            const bool there = row < T.rows;
            const uint32_t col1 = C::kColO + D;
            if (!seg.whole()) {
                const int slot = static_cast<int>(blockIdx.x) * 2 + seg.slot();
                float* part = args.part + slot * part_floats(D, args.part_rows);
                const int at = row + (seg.solo ? 0 : t * kPartTile);
                if (busy) {
#pragma unroll
                    for (int q4 = 0; q4 < D / 32; ++q4) {
                        float x[32];
                        weighted32(lane_base + colO + 32 * q4, w0, lane_base + col1 + 32 * q4, w1, two, x);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            reinterpret_cast<float4*>(part)[static_cast<size_t>(8 * q4 + e) * args.part_rows + at] =
                                make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                    }
                    float* ml = part + static_cast<size_t>(args.part_rows) * D;
                    ml[at] = m_ref;
                    ml[args.part_rows + at] = l;
                }
            } else {
                const size_t out = there ? global_row(args, T, seg.h, row) : 0;
                const RowEnd e = row_end(args, m_ref, l, out, there);
                if (!seg.solo && args.nb == 1 && args.o_own == nullptr) {
                    store_rows<D>(tm_o, smem_base + C::kOffO + (warp - 4) * 4096, lane_base + colO, e.f, T.r0 + wq * 32,
                                  T.b * args.H_kv + seg.h, args.R);
                } else if (busy) {
#pragma unroll
                    for (int q4 = 0; q4 < D / 32; ++q4) {
                        float x[32];
                        weighted32(lane_base + colO + 32 * q4, w0 * e.f, lane_base + col1 + 32 * q4, w1 * e.f, two, x);
                        if (there) store32(args, x, e.f_own, out * D + 32 * q4);
                    }
                }
                if (there && args.lse != nullptr) args.lse[out] = e.lse;
            }
            if (seg.solo) {
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.merge_done));
            }
        }
        if (!ok && lane == 0) record_timeout(args.ctl, &abort_flag);
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

// Items that were cut: CTA boundary c = blockIdx.x + 1, if it is the first inside its item, adds up the
// item's parts in order, kJoinRows of its rows at a time (blockIdx.y).  A warp takes 8 rows x 32 columns:
// 128-byte runs of the parts, 64-byte runs of the result.
constexpr int kJoinRows = 32;
template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 8) cross_join_kernel(const CrossArgs args) {
    griddep_wait();
    griddep_launch_dependents();
    const int c = static_cast<int>(blockIdx.x) + 1;
    const long long total = total_units(args), u = first_unit(args, total, c);
    if (u >= total) return;
    const UnitPlace p = unit_place(args, u);
    if (p.kb == 0 || u - p.kb < first_unit(args, total, c - 1)) return;
    const int blocks = cross_blocks(cross_length(args, p.b));
    const int h = p.item / args.n_pairs, pair = p.item - h * args.n_pairs;
    int last = c;  // the last CTA with a part of the item
    while (first_unit(args, total, last + 1) < u - p.kb + blocks) ++last;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int kCols = D / 32;
    const int vec = warp % kCols * 4 + lane / 8;  // 8 columns
    const int at = blockIdx.y * kJoinRows + warp / kCols * 8 + lane % 8;
    const int tile = 2 * pair + at / kPartTile;
    if (tile >= args.tiles || at >= args.part_rows) return;
    const TileRows T = tile_rows(args, p.b, tile);
    const int row = at % kPartTile;
    if (row >= T.rows) return;
    const size_t size = part_floats(D, args.part_rows);
    auto part = [&](int cta) { return args.part + (cta * 2 + (cta < c ? 1 : 0)) * size; };
    const size_t ml = static_cast<size_t>(args.part_rows) * D + at;
    float m = -INFINITY;
    for (int k = c - 1; k <= last; ++k) m = fmaxf(m, part(k)[ml]);
    float l = 0.f, x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll 4
    for (int k = c - 1; k <= last; ++k) {
        const float* src = part(k);
        const float mk = src[ml], lk = src[ml + args.part_rows];
        const float w = mk == -INFINITY ? 0.f : exp2f(mk - m);
        const float4* o = reinterpret_cast<const float4*>(src) + static_cast<size_t>(2 * vec) * args.part_rows + at;
        const float4 y = o[0], z = o[args.part_rows];
        l = fmaf(w, lk, l);
        x[0] = fmaf(w, y.x, x[0]), x[1] = fmaf(w, y.y, x[1]), x[2] = fmaf(w, y.z, x[2]), x[3] = fmaf(w, y.w, x[3]);
        x[4] = fmaf(w, z.x, x[4]), x[5] = fmaf(w, z.y, x[5]), x[6] = fmaf(w, z.z, x[6]), x[7] = fmaf(w, z.w, x[7]);
    }
    const size_t out = global_row(args, T, h, row);
    const RowEnd e = row_end(args, m, l, out, true);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= e.f;
    if (e.f_own != 0.f) {
        const uint4 v = reinterpret_cast<const uint4*>(args.o_own)[out * (D / 8) + vec];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = fmaf(__uint_as_float(w[i] << 16), e.f_own, x[2 * i]);
            x[2 * i + 1] = fmaf(__uint_as_float(w[i] & 0xFFFF0000u), e.f_own, x[2 * i + 1]);
        }
    }
    reinterpret_cast<uint4*>(args.o)[out * (D / 8) + vec] =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    if (vec == 0 && args.lse != nullptr) args.lse[out] = e.lse;
}

// How a call's rows are tiled and its work dealt, from its sizes alone.
CrossArgs deal(int B, int B_kv, int H, int H_kv, int N_q, int N_kv) {
    CrossArgs a = {};
    a.R = H / H_kv * N_q;
    a.share = B / B_kv;
    a.H_kv = H_kv;
    a.B_kv = B_kv;
    a.N_kv = N_kv;
    a.nb = 1;
    if (a.R <= kBM / 2 && a.share > 1) a.nb = a.share < kBM / a.R ? a.share : kBM / a.R;
    a.tiles_b = (a.R + kBM - 1) / kBM;
    a.tiles = a.nb > 1 ? (a.share + a.nb - 1) / a.nb : a.share * a.tiles_b;
    a.n_pairs = (a.tiles + 1) / 2;
    const int rows = a.nb > 1 ? a.nb * a.R : a.R;  // of a lone tile
    a.part_rows = a.tiles > 1 ? 2 * kBM : round_up(rows < kBM ? rows : kBM, 32);
    const long long items = static_cast<long long>(B_kv) * H_kv * a.n_pairs;
    a.stream = items < 8 * kMaxCtas;
    const long long units = items * ((N_kv + kBN - 1) / kBN);
    a.ctas = static_cast<int>(units < kMaxCtas ? units : kMaxCtas);
    return a;
}

// q or o as [B][H_kv][R][d], read in boxes of `rows` rows of `nb` batches.
int row_map(CUtensorMap* map, const void* base, int D, const CrossArgs& a, int rows, int nb) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr) return -1;
    const cuuint64_t line = static_cast<cuuint64_t>(D) * 2;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.R), static_cast<cuuint64_t>(a.H_kv),
                          static_cast<cuuint64_t>(a.B_kv) * a.share};
    cuuint64_t strides[3] = {line, line * a.R, line * a.R * a.H_kv};
    cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, static_cast<cuuint32_t>(nb)};
    cuuint32_t one[4] = {1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? 0 : static_cast<int>(r);
}

template <int D>
int launch_impl(const void* q, const void* k, const void* v, const CrossArgs& a, cudaStream_t s) {
    const int BH_kv = a.B_kv * a.H_kv;
    CUtensorMap tq, tk, tv, to;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = row_map(&tq, q, D, a, a.nb > 1 ? a.R : kBM, a.nb);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, D, a.N_kv, BH_kv, 64, kBN);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, D, a.N_kv, BH_kv, 64, kBN);
    if (rc == 0) rc = make_map_3d(&to, a.o, dt, 2, D, a.R, static_cast<uint64_t>(BH_kv) * a.share, 64, 32);
    if (rc != 0) return rc;
    static std::atomic<uint64_t> smem_done;
    cudaError_t e = allow_smem(cross_fwd_kernel<D>, Cfg<D>::kSmemAlloc, smem_done);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    CrossArgs x = a;
    if (x.ctas > sms) x.ctas = sms;
    e = launch_pdl(cross_fwd_kernel<D>, dim3(x.ctas), dim3(kThreads), Cfg<D>::kSmemAlloc, s, tq, tk, tv, to, x);
    if (e == cudaSuccess && x.stream && x.ctas > 1)
        e = launch_pdl(cross_join_kernel<D>, dim3(x.ctas - 1, (x.part_rows + kJoinRows - 1) / kJoinRows),
                       dim3(kJoinRows * D / 8), 0, s, x);
    return static_cast<int>(e);
}

}  // namespace

size_t fwd_cross_workspace_bytes(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    const CrossArgs a = deal(B, B_kv, H, H_kv, N_q, N_kv);
    return a.stream && a.ctas > 1 ? 2 * a.ctas * part_floats(d, a.part_rows) * sizeof(float) : 0;
}

int launch_fwd_cross(const void* q, const void* k, const void* v, const int* lengths, const void* o_own,
                     const float* lse_own, void* o, float* lse, void* workspace, int B, int B_kv, int H, int H_kv, int N_q,
                     int N_kv, int d, float c_log2, DevCtl ctl, cudaStream_t s) {
    CrossArgs a = deal(B, B_kv, H, H_kv, N_q, N_kv);
    a.lengths = lengths;
    a.o = o;
    a.lse = lse;
    a.o_own = o_own;
    a.lse_own = lse_own;
    a.part = static_cast<float*>(workspace);
    // a scale of 0 makes all scores 0; the mask multiplies -inf by c, which has to stay -inf
    a.c_log2 = c_log2 == 0.f ? 1e-30f : c_log2;
    a.ctl = ctl;
    return d == 64 ? launch_impl<64>(q, k, v, a, s) : launch_impl<128>(q, k, v, a, s);
}

}  // namespace fa
